"""GPU tests of the serving step's operators at the edges of what their calls
allow: several host threads, refused requests, bad pages, values that are not
finite, scales that differ widely, and closer bounds on the attention's error."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import dsa_sparse_mla_topk_gb300 as dsa
import oracle
import step_reference as ref
import test_gpu_step_ops as ops

pytestmark = pytest.mark.gpu
I32 = torch.int32
SHAPES = [(16, 64, 16), (64, 512, 64)]
both_shapes = pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dsa_sparse_mla_topk_gb300 import build
    build.build()
    oracle.build()
    dsa.load_library()


# ---- batch_layout ------------------------------------------------------------------


def test_layout_large_batches_from_several_threads():
    """Batches past 48 KB of shared memory, of different sizes, from three threads: the
    kernel's limit is one for all of them."""
    errors = []

    def work(R):
        c, n, held, table, free, pages = ops._layout_case(R, 2, 20, 16, seed=R)
        want, _ = ref.batch_layout(c, n, held, table, free, 0, page_size=16, num_pages=pages, capacity=int(n.sum()))
        args = (ops.i32(c), ops.i32(n), ops.i32(held), torch.from_numpy(table).cuda(), ops.i32(free), ops.i32([0]))
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        try:
            for _ in range(2000):
                lay = dsa.batch_layout(*args, page_size=16, num_pages=pages, capacity=int(n.sum()), stream=stream)
            stream.synchronize()
            for k, v in lay._asdict().items():
                assert np.array_equal(ops.host(v), want[k]), (R, k)
        except Exception as e:  # noqa: BLE001
            errors.append((R, repr(e)))

    threads = [threading.Thread(target=work, args=(R,)) for R in (8192, 4000, 6000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_layout_state_does_not_keep_the_token_arrays():
    """A loop keeps the lengths, pages and counts: a few words a request, and no more than 64 KB
    of the step's tokens."""
    c, n, held, table, free, pages = ops._layout_case(50, 60, 100, 16, seed=8)
    a = (ops.i32(c), ops.i32(n), ops.i32(held), torch.from_numpy(table).cuda(), ops.i32(free), ops.i32([0]))
    for run in (lambda f: f(), ops._without_cpp):
        for cap in (3001, 5460, 5461, 100_001):  # 64 KB of token arrays: 5,461 tokens
            lay = run(lambda: dsa.batch_layout(*a, page_size=16, num_pages=pages, capacity=cap))
            for name in ("cu_q", "ctx_len", "pages_held", "free_used"):
                assert getattr(lay, name).untyped_storage().nbytes() <= 64 * 1024 + 4 * (3 * 50 + 2), name
            want, _ = ref.batch_layout(c, n, held, table, free, 0, page_size=16, num_pages=pages, capacity=cap)
            for k, v in lay._asdict().items():
                assert v.is_contiguous() and np.array_equal(ops.host(v), want[k]), k


def test_layout_pages_given_back_to_the_list():
    """A finished request's pages, written over the last taken entries of the list, are the
    next ones that a request gets, and no page is two requests'."""
    page, pages = 16, 12
    free = ops.i32([7, 3, 9, 1, 11, 5])
    table = torch.full((3, 4), -1, dtype=I32, device="cuda")
    zero = ops.i32([0, 0, 0])
    kw = dict(page_size=page, num_pages=pages, capacity=100)
    a = dsa.batch_layout(zero, ops.i32([20, 40, 0]), zero, table, free, ops.i32([0]), **kw)
    assert table.tolist() == [[7, 3, -1, -1], [9, 1, 11, -1], [-1] * 4] and a.free_used.tolist() == [5]
    used = a.free_used.clone()  # request 0 ends
    free[3:5] = table[0, :2]
    used -= 2
    table[0] = -1
    ctx, held = a.ctx_len.clone(), a.pages_held.clone()
    ctx[0] = held[0] = 0
    st = torch.zeros(1, dtype=I32, device="cuda")
    b = dsa.batch_layout(ctx, ops.i32([0, 0, 33]), held, table, free, used, dev_status=st, **kw)
    assert table.tolist() == [[-1] * 4, [9, 1, 11, -1], [7, 3, 5, -1]] and int(st) == 0
    assert b.free_used.tolist() == [6] and b.pages_held.tolist() == [0, 3, 3]
    assert b.slot.tolist()[:33] == [7 * page + x for x in range(16)] + [3 * page + x for x in range(16)] + [5 * page]


# ---- qk_norm_rope ------------------------------------------------------------------


def test_norm_rope_same_slot_twice_leaves_the_other_slots_right():
    """Two rows aimed at one slot leave some mixture there, and everything else as written."""
    T, d = 40, 576
    q, k, g = ops._qk_inputs(T, 2, 1, d, torch.bfloat16, seed=5)
    slot = torch.arange(T, dtype=I32) + 3
    slot[7] = slot[30]
    kv = torch.full((T + 6, d), 0xAA, dtype=torch.uint8, device="cuda")
    sc = torch.full((T + 6,), -1.0, device="cuda")
    dsa.qk_norm_rope(q, k, None, None, d_rope=0, slot=slot.cuda(), kv=kv, kv_scale=sc)
    rows = [t for t in range(T) if t not in (7, 30)]
    ops._check_codes(kv[slot[rows].long().cuda()], sc[slot[rows].long().cuda()], ops.host(k.double())[rows, 0])
    for at in (0, 1, 2, 10, T + 3, T + 4, T + 5):  # no row's
        assert (kv[at] == 0xAA).all() and sc[at] == -1.0


# ---- chunk_mla ---------------------------------------------------------------------


@both_shapes
@pytest.mark.parametrize("bad", [-1, -2, -3, -2**31, 1 << 20, 2**31 - 1])
def test_chunk_any_page_id_out_of_range_is_told(shape, bad):
    c = ops._chunk_case(*shape, [200, 100], [2, 1], 64, seed=9)
    c["table"][0, 1] = bad
    want = ops._chunk_ref(dict(c, table=torch.where(c["table"] == bad, torch.tensor(1 << 20, dtype=I32), c["table"])))
    for splits in (1, 3):
        out, lse, st = ops._run_chunk(c, splits)
        assert st == dsa.DEV_BAD_PAGE
        ops._check_chunk(out, lse, want)


@both_shapes
@pytest.mark.parametrize("size", [2.0**-133, 2.0**-125, 2.0**-121, 2.0**-110, 3.3e38])
def test_chunk_smallest_and_largest_queries(shape, size):
    """One element of a head's query is not zero: next to the type's smallest value the
    result is the mean of the visible rows; next to the largest, the one row that it picks."""
    c = ops._chunk_case(*shape, [300, 130], [2, 1], 64, seed=3)
    c["q"][0] = 0
    c["q"][0, :, 0] = size
    assert float(c["q"][0, 0, 0]) != 0 and np.isfinite(float(c["q"][0, 0, 0]))
    want = ops._chunk_ref(c)
    for splits in (1, 3, 12):
        out, lse, st = ops._run_chunk(c, splits)
        assert st == 0
        if size < 1:
            ops._check_chunk(out, lse, want)
        else:  # (an lse of 1e37 has no absolute bound: its own rounding and two products')
            ops._check_chunk(out, torch.zeros_like(lse), (want[0], np.zeros_like(want[1]), *want[2:]))
            assert (np.abs(ops.host(lse) - want[1]) <= 2.0**-20 * np.abs(want[1]) + 1e-3).all()


@both_shapes
def test_chunk_nan_and_infinite_queries(shape):
    """Their heads are NaN, out and lse, for every number of splits; the others exact."""
    c = ops._chunk_case(*shape, [300, 130], [2, 2], 64, seed=3, pad=1)
    want = ops._chunk_ref(c)
    clean = {S: ops._run_chunk(c, S) for S in (1, 3, 8, 12)}
    heads = {0: (3, float("nan")), 1: (2, float("inf")), 2: (0, float("-inf"))}
    for t, (h, v) in heads.items():
        c["q"][t, h, 5] = v
    c["q"][1, 4, shape[1] + 1] = float("nan")  # in the rope part, beside an infinity in the token
    bad = np.zeros(c["q"].shape[:2], dtype=bool)
    for t, (h, _) in heads.items():
        bad[t, h] = True
    bad[1, 4] = True
    for splits in clean:
        out, lse, st = ops._run_chunk(c, splits)
        o, n = ops.host(out.float()), ops.host(lse)
        assert st == 0 and np.isnan(o[bad]).all() and np.isnan(n[bad]).all()
        assert not np.isnan(o[~bad]).any() and not np.isnan(n[~bad]).any()
        keep = ~bad
        fixed = torch.where(torch.from_numpy(bad).cuda()[..., None], clean[splits][0], out)
        ops._check_chunk(fixed, torch.where(torch.from_numpy(bad).cuda(), clean[splits][1], lse), want)
        assert keep[-1].all() and (o[-1] == 0).all() and np.isneginf(n[-1]).all()


@both_shapes
@pytest.mark.parametrize("what", ["scale", "code"])
@pytest.mark.parametrize("where", [0, 77, 299])
def test_chunk_nan_in_a_visible_row(shape, what, where):
    """Every token that sees it is NaN, out and lse, for every number of splits."""
    c = ops._chunk_case(*shape, [300, 130], [3, 2], 64, seed=3)
    want = ops._chunk_ref(c)
    slot = int(c["table"][0, where // 64]) * 64 + where % 64
    if what == "scale":
        c["sc"][slot] = float("nan")
    else:
        c["kv"][slot, :] = 0x7F
    hit = (c["req"] == 0).numpy() & (c["pos"].numpy() >= where)
    assert hit.any() and not hit.all()
    for splits in (1, 2, 3, 8, 12):
        out, lse, st = ops._run_chunk(c, splits)
        assert st == 0 and torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
        ops._check_chunk(out[~hit], lse[~hit], [x[~hit] for x in want])


def test_combine_splits_of_nan():
    """A head whose splits are all NaN is NaN, not empty; one NaN split is enough."""
    o, n = torch.zeros((3, 2, 4, 8), device="cuda"), torch.zeros((3, 2, 4), device="cuda")
    n[:, 0, 1] = float("nan")
    n[1, 0, 2] = float("nan")
    n[:, 1, 3] = float("-inf")
    n[0, 1, 0], n[1:, 1, 0] = float("nan"), float("-inf")
    out, lse = dsa.combine(o, n)
    bad = torch.zeros((2, 4), dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[0, 2] = bad[1, 0] = True
    assert torch.equal(torch.isnan(lse), bad) and torch.isneginf(lse[1, 3])
    assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(out).any(-1), bad)


def _split_q(q, heads):
    """The query as the kernel multiplies it, fp64: 64 heads, two E4M3 numbers of the
    head scaled to 2^8; 16 heads, fp16 of the token scaled to 2^14."""
    top = q.float().abs().amax(2 if heads == 64 else (1, 2), keepdim=True)
    e = torch.frexp(top)[1]
    y = torch.ldexp(q.float(), (8 if heads == 64 else 14) - e).half()
    if heads == 64:
        hi = y.to(torch.float8_e4m3fn)
        lo = (y - hi.half()).to(torch.float8_e4m3fn)
        y = hi.double() + lo.double()
    return torch.ldexp(y.double(), e - (8 if heads == 64 else 14))


def _close_bounds(c):
    """Oracle, and the bounds of the weights as they are stated (P' = p s F as E4M3 + E5M2
    with the head's largest at 16 or more; 16 heads: fp16 with the largest scale at 2^11):
      elements  2^-8 of the result (its own rounding), 2^-8 + 2^-11 + 2^-12 of A = sum_j
                softmax_j |x_j| (the two parts; fp16 before the split; fp32 sums), and
                2^-14 of a unit below 2^-6: 2^-18 M sum_j |code_j|, M the head's largest
                softmax_j s_j.  16 heads: 2^-11 and 2^-12 of A, 2^-25 of a unit below
                2^-14: 2^-36 s_max sum_j |code_j|.
      L2        the rounding of the result, and of independent weights: 1.30e-3 (16 heads
                2.1e-4) root mean square of the formats over their range, 1.4e-3 (2.5e-4)
                with the smaller weights, times G = sqrt(sum_j (softmax_j x_j)^2); a tenth
                above for the draw.  (With a bit less in a weight 1.30e-3 is 2.54e-3.)
      lse       what the query's own split moves it by, 36 additions of partial products
                with 2^-22 of sum_d |q_d x_d| scale each, and 2^-20 for the rest."""
    o, l, A, _ = ops._chunk_ref(c)
    n, H, dl = o.shape
    big = H == 64
    x = (c["kv"].view(torch.float8_e4m3fn).double() * c["sc"].double()[:, None]).numpy()
    code = c["kv"].view(torch.float8_e4m3fn).double().abs().numpy()
    qs = _split_q(c["q"], H).numpy()
    tol = 2.0**-8 * np.abs(o) + ((2.0**-8 if big else 0) + 2.0**-11 + 2.0**-12) * A
    G2, ltol = 0.0, np.zeros_like(l)
    for t in range(n):
        if c["req"][t] < 0 or c["pos"][t] < 0:
            continue
        p = np.arange(int(c["pos"][t]) + 1)
        slot = c["table"].numpy()[c["req"][t], p // c["page"]].astype(np.int64) * c["page"] + p % c["page"]
        q, v, sc = c["q"][t].double().numpy(), x[slot], np.abs(c["sc"].double().numpy()[slot])
        w = np.exp((q @ v.T) * c["scale"] - l[t][:, None])
        if big:
            tol[t] += 2.0**-18 * (w * sc).max(1)[:, None] * code[slot][:, :dl].sum(0)
        else:
            tol[t] += 2.0**-36 * sc.max() * code[slot][:, :dl].sum(0)
        G2 += ((w**2) @ (v[:, :dl]**2)).sum()
        z = (qs[t] @ v.T) * c["scale"]
        m = z.max(1)
        near = m + np.log(np.exp(z - m[:, None]).sum(1))
        mass = (np.abs(q) @ np.abs(v).T).max(1) * abs(c["scale"])
        ltol[t] = np.abs(near - l[t]) + 36 * 2.0**-22 * mass + 2.0**-20 * (1 + np.abs(l[t]))
    own = torch.from_numpy(o).to(torch.bfloat16).double().numpy() - o
    norm = 1.1 * np.sqrt((own**2).sum() + (1.4e-3 if big else 2.5e-4)**2 * G2)
    return o, l, tol, norm, ltol


def _check_close(out, lse, bounds):
    o, l, tol, norm, ltol = bounds
    got, gl = ops.host(out.double()), ops.host(lse.double())
    assert (np.abs(got - o) <= tol).all(), float((np.abs(got - o) - tol).max())
    assert np.linalg.norm(got - o) <= norm, (np.linalg.norm(got - o) / np.linalg.norm(o), norm / np.linalg.norm(o))
    seen = ~np.isneginf(l)
    assert np.array_equal(seen, ~np.isneginf(gl)) and (np.abs(gl[seen] - l[seen]) <= ltol[seen]).all()


@both_shapes
@pytest.mark.parametrize("lens,new,sharp", [([700, 130], [3, 4], 1.0), ([3000], [2], 1.0), ([900, 64], [4, 2], 3.0),
                                            ([2000], [3], 0.1), ([1], [1], 1.0)], ids=str)
def test_chunk_error_is_that_of_the_stated_weights(shape, lens, new, sharp):
    c = ops._chunk_case(*shape, lens, new, 64, seed=sum(lens), sharp=sharp, pad=1)
    bounds = _close_bounds(c)
    for splits in (1, 3, 12):
        out, lse, st = ops._run_chunk(c, splits)
        assert st == 0
        _check_close(out, lse, bounds)


@both_shapes
def test_chunk_one_head_with_far_larger_queries(shape):
    """A head's query 2^12 times the others' takes none of their bits."""
    c = ops._chunk_case(*shape, [500, 90], [3, 2], 64, seed=23)
    c["q"][:, 5] *= 2.0**12
    bounds = _close_bounds(c)
    for splits in (1, 3, 12):
        _check_close(*ops._run_chunk(c, splits)[:2], bounds)


@pytest.mark.parametrize("shape,log2", [(s, x) for s in SHAPES for x in (10, 12, 14, 20, 22, 40) if s[0] == 64 or x <= 24],
                         ids=lambda v: f"h{v[0]}" if isinstance(v, tuple) else str(v))
@pytest.mark.parametrize("at", [0, 150, 299])
def test_chunk_a_row_of_a_huge_scale_that_weighs_nothing(shape, log2, at):
    """One row's scale is 2^10 to 2^40 times the others', and its logit so low that it does
    not count: the others' weights keep their bits (16 heads: up to 2^24, as documented)."""
    c = ops._chunk_case(*shape, [300, 70], [1, 2], 64, seed=4)
    slot = int(c["table"][0, at // 64]) * 64 + at % 64
    c["sc"][slot] = c["sc"].max() * 2.0**log2
    c["kv"][slot] = 0
    c["kv"][slot, -1] = 0x38  # 1
    c["q"][:, :, -1] = -40.0
    bounds = _close_bounds(c)
    for splits in (1, 2, 5, 12):
        out, lse, st = ops._run_chunk(c, splits)
        assert st == 0
        _check_close(out, lse, bounds)


@both_shapes
def test_chunk_heads_that_look_at_rows_of_different_scales(shape):
    """Scales over 2^16 (16 heads: 2^12) along the context; each head's query picks another
    stretch of it: every head has its own largest weight."""
    span = 16 if shape[0] == 64 else 12
    c = ops._chunk_case(*shape, [1024], [2], 64, seed=14)
    pos_of = torch.zeros(len(c["sc"]))
    for j, p in enumerate(c["table"][0].tolist()):
        pos_of[p * 64:(p + 1) * 64] = torch.arange(64) + 64 * j
    part = (pos_of / 128).long().clamp(max=7)  # eight stretches, each a direction of the rope part
    scale = torch.exp2(-part.float() * span / 8)
    c["sc"] = torch.full_like(c["sc"], 2.0**-6) * scale
    c["kv"][:, shape[1]:] = 0
    c["kv"][torch.arange(len(part)), shape[1] + part] = 0x78  # 256
    c["q"] = c["q"] * 2.0**-9
    for h in range(shape[0]):
        c["q"][:, h, shape[1] + h % 8] = float(16 / (256 * 2.0**-6 * 2.0**(-(h % 8) * span / 8) * c["scale"]))
    c["q"] = c["q"].to(torch.bfloat16)
    bounds = _close_bounds(c)
    for splits in (1, 4):
        _check_close(*ops._run_chunk(c, splits)[:2], bounds)


@both_shapes
def test_chunk_live_tokens_only_choose_the_splits(shape):
    """Any count of live tokens, right or wrong, gives the call's result."""
    c = ops._chunk_case(*shape, [900, 130], [9, 4], 64, seed=31, pad=20)
    want = ops._chunk_ref(c)
    for run in (lambda f: f(), ops._without_cpp):
        for live in (None, 0, 1, 13, 33, 99):
            ops._check_chunk(*run(lambda: ops._run_chunk(c, None, max_ctx=900, live=live))[:2], want)


@both_shapes
@pytest.mark.parametrize("size", [2.0**-133, 2.0**-125, 2.0**-121, 2.0**-110])
def test_sparse_call_smallest_queries(shape, size):
    """The selecting call with the same queries: the mean of the selected rows, not NaN."""
    c = ops._chunk_case(*shape, [300, 130], [2, 1], 64, seed=3)
    c["q"][0] = 0
    c["q"][0, :, 0] = size
    want = ops._chunk_ref(c)
    g = ops._cuda(c)
    idx = np.where(np.arange(300)[None, :] <= c["pos"].numpy()[:, None], np.arange(300)[None, :], -1).astype(np.int32)
    for splits in (1, 2):
        st = torch.zeros(1, dtype=I32, device="cuda")
        r = dsa.sparse_mla_fwd(g["q"], g["kv"], g["sc"], g["table"], g["req"], torch.from_numpy(idx).cuda(),
                               d_latent=shape[1], d_rope=shape[2], page_size=64, softmax_scale=c["scale"],
                               num_splits=splits, dev_status=st)
        out, lse = r if splits == 1 else dsa.combine(*r)
        assert int(st) == 0
        ops._check_chunk(out, lse, want)


# ---- verify_draft and whole steps ----------------------------------------------------


@pytest.mark.parametrize("probs", [True, False])
def test_verify_requests_that_the_layout_refused(probs):
    p, q, tok, cu, ua, us = ops._verify_case(20, 5, 1003, probs, seed=3)
    rows, ctx = p.shape[0], torch.arange(20, dtype=I32, device="cuda") + 7
    cuh = ops.host(cu)
    own = np.repeat(np.arange(20), np.diff(cuh)).astype(np.int32)
    refused = {2, 3, 11, 19}
    for r in refused:
        own[cuh[r]:cuh[r + 1]] = -1
    own[cuh[6]] = 5       # another request's: told
    own[cuh[8] + 1:cuh[9]] = -9  # not a first row: not looked at
    own = np.concatenate([own, [-1, -1]]).astype(np.int32)  # a longer capacity
    want, wnum, _ = ref.verify_draft(ops.host(p), None if q is None else ops.host(q), ops.host(tok), cuh, ops.host(ua),
                                     ops.host(us), 6)
    gone = sorted(refused | {6})
    want[gone], wnum[gone] = -1, 0
    for run in (lambda f: f(), ops._without_cpp):
        st = torch.zeros(1, dtype=I32, device="cuda")
        t, n, c = run(lambda: dsa.verify_draft(p, tok, cu, ua, us, draft_probs=q, ctx_len=ctx, q_req=ops.i32(own), max_out=6,
                                               dev_status=st))
        assert np.array_equal(ops.host(t), want) and np.array_equal(ops.host(n), wnum)
        assert np.array_equal(ops.host(c), ops.host(ctx) + wnum) and int(st) == dsa.DEV_BAD_INDEX
        with pytest.raises(ValueError):
            run(lambda: dsa.verify_draft(p, tok, cu, ua, us, q_req=ops.i32(own[:rows - 1]), max_out=6))


@pytest.mark.parametrize("why", ["pages", "table"])
def test_a_refused_request_waits_through_the_whole_step(why):
    """Two requests of 16 positions with 3 new tokens each, and a page (or a block table
    row) for the first alone: the second one's length stays 16, it gets no tokens, and
    once there is room its next step attends to rows that were written."""
    H, dl, dr, page, V = 64, 512, 64, 16, 50
    d = dl + dr
    g = torch.Generator().manual_seed(17)
    kv = torch.full((6 * page, d), 0x7F, dtype=torch.uint8, device="cuda")  # NaN until written
    sc = torch.full((6 * page,), float("nan"), device="cuda")
    rows = torch.randn((32, 1, d), generator=g).to(torch.bfloat16).cuda()
    dsa.qk_norm_rope(None, rows, None, None, d_rope=0, slot=torch.arange(32, dtype=I32, device="cuda"), kv=kv, kv_scale=sc)
    cs = torch.from_numpy(ops._tables(64, dr)).cuda()
    wide = 3 if why == "pages" else 1
    tables = [torch.full((2, w), -1, dtype=I32, device="cuda") for w in (wide, 3)]
    for t in tables:
        t[:, 0] = ops.i32([0, 1])
    ctx, held, used = ops.i32([16, 16]), ops.i32([1, 1]), ops.i32([0])
    new = [3, 3] if why == "pages" else [0, 3]
    for step, (table, free) in enumerate(((tables[0], [2] if why == "pages" else [2, 3, 4]), (tables[1], [2, 3, 4]))):
        if step and why == "pages":
            table = tables[0]
        st = torch.zeros(1, dtype=I32, device="cuda")
        lay = dsa.batch_layout(ctx, ops.i32(new), held, table, ops.i32(free), used, page_size=page, num_pages=6,
                               capacity=7, dev_status=st)
        q = torch.randn((7, H, d), generator=g).to(torch.bfloat16).cuda()
        k = torch.randn((7, 1, d), generator=g).to(torch.bfloat16).cuda()
        qo, _ = dsa.qk_norm_rope(q, k, lay.q_pos, cs, d_rope=dr, slot=lay.slot, kv=kv, kv_scale=sc)
        out, lse = dsa.chunk_mla(qo, kv, sc, table, lay.q_req, lay.q_pos, d_latent=dl, d_rope=dr, page_size=page,
                                 softmax_scale=d**-0.5)
        p = torch.softmax(torch.randn((7, V), generator=g), 1).cuda()
        tok = torch.zeros(7, dtype=I32, device="cuda")
        before = ctx
        tokens, num, ctx = dsa.verify_draft(p, tok, lay.cu_q, torch.zeros(7, device="cuda"),
                                            torch.rand(2, generator=g).cuda(), q_req=lay.q_req, ctx_len=before, max_out=3)
        live = ops.host(lay.q_req) >= 0
        assert torch.isfinite(out).all() and np.isfinite(ops.host(lse)[live]).all()
        ran = [new[0] > 0, step == 1]
        assert int(st) == (0 if step else dsa.DEV_NO_PAGES if why == "pages" else dsa.DEV_BAD_INDEX)
        for r in range(2):
            # (u = 0 takes every draft: a token out for each one in)
            assert int(num[r]) == (new[r] if ran[r] else 0) and (not ran[r]) == bool((tokens[r] == -1).all())
            assert int(ctx[r]) == int(before[r]) + int(num[r])
            assert int(lay.ctx_len[r]) == int(before[r]) + (new[r] if ran[r] else 0)
        # every position that attention may read from now on lies on a page the request holds
        assert (ops.host(lay.pages_held) * page >= ops.host(ctx)).all()
        held, used = lay.pages_held, lay.free_used
        new = [1, 3]
        if step == 0:
            assert int(ctx[1]) == 16


# ---- errors ------------------------------------------------------------------------


def test_a_refused_launch_leaves_no_error_behind():
    """A launch that the runtime refuses (the legacy stream while a blocking stream is
    captured) comes back as a status, and the next, unrelated check finds nothing."""
    rt = ctypes.CDLL("libcudart.so.13")
    c, n, held, table, free, pages = ops._layout_case(9, 6, 100, 16, seed=11)
    lay = (ops.i32(c), ops.i32(n), ops.i32(held), torch.from_numpy(table).cuda(), ops.i32(free), ops.i32([0]))
    out = dsa.BatchLayout(*[torch.empty(m, dtype=I32, device="cuda") for m in (10, 70, 70, 70, 9, 9, 1)])
    p, q, tok, cu, ua, us = ops._verify_case(3, 2, 100, True, seed=1)
    vo = dict(tokens=torch.empty((3, 3), dtype=I32, device="cuda"), num_out=torch.empty(3, dtype=I32, device="cuda"))
    calls = [lambda: dsa.batch_layout(*lay, page_size=16, num_pages=pages, capacity=70, out=out),
             lambda: dsa.verify_draft(p, tok, cu, ua, us, draft_probs=q, max_out=3, **vo)]
    for f in calls:
        f()
    for shape in SHAPES:
        ch = ops._cuda(ops._chunk_case(*shape, [300, 100], [3, 2], 64, seed=10))
        buf = dict(out=torch.empty((5, shape[0], shape[1]), dtype=torch.bfloat16, device="cuda"),
                   lse=torch.empty((5, shape[0]), device="cuda"))
        calls.append(lambda ch=ch, buf=buf, shape=shape: dsa.chunk_mla(
            ch["q"], ch["kv"], ch["sc"], ch["table"], ch["req"], ch["pos"], d_latent=shape[1], d_rope=shape[2],
            page_size=64, softmax_scale=0.04, num_splits=2, buffers=buf))
        calls[-1]()
    torch.cuda.synchronize()
    assert torch.cuda.current_stream().cuda_stream == 0 and rt.cudaGetLastError() == 0
    for i, f in enumerate(calls):
        s, g = ctypes.c_void_p(), ctypes.c_void_p()
        assert rt.cudaStreamCreate(ctypes.byref(s)) == 0
        assert rt.cudaStreamBeginCapture(s, 0) == 0
        with pytest.raises(dsa.DsaError) as e:
            f()
        left = rt.cudaPeekAtLastError()
        rt.cudaStreamEndCapture(s, ctypes.byref(g))
        rt.cudaStreamDestroy(s)
        rt.cudaGetLastError()
        assert e.value.status == 4 and left == 0, (i, left)
    for f in calls:  # as before
        f()
    torch.cuda.synchronize()
