"""GPU tests of the serving step's operators (batch_layout, qk_norm_rope,
chunk_mla, verify_draft) against plain 64-bit definitions.

Tolerances, each from the arithmetic:
  bf16 / fp16 results  half a step of the type, 2^-8 / 2^-11 of the value, plus
      2^-16 of the row's largest value for the fp32 work (sums of up to 1,024
      squares in at most 130 sequential additions, 130 * 2^-24 < 2^-16), and
      2^-25 for fp16 subnormals.
  E4M3 codes           half a step, 2^-4 of the value, or 2^-10 scales below the
      normal range, plus the fp32 term.
  attention            half a bf16 step of the output, plus the weights' rounding:
      on the tensor cores a weight is E4M3 + 8 bits, relative error at most
      2^-7, so 2^-7 of A = sum_p softmax_p |x_p|, plus 2^-12 of A for fp32 sums.
      Below 2^-14 the weight's second part (E5M2) is subnormal: steps of 2^-16,
      an absolute error of at most 2^-17.  In these units a row of weight p (1 at
      the head's reference) and scale s weighs p s 2^E, with s_max 2^E >= 16, and l >=
      1 (the reference is one of the logits): row j adds at most 2^-17 |code_j| 2^-E
      <= 2^-21 s_max |code_j| to the output.  (An emulation of this rounding in numpy
      gives the kernel's largest excess over the first two terms, 0.00182809 on
      the growing scales below, to eight digits.)  The small head shape's weights are
      fp16, 2^-11: within the first two terms.
"""
import numpy as np
import pytest
import torch

import dsa_sparse_mla_topk_gb300 as dsa
import oracle
import step_reference as ref
from dsa_sparse_mla_topk_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dsa_sparse_mla_topk_gb300 import build
    build.build()
    oracle.build()
    dsa.load_library()


def host(t):
    return t.detach().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


# ---- batch_layout ------------------------------------------------------------------


def _layout_case(R, new, ctx, page, seed, num_free=None, extra=1):
    g = np.random.default_rng(seed)
    c = g.integers(0, ctx + 1, R).astype(np.int32)
    n = g.integers(0, new + 1, R).astype(np.int32)
    held = (-(-c // page) + g.integers(0, extra + 1, R)).astype(np.int32)
    stride = int(-(-(ctx + new) // page) + extra)
    perm = g.permutation(R * stride).astype(np.int32)
    table = perm.reshape(R, stride).copy()
    mask = np.arange(stride)[None, :] < held[:, None]
    free = g.permutation(table[~mask]).astype(np.int32)
    table[~mask] = -1
    if num_free is not None:
        free = free[:num_free]
    return c, n, held, table, free, R * stride


def _run_layout(c, n, held, table, free, used, page, num_pages, capacity, out=None):
    t = torch.from_numpy(table.copy()).cuda()
    st = torch.zeros(1, dtype=I32, device="cuda")
    lay = dsa.batch_layout(i32(c), i32(n), i32(held), t, i32(free), i32([used]), page_size=page, num_pages=num_pages,
                           capacity=capacity, out=out, dev_status=st)
    torch.cuda.synchronize()
    got = {k: host(v) for k, v in lay._asdict().items()}
    got["table"] = host(t)
    want, status = ref.batch_layout(c, n, held, table, free, used, page_size=page, num_pages=num_pages, capacity=capacity)
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    assert int(st) == status
    return got, status


@pytest.mark.parametrize("R,new,ctx,page", [(1, 1, 0, 1), (1, 1, 63, 64), (1, 4000, 100, 16), (7, 5, 100, 16),
                                            (33, 300, 1000, 48), (511, 3, 700, 64), (513, 17, 50, 1), (2000, 9, 90, 7)])
@pytest.mark.parametrize("slack", [0, 5])
def test_layout_matches_the_definition(R, new, ctx, page, slack):
    c, n, held, table, free, pages = _layout_case(R, new, ctx, page, seed=R + new)
    used = min(3, len(free))
    free = np.concatenate([np.full(used, -7, dtype=np.int32), free])
    _run_layout(c, n, held, table, free, used, page, pages, int(n.sum()) + slack)


def test_layout_largest_batch_and_no_tokens():
    c, n, held, table, free, pages = _layout_case(8192, 3, 40, 16, seed=4)
    _run_layout(c, n, held, table, free, 0, 16, pages, int(n.sum()) + 3)
    _run_layout(c, n * 0, held, table, free, 0, 16, pages, 0)
    _run_layout(c, n * 0, held, table, free[:0], 0, 16, pages, 9)


def test_layout_page_shortage_takes_requests_in_order():
    c, n, held, table, free, pages = _layout_case(40, 60, 100, 16, seed=8, num_free=31, extra=0)
    got, status = _run_layout(c, n, held, table, free, 0, 16, pages, int(n.sum()))
    assert status == dsa.DEV_NO_PAGES and 0 < got["free_used"][0] <= 31 and (got["q_req"] == -1).any()
    # requests that need no page go on after the shortage
    c[30:], n[30:], held[30:] = 5, 2, 1
    table[30:, 0] = np.arange(10)
    got, status = _run_layout(c, n, held, table, free, 0, 16, pages, int(n.sum()))
    assert (got["q_req"] == 39).sum() == 2


def test_layout_bad_inputs_leave_the_request_as_it_is():
    c, n, held, table, free, pages = _layout_case(12, 9, 100, 16, seed=3)
    c[2], n[5], held[7] = -4, -1, -2
    c[9] = 16 * table.shape[1]  # no room in the row
    n[9] = 3
    table[10, :] = pages + 5    # held pages that do not exist
    c[10], n[10], held[10] = 3, 4, 2
    _, status = _run_layout(c, n, held, table, free, 0, 16, pages, int(n.clip(0).sum()))
    assert status == dsa.DEV_BAD_QPOS | dsa.DEV_BAD_INDEX | dsa.DEV_BAD_PAGE
    c, n, held, table, free, pages = _layout_case(6, 9, 100, 16, seed=3)
    c[1], n[1] = 2**31 - 5, 10  # positions past 31 bits
    for used in (-1, len(free) + 1):
        _run_layout(c, n, held, table, free, used, 16, pages, int(n.sum()))


def test_layout_tokens_past_the_capacity():
    c, n, held, table, free, pages = _layout_case(20, 9, 100, 16, seed=5)
    n += 1
    got, status = _run_layout(c, n, held, table, free, 0, 16, pages, int(n[:13].sum()) + 2)
    assert status & dsa.DEV_BAD_INDEX and got["cu_q"][-1] == n[:13].sum()


def test_layout_given_outputs_and_captured_graph():
    page = 16
    c, n, held, table, free, pages = _layout_case(9, 6, 100, page, seed=11)
    cap = 9 * 6 + 1
    new = [torch.empty(k, dtype=I32, device="cuda") for k in (10, cap, cap, cap, 9, 9, 1)]
    out = dsa.BatchLayout(*new)
    _run_layout(c, n, held, table, free, 0, page, pages, cap, out=out)
    # unaligned token arrays take the scalar stores
    odd = [torch.empty(k + 1, dtype=I32, device="cuda")[1:] for k in (10, cap, cap, cap, 9, 9, 1)]
    _run_layout(c, n, held, table, free, 0, page, pages, cap, out=dsa.BatchLayout(*odd))
    # a captured step follows lengths that change: two steps in turn, the state double buffered
    ctx, hel, used, nw, t = i32(c), i32(held), i32([0]), i32(n), torch.from_numpy(table.copy()).cuda()
    fr = i32(free)
    a = dsa.BatchLayout(*[torch.empty(k, dtype=I32, device="cuda") for k in (10, cap, cap, cap, 9, 9, 1)])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        dsa.batch_layout(ctx, nw, hel, t, fr, used, page_size=page, num_pages=pages, capacity=cap, out=a)
    torch.cuda.synchronize()
    t.copy_(torch.from_numpy(table))
    with torch.cuda.graph(g):
        dsa.batch_layout(ctx, nw, hel, t, fr, used, page_size=page, num_pages=pages, capacity=cap, out=a)
    wc, wh, wt, wu = c, held, table, 0
    for step in range(3):
        wn = ((n + step) % 4).astype(np.int32)
        nw.copy_(torch.from_numpy(wn))
        g.replay()
        torch.cuda.synchronize()
        want, _ = ref.batch_layout(wc, wn, wh, wt, free, wu, page_size=page, num_pages=pages, capacity=cap)
        for k, v in a._asdict().items():
            assert np.array_equal(host(v), want[k]), (step, k)
        assert np.array_equal(host(t), want["table"])
        ctx.copy_(a.ctx_len), hel.copy_(a.pages_held), used.copy_(a.free_used)
        wc, wh, wt, wu = (want["ctx_len"].astype(np.int32), want["pages_held"].astype(np.int32), want["table"],
                          int(want["free_used"][0]))


# ---- qk_norm_rope ------------------------------------------------------------------


def _tables(max_pos, rope):
    f = 10000.0 ** (-np.arange(0, rope, 2) / max(1, rope))
    a = np.arange(max_pos)[:, None] * f[None, :]
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def _check_rows(got, want, dtype):
    got, top = host(got.double()), np.abs(want).max(-1, keepdims=True)
    tol = (2.0**-8 if dtype == torch.bfloat16 else 2.0**-11) * np.abs(want) + 2.0**-16 * top
    tol = tol + (2.0**-25 if dtype == torch.float16 else 0)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())


def _check_codes(kv, scale, want):
    """kv [n, d] uint8, scale [n] against rows want [n, d]."""
    code = host(kv.view(torch.float8_e4m3fn).double())
    s, top = host(scale.double()), np.abs(want).max(-1)
    assert (np.abs(s - top / 448) <= 2.0**-15 * top / 448).all()
    v = code * s[:, None]
    tol = 2.0**-4 * np.abs(want) + (2.0**-10 * s + 2.0**-14 * top)[:, None]
    assert (np.abs(v - want) <= tol).all()


def _qk_inputs(T, hq, hk, d, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    mag = torch.exp2(torch.randint(-6, 7, (T, 1, 1), generator=g).float())
    wide = (torch.randn((T, hq + hk, d + pad), generator=g) * mag).to(dtype)
    if T > 2:
        wide[1] = 0.0  # an all-zero row
    wide = wide.cuda()
    return wide[:, :hq, :d], wide[:, hq:, :d], g


@pytest.mark.parametrize("d,rope,qn,kn", [(576, 64, 576, 512), (576, 64, 0, 512), (80, 16, 80, 64), (128, 128, 128, 128),
                                          (64, 32, 64, 0), (256, 64, 256, 256), (1024, 512, 1024, 8), (8, 0, 8, 8),
                                          (16, 16, 0, 0), (584, 64, 584, 512), (512, 0, 512, 504)])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_norm_rope_matches_the_definition(d, rope, qn, kn, interleaved, dtype):
    for T, hq, hk in ((1, 1, 1), (5, 3, 2), (67, 16, 1)):
        q, k, g = _qk_inputs(T, hq, hk, d, dtype, seed=d + rope + T, pad=8)
        qw = (1 + 0.3 * torch.randn(qn, generator=g)).cuda() if qn else None
        kw = (1 + 0.3 * torch.randn(kn, generator=g)).cuda() if kn else None
        cs = _tables(97, rope) if rope else None
        pos = torch.randint(0, 97, (T,), generator=g, dtype=I32)
        qo, ko = dsa.qk_norm_rope(q, k, pos.cuda() if rope else None, None if cs is None else torch.from_numpy(cs).cuda(),
                                  d_rope=rope, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=interleaved)
        torch.cuda.synchronize()
        for x, o, w in ((q, qo, qw), (k, ko, kw)):
            want = ref.norm_rope(host(x.double()), None if w is None else host(w), pos.numpy(), cs, rope, interleaved, 1e-5)
            assert o.shape == x.shape and o.is_contiguous()
            _check_rows(o, want, dtype)


@pytest.mark.parametrize("d,rope,kn,T", [(576, 64, 512, 1), (576, 64, 512, 130), (80, 16, 64, 33), (256, 256, 256, 9)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_rope_cache_write(d, rope, kn, T, interleaved):
    q, k, g = _qk_inputs(T, 4, 1, d, torch.bfloat16, seed=T)
    kw = (1 + 0.3 * torch.randn(kn, generator=g)).cuda()
    cs = _tables(500, rope)
    pos = torch.randint(0, 500, (T,), generator=g, dtype=I32)
    slots = 2 * T + 3
    slot = torch.randperm(slots, generator=g)[:T].to(I32)
    if T > 8:
        slot[4] = -1   # not cached
        pos[6] = -1    # padding
    kv = torch.full((slots, d), 0xAA, dtype=torch.uint8, device="cuda")
    sc = torch.full((slots,), -1.0, device="cuda")
    qo = torch.full((T, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=I32, device="cuda")
    _, ko = dsa.qk_norm_rope(q, k, pos.cuda(), torch.from_numpy(cs).cuda(), d_rope=rope, k_weight=kw,
                             interleaved=interleaved, slot=slot.cuda(), kv=kv, kv_scale=sc, q_out=qo, dev_status=st)
    torch.cuda.synchronize()
    assert ko is None and int(st) == 0
    rows = [t for t in range(T) if slot[t] >= 0 and pos[t] >= 0]
    want = ref.norm_rope(host(k.double()), host(kw), pos.clamp(min=0).numpy(), cs, rope, interleaved, 1e-6)[rows, 0]
    at = slot[rows].long()
    _check_codes(kv[at.cuda()], sc[at.cuda()], want)
    rest = torch.ones(slots, dtype=torch.bool)
    rest[at] = False
    assert (kv.cpu()[rest] == 0xAA).all() and (sc.cpu()[rest] == -1).all()
    pad = pos < 0
    assert (qo.cpu()[pad] == 7.0).all()
    # both at once: the cache and 16-bit keys
    _, ko = dsa.qk_norm_rope(None, k, pos.cuda(), torch.from_numpy(cs).cuda(), d_rope=rope, k_weight=kw,
                             interleaved=interleaved, slot=slot.cuda(), kv=kv, kv_scale=sc, k_out=torch.zeros_like(k))
    live = torch.arange(T)[pos >= 0]
    full = ref.norm_rope(host(k.double()), host(kw), pos.clamp(min=0).numpy(), cs, rope, interleaved, 1e-6)
    _check_rows(ko[live.cuda()], full[live.numpy()], torch.bfloat16)


def test_norm_rope_flags_bad_positions_and_slots():
    T, d = 6, 80
    q, k, g = _qk_inputs(T, 2, 1, d, torch.bfloat16, seed=1)
    pos = i32([0, 97, -2, 3, 4, 5])
    slot = i32([0, 1, 2, 99, -5, 3])
    kv = torch.full((8, d), 0xAA, dtype=torch.uint8, device="cuda")
    sc = torch.full((8,), -1.0, device="cuda")
    st = torch.zeros(1, dtype=I32, device="cuda")
    qo = torch.full((T, 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    dsa.qk_norm_rope(q, k, pos, torch.from_numpy(_tables(97, 16)).cuda(), d_rope=16, slot=slot, kv=kv, kv_scale=sc,
                     q_out=qo, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == dsa.DEV_BAD_QPOS | dsa.DEV_BAD_INDEX
    assert (qo[1:3] == 7.0).all() and not (qo[3:] == 7.0).all()
    assert [int(s) == -1 for s in sc] == [False, True, True, False] + [True] * 4


def test_norm_rope_in_place_and_overlaps():
    T, d, rope = 40, 128, 128
    for interleaved in (True, False):
        q, k, g = _qk_inputs(T, 8, 2, d, torch.bfloat16, seed=2)
        q, k = q.contiguous(), k.contiguous()
        pos = torch.randint(0, 50, (T,), generator=g, dtype=I32).cuda()
        cs = torch.from_numpy(_tables(50, rope)).cuda()
        w = (1 + 0.3 * torch.randn(d, generator=g)).cuda()
        kw = dict(d_rope=rope, q_weight=w, k_weight=w, interleaved=interleaved)
        qo, ko = dsa.qk_norm_rope(q, k, pos, cs, **kw)
        q2, k2 = q.clone(), k.clone()
        a, b = dsa.qk_norm_rope(q2, k2, pos, cs, q_out=q2, k_out=k2, **kw)
        assert a is q2 and torch.equal(qo, q2) and torch.equal(ko, k2)
        with pytest.raises(ValueError):
            dsa.qk_norm_rope(q2, k2, pos, cs, q_out=q2, k_out=q2.view(-1)[:T * 2 * d].view(T, 2, d), **kw)
        wide = torch.zeros(T, 8, d + 8, dtype=torch.bfloat16, device="cuda")[:, :, :d]
        with pytest.raises(ValueError):
            dsa.qk_norm_rope(wide, None, pos, cs, q_out=wide, d_rope=rope)


def test_norm_rope_single_tokens_and_heads_with_odd_strides():
    """A dimension of one may have any stride; broadcast tokens may have stride 0."""
    d = 80
    g = torch.Generator().manual_seed(3)
    base = torch.randn((3 * 7 * 81,), generator=g).to(torch.bfloat16).cuda()
    one = base.as_strided((1, 2, d), (13, d, 1))          # one token: its token stride is not looked at
    key = base.as_strided((5, 1, d), (d, 3, 1))           # one head
    same = base.as_strided((5, 2, d), (0, d, 1))          # five times the same token
    for x in (one, key, same):
        for run in (lambda: dsa.qk_norm_rope(x, None, None, None, d_rope=0, q_weight=torch.ones(d, device="cuda")),
                    lambda: _without_cpp(lambda: dsa.qk_norm_rope(x, None, None, None, d_rope=0,
                                                                  q_weight=torch.ones(d, device="cuda")))):
            y = run()[0]
            _check_rows(y, ref.norm_rope(host(x.double()), np.ones(d), None, None, 0, True, 1e-6), torch.bfloat16)


# ---- verify_draft ------------------------------------------------------------------


def _verify_case(R, n, V, probs, seed, pad_cols=0, sharp=3.0):
    g = torch.Generator().manual_seed(seed)
    rows_of = torch.randint(1, n + 2, (R,), generator=g)
    cu = torch.zeros(R + 1, dtype=I32)
    cu[1:] = rows_of.cumsum(0)
    rows = int(cu[-1])
    t = torch.randn((rows, V), generator=g) * sharp
    q = torch.softmax(t + torch.randn((rows, V), generator=g), 1)
    p = torch.softmax(t, 1)
    tok = torch.multinomial(q, 1, generator=g)[:, 0].to(I32)
    ua, us = torch.rand(rows, generator=g), torch.rand(R, generator=g)

    def wide(x):
        b = torch.full((rows, V + pad_cols), float("nan"), device="cuda")
        b[:, :V] = x.cuda()
        return b[:, :V]
    return wide(p), wide(q) if probs else None, tok.cuda(), cu.cuda(), ua.cuda(), us.cuda()


def _run_verify(p, q, tok, cu, ua, us, max_out, ctx=None):
    st = torch.zeros(1, dtype=I32, device="cuda")
    tokens, num, co = dsa.verify_draft(p, tok, cu, ua, us, draft_probs=q, ctx_len=ctx, max_out=max_out, dev_status=st)
    torch.cuda.synchronize()
    want, wnum, status = ref.verify_draft(host(p), None if q is None else host(q), host(tok), host(cu), host(ua),
                                          host(us), max_out)
    assert np.array_equal(host(num), wnum)
    assert np.array_equal(host(tokens), want)
    assert int(st) == status
    if ctx is not None:
        assert np.array_equal(host(co), host(ctx) + wnum)
    return tokens, num, status


@pytest.mark.parametrize("R,n,V", [(1, 0, 1), (1, 1, 2), (3, 4, 127), (16, 8, 1000), (5, 3, 32003), (2, 40, 513),
                                   (70, 2, 4096), (200, 1, 129)])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("pad", [0, 5, 4])
def test_verify_matches_the_definition(R, n, V, probs, pad):
    for seed in range(3):
        case = _verify_case(R, n, V, probs, seed=100 * seed + V + R, pad_cols=pad)
        _run_verify(*case, n + 1, ctx=torch.arange(R, dtype=I32, device="cuda"))


def test_verify_every_border_of_a_row():
    """u on and next to every border of a distribution whose sums are exact."""
    V = 64
    p = torch.full((1, V), 1.0 / V)
    p[0, 5] = 0.0
    p[0, 6] = 2.0 / V
    us = torch.tensor(sorted({min(max(j / V + e, 0.0), 1 - 2.0**-24) for j in range(V) for e in (-2.0**-25, 0.0, 2.0**-24)}))
    R = len(us)
    cu = torch.arange(R + 1, dtype=I32)
    tok = torch.zeros(R, dtype=I32)
    _run_verify(p.expand(R, V).contiguous().cuda(), None, tok.cuda(), cu.cuda(), torch.zeros(R).cuda(), us.cuda(), 3)


def test_verify_accept_borders_and_numbers_out_of_range():
    V, n = 300, 6
    p, q, tok, cu, ua, us = _verify_case(8, n, V, True, seed=9)
    r = torch.arange(p.shape[0], device="cuda")
    t = tok.long()
    ua = (p[r, t] / q[r, t]).clamp(max=1)  # u q next to p: one step to each side and on it
    for e in (0.0, -2.0**-24, 2.0**-24):
        _run_verify(p, q, tok, cu, (ua + e).clamp(min=0), us, n + 1)
    _run_verify(p, q, tok, cu, torch.zeros_like(ua), torch.zeros_like(us), n + 1)
    _run_verify(p, q, tok, cu, torch.ones_like(ua), us.fill_(1 - 2.0**-24), n + 1)
    bad = tok.clone()
    bad[::3] = -1
    bad[1::3] = V
    _, _, status = _run_verify(p, q, bad, cu, ua * 0, us, n + 1)
    assert status == dsa.DEV_BAD_INDEX
    _run_verify(p, None, bad, cu, ua * 0, us, n + 1)


def test_verify_rows_with_nothing_left_and_odd_values():
    V, n = 1500, 3
    p, q, tok, cu, ua, us = _verify_case(6, n, V, True, seed=4)
    # the same distribution: a rejection (u q >= p at u = 1) leaves nothing, the token comes from p
    _run_verify(p, p.clone(), tok, cu, torch.full_like(ua, 1.0), us, n + 1)
    z = torch.zeros_like(p)  # no probability anywhere: the last column
    _run_verify(z, q, tok, cu, ua, us, n + 1)
    _run_verify(z, None, tok, cu, ua, us, n + 1)
    odd = p.clone()
    odd[:, ::7] = float("nan")
    odd[:, 3::11] = -0.5
    _run_verify(odd, q, tok, cu, ua, us, n + 1)


def test_verify_empty_requests_bad_rows_and_short_outputs():
    V, n = 64, 4
    p, q, tok, cu, ua, us = _verify_case(8, n, V, True, seed=5)
    rows = p.shape[0]
    c = host(cu).copy()
    c[6:] = c[5]                   # trailing requests without rows
    _run_verify(p, q, tok, i32(c), ua, us, n + 1)
    c[3], c[7] = rows + 9, -3      # out of range
    _, _, status = _run_verify(p, q, tok, i32(c), ua, us, n + 1)
    assert status == dsa.DEV_BAD_INDEX
    _run_verify(p, q, tok, cu, ua * 0, us, 2)   # more rows than the output holds
    _run_verify(p, q, tok, cu, ua * 0, us, 1)
    tokens, num, _ = dsa.verify_draft(p, tok, cu[:1], ua, us[:0], max_out=3)
    assert tokens.shape == (0, 3) and num.shape == (0,)


def test_verify_same_buffer_for_the_lengths_and_repeatability():
    p, q, tok, cu, ua, us = _verify_case(32, 5, 20000, True, seed=6)
    ctx = torch.arange(32, dtype=I32, device="cuda")
    first = dsa.verify_draft(p, tok, cu, ua, us, draft_probs=q, max_out=6, ctx_len=ctx)
    again = dsa.verify_draft(p, tok, cu, ua, us, draft_probs=q, max_out=6, ctx_len=ctx, ctx_out=ctx)
    assert again[2] is ctx and all(torch.equal(a, b) for a, b in zip(first, again))


# ---- chunk_mla ---------------------------------------------------------------------


def _chunk_case(H, dl, dr, lens, new, page, seed, sharp=1.0, pad=0):
    """Ragged requests: lens[r] positions, the last new[r] of them the chunk's."""
    g = torch.Generator().manual_seed(seed)
    R, dqk = len(lens), dl + dr
    stride = max(1, -(-max(lens) // page))
    pages = R * stride + 1
    table = torch.randperm(pages, generator=g)[:R * stride].to(I32).view(R, stride)
    rows = torch.randn((pages * page, dqk), generator=g)
    kv, sc = wl.quantize_rows(rows)
    req = sum(([r] * new[r] for r in range(R)), []) + [-1] * pad
    pos = sum((list(range(lens[r] - new[r], lens[r])) for r in range(R)), []) + [-1] * pad
    q = (torch.randn((len(req), H, dqk), generator=g) * sharp).to(torch.bfloat16)
    return dict(q=q, kv=kv, sc=sc, table=table, req=torch.tensor(req, dtype=I32), pos=torch.tensor(pos, dtype=I32),
                H=H, dl=dl, dr=dr, page=page, scale=dqk**-0.5)


def _chunk_ref(c):
    """fp64 oracle (every visible position selected), and the tolerance's A =
    sum_p softmax_p |x_p| and B = s_max sum_p |code_p| (tensor cores only)."""
    n = len(c["pos"])
    width = max(1, int(c["pos"].max()) + 1)
    idx = np.where(np.arange(width)[None, :] <= c["pos"].numpy()[:, None], np.arange(width)[None, :], -1)
    idx[c["req"].numpy() < 0] = -1
    kw = dict(d_latent=c["dl"], d_rope=c["dr"], page_size=c["page"], softmax_scale=c["scale"], check=False)
    args = (c["table"].numpy(), c["req"].clamp(min=0).numpy(), idx.astype(np.int32))
    q = c["q"].view(torch.int16).numpy()
    out, lse = oracle.sparse_mla(q, c["kv"].numpy(), c["sc"].numpy(), *args, **kw)
    x = (c["kv"].view(torch.float8_e4m3fn).double() * c["sc"].double()[:, None]).numpy()
    A, B = np.zeros_like(out), np.zeros_like(out)
    code = c["kv"].view(torch.float8_e4m3fn).double().numpy()
    for t in range(n):
        p = idx[t][idx[t] >= 0]
        if not len(p):
            continue
        slot = c["table"].numpy()[c["req"][t], p // c["page"]].astype(np.int64) * c["page"] + p % c["page"]
        ok = (slot >= 0) & (slot < len(x))
        v = x[slot[ok]]
        z = (c["q"][t].double().numpy() @ v.T) * c["scale"] - lse[t][:, None]
        A[t] = np.exp(z) @ np.abs(v[:, :c["dl"]])
        if c["H"] == 64 and ok.any():
            B[t] = c["sc"].double().numpy()[slot[ok]].max() * np.abs(code[slot[ok]][:, :c["dl"]]).sum(0)
    return out, lse, A, B


def _cuda(c):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}


def _run_chunk(c, splits=None, **kw):
    g = _cuda(c)
    st = torch.zeros(1, dtype=I32, device="cuda")
    r = dsa.chunk_mla(g["q"], g["kv"], g["sc"], g["table"], g["req"], g["pos"], d_latent=c["dl"], d_rope=c["dr"],
                      page_size=c["page"], softmax_scale=c["scale"], num_splits=splits, dev_status=st, **kw)
    torch.cuda.synchronize()
    return r[0], r[1], int(st)


def _check_chunk(out, lse, want):
    o, l, A, B = want
    got = host(out.double())
    # the output's rounding plus the weights' (see the module's head)
    tol = 2.0**-8 * np.abs(o) + (2.0**-7 + 2.0**-12) * A + 2.0**-21 * B
    assert np.isfinite(got).all()
    assert (np.abs(got - o) <= tol).all(), float((np.abs(got - o) - tol).max())
    norm = np.linalg.norm(o)
    if norm > 0:
        assert np.linalg.norm(got - o) <= 5e-3 * norm
    gl = host(lse.double())
    empty = np.isneginf(l)
    assert np.array_equal(empty, np.isneginf(gl))
    assert (np.abs(gl - l)[~empty] <= 1e-3).all()


SHAPES = [(16, 64, 16), (64, 512, 64)]
LENS = [([1], [1], 16), ([2], [2], 16), ([64], [1], 64), ([65], [65], 64), ([127, 1, 64], [3, 1, 2], 64),
        ([700, 129, 63], [5, 9, 63], 48), ([300, 31], [40, 31], 1), ([513, 200], [2, 7], 7), ([1000], [4], 128),
        ([257, 640], [1, 1], 24)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")
@pytest.mark.parametrize("lens,new,page", LENS, ids=lambda v: str(v))
def test_chunk_matches_the_oracle(shape, lens, new, page):
    c = _chunk_case(*shape, lens, new, page, seed=sum(lens) + page, pad=2)
    want = _chunk_ref(c)
    for splits in (1, 3):
        out, lse, st = _run_chunk(c, splits)
        assert st == 0
        _check_chunk(out, lse, want)
        assert (out[-2:] == 0).all() and torch.isneginf(lse[-2:]).all()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")
@pytest.mark.parametrize("page", [64, 5])
def test_chunk_splits_merged_by_the_call_and_by_combine(shape, page):
    """2 to 8 splits, more than some tokens have tiles, padding and empty tokens among
    them: merged in the call, and as partials through combine."""
    c = _chunk_case(*shape, [700, 40, 130], [2, 1, 3], page, seed=21, pad=2)
    c["pos"][1] = -1
    want = _chunk_ref(c)
    g = _cuda(c)
    args = (g["q"], g["kv"], g["sc"], g["table"], g["req"], g["pos"])
    kw = dict(d_latent=c["dl"], d_rope=c["dr"], page_size=page, softmax_scale=c["scale"])
    for S in range(2, 10):
        out, lse, st = _run_chunk(c, S)
        assert st == 0
        _check_chunk(out, lse, want)
        if S <= 8:
            st = torch.zeros(1, dtype=I32, device="cuda")
            _check_chunk(*dsa.chunk_mla_fwd(*args, num_splits=S, merge=True, dev_status=st, **kw), want)
        _check_chunk(*dsa.combine(*dsa.chunk_mla_fwd(*args, num_splits=S, **kw)), want)
        n, H = g["q"].shape[:2]
        buf = dict(o_part=torch.empty((S, n, H, c["dl"]), device="cuda"), lse_part=torch.empty((S, n, H), device="cuda"))
        _check_chunk(*dsa.chunk_mla(*args, num_splits=S, buffers=buf, **kw), want)
    with pytest.raises(dsa.DsaError):
        dsa.chunk_mla_fwd(*args, num_splits=9, merge=True, **kw)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")
def test_chunk_long_context_every_split_count(shape):
    c = _chunk_case(*shape, [5000, 2611], [1, 2], 64, seed=3)
    want = _chunk_ref(c)
    for splits in (None, 1, 2, 7, 64):
        out, lse, st = _run_chunk(c, splits, max_ctx=5000)
        assert st == 0
        _check_chunk(out, lse, want)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")
def test_chunk_sharp_logits_and_growing_scales(shape):
    """Logits ~ N(0, 36) that keep raising the running maximum, and rows whose
    scales grow a thousandfold along the context."""
    c = _chunk_case(*shape, [2000, 900], [3, 40], 64, seed=5, sharp=6.0)
    _check_chunk(*_run_chunk(c, 1)[:2], _chunk_ref(c))
    c = _chunk_case(*shape, [1500], [5], 64, seed=6)
    pos_of = torch.zeros(len(c["sc"]))
    for j, p in enumerate(c["table"][0].tolist()):
        pos_of[p * 64:(p + 1) * 64] = torch.arange(64) + 64 * j
    c["sc"] = c["sc"] * torch.exp2(pos_of / 150)
    c["q"] = (c["q"].float() / 64).to(torch.bfloat16)
    for splits in (1, 4):
        _check_chunk(*_run_chunk(c, splits)[:2], _chunk_ref(c))


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")
@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-20])
def test_chunk_other_softmax_scales(shape, scale):
    """No scale (every position weighs the same), a negative and a tiny one."""
    c = _chunk_case(*shape, [700, 90], [2, 1], 16, seed=12)
    c["scale"] = scale
    for splits in (1, 3):
        _check_chunk(*_run_chunk(c, splits)[:2], _chunk_ref(c))


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")
def test_chunk_rows_of_scale_zero_and_zero_queries(shape):
    """All-zero cache rows (scale 0) take part with logit 0; a zero query weighs every row the same."""
    c = _chunk_case(*shape, [260, 130], [3, 2], 64, seed=13)
    c["sc"][::3] = 0.0
    c["sc"][int(c["table"][1, 0]) * 64:][:64] = 0.0  # the whole first tile of request 1
    c["q"][1] = 0.0
    for splits in (1, 2):
        _check_chunk(*_run_chunk(c, splits)[:2], _chunk_ref(c))


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")
def test_chunk_tokens_in_any_order_and_shared_pages(shape):
    c = _chunk_case(*shape, [300, 300, 200], [4, 4, 4], 16, seed=14)
    c["table"][1, :10] = c["table"][0, :10]  # a shared prefix
    g = torch.Generator().manual_seed(1)
    order = torch.randperm(len(c["pos"]), generator=g)
    c["req"], c["pos"] = c["req"][order].contiguous(), c["pos"][order].contiguous()
    for splits in (1, 2):
        _check_chunk(*_run_chunk(c, splits)[:2], _chunk_ref(c))


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")
def test_chunk_one_peak_over_a_long_flat_tail(shape):
    """A peak at the first position and a tail of rows 2^-13 below it, together
    as heavy as the peak: the tail may not be rounded away."""
    H, dl, dr = shape
    c = _chunk_case(*shape, [8193], [1], 64, seed=7)
    dqk = dl + dr
    rows = torch.zeros((len(c["sc"]), dqk))
    rows[:, 0] = 1.0          # every row: value 1 in dimension 0 ...
    rows[:, dl - 1] = 0.5
    c["kv"], c["sc"] = wl.quantize_rows(rows)
    first = int(c["table"][0, 0]) * 64
    row = torch.zeros((1, dqk))
    row[0, 0], row[0, dqk - 1], row[0, 1] = 1.0, 1.0, -1.0   # ... the peak differs in the last dimension
    kv1, sc1 = wl.quantize_rows(row)
    c["kv"][first], c["sc"][first] = kv1[0], sc1[0]
    q = torch.zeros((1, H, dqk))
    q[:, :, dqk - 1] = 13 * np.log(2) / c["scale"]
    c["q"] = q.to(torch.bfloat16)
    _check_chunk(*_run_chunk(c, 1)[:2], _chunk_ref(c))
    _check_chunk(*_run_chunk(c, 5)[:2], _chunk_ref(c))


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")
@pytest.mark.parametrize("page", [64, 16, 5])
def test_chunk_ignores_what_lies_past_the_last_position(shape, page):
    """NaN codes and NaN or infinite scales in rows no token may see."""
    c = _chunk_case(*shape, [70, 130, 64], [2, 1, 3], page, seed=8)
    want = _chunk_ref(c)
    clean = _run_chunk(c, 1)
    seen = torch.zeros(len(c["sc"]), dtype=torch.bool)
    for r, n in enumerate((70, 130, 64)):
        p = torch.arange(n)
        seen[c["table"][r].long()[p // page] * page + p % page] = True
    c["kv"][~seen] = 0x7F
    c["sc"][~seen] = torch.where(torch.arange(int((~seen).sum())) % 2 == 0, float("nan"), float("inf"))
    for splits in (1, 2):
        out, lse, st = _run_chunk(c, splits)
        assert st == 0
        _check_chunk(out, lse, want)
    assert torch.equal(_run_chunk(c, 1)[0], clean[0])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}")
@pytest.mark.parametrize("page", [64, 16])
def test_chunk_bad_positions_requests_and_pages(shape, page):
    c = _chunk_case(*shape, [200, 200, 200, 200], [2, 2, 2, 2], page, seed=9)
    c["req"][2], c["req"][3] = 4, -2                     # no such request
    c["pos"][4], c["pos"][5] = -2, page * c["table"].shape[1]  # no such position
    c["table"][3, 1] = 1 << 20                           # no such page: its rows are skipped
    out, lse, st = _run_chunk(c, 1)
    assert st == dsa.DEV_BAD_QPOS | dsa.DEV_BAD_PAGE
    assert (out[2:6] == 0).all() and torch.isneginf(lse[2:6]).all()
    for t in (2, 3, 4, 5):
        c["req"][t], c["pos"][t] = 0, -1
    want = _chunk_ref(c)
    for splits in (1, 3):
        out, lse, _ = _run_chunk(c, splits)
        _check_chunk(out, lse, want)
    c["table"][3, :] = -1                                # a request without any page
    out, lse, st = _run_chunk(c, 1)
    assert st == dsa.DEV_BAD_PAGE and (out[6:] == 0).all() and torch.isneginf(lse[6:]).all()


def test_chunk_no_tokens_other_stream_and_captured_graph():
    c = _chunk_case(64, 512, 64, [300, 100], [3, 2], 64, seed=10)
    g = _cuda(c)
    kw = dict(d_latent=512, d_rope=64, page_size=64, softmax_scale=c["scale"])
    for S in (1, 2):
        o, l = dsa.chunk_mla(g["q"][:0], g["kv"], g["sc"], g["table"], g["req"][:0], g["pos"][:0], num_splits=S, **kw)
        assert o.shape == (0, 64, 512) and l.shape == (0, 64)
    want = _chunk_ref(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = dsa.chunk_mla(g["q"], g["kv"], g["sc"], g["table"], g["req"], g["pos"], num_splits=2, stream=s, **kw)
    s.synchronize()
    _check_chunk(out, lse, want)
    graph = torch.cuda.CUDAGraph()
    buf = dict(out=torch.empty_like(out), lse=torch.empty_like(lse))
    with torch.cuda.graph(graph):
        dsa.chunk_mla(g["q"], g["kv"], g["sc"], g["table"], g["req"], g["pos"], num_splits=1, buffers=buf, **kw)
    graph.replay()
    torch.cuda.synchronize()
    _check_chunk(buf["out"], buf["lse"], want)
    # the graph follows its inputs: other tokens, one of them padding now
    g["req"][0] = -1
    g["pos"][1] = 7
    graph.replay()
    torch.cuda.synchronize()
    c["req"][0], c["pos"][1] = -1, 7
    _check_chunk(buf["out"], buf["lse"], _chunk_ref(c))


def test_chunk_agrees_with_the_sparse_call_over_every_position():
    w = wl.Workload("dense", 3, 2, 64, 512, 64, 900, 640, 64, 900, seed=31)
    inp = wl.make_inputs(w, device="cuda")
    kw = dict(d_latent=512, d_rope=64, page_size=64, softmax_scale=w.scale)
    so, sl, _ = dsa.sparse_mla_topk(inp.q, inp.kv, inp.kv_scale, inp.block_table, inp.q_req, inp.q_pos, inp.scores, 900,
                                    num_splits=1, **kw)
    co, cl = dsa.chunk_mla(inp.q, inp.kv, inp.kv_scale, inp.block_table, inp.q_req, inp.q_pos, **kw)
    torch.cuda.synchronize()
    # both round their weights and their outputs: the sum of two bounds of 2^-8
    assert float((so.float() - co.float()).norm() / so.float().norm()) <= 2.0**-7
    assert float((sl - cl).abs().max()) <= 1e-3


# ---- offsets past 32 bits ------------------------------------------------------------


@pytest.mark.parametrize("shape,slots", [((64, 512, 64), 8 << 20), ((16, 64, 16), 60 << 20)], ids=["h64", "h16"])
@pytest.mark.parametrize("page", [64, 5])
def test_cache_rows_past_4_gib(shape, slots, page):
    """The same pages at the end of a cache of more than 2^32 bytes give the same
    bits, and a row written there arrives there."""
    c = _chunk_case(*shape, [300, 130], [3, 2], page, seed=61)
    d = shape[1] + shape[2]
    few = len(c["sc"]) // page
    pages = slots // page
    assert (pages - few) * page * d > 1 << 32
    kv = torch.empty((pages * page, d), dtype=torch.uint8, device="cuda")
    sc = torch.empty(pages * page, device="cuda")
    kv[-few * page:].copy_(c["kv"])
    sc[-few * page:].copy_(c["sc"])
    for splits in (1, 3, 12):
        want = _run_chunk(c, splits)
        big = dict(c, kv=kv, sc=sc, table=c["table"] + (pages - few))
        got = _run_chunk(big, splits)
        assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k = torch.randn((2, 1, d), device="cuda").to(torch.bfloat16)
    last = i32([few * page - 1, 3])
    kv2, sc2 = c["kv"].cuda(), c["sc"].cuda()
    dsa.qk_norm_rope(None, k, None, None, d_rope=0, slot=last, kv=kv2, kv_scale=sc2)
    dsa.qk_norm_rope(None, k, None, None, d_rope=0, slot=last + (pages - few) * page, kv=kv, kv_scale=sc)
    assert torch.equal(kv[-few * page:], kv2) and torch.equal(sc[-few * page:], sc2)


def test_verify_rows_past_32_bit_offsets():
    rows, V, ld = 3, 1000, 1 << 30
    g = torch.Generator().manual_seed(62)
    p, q = (torch.softmax(3 * torch.randn((rows, V), generator=g), 1).cuda() for _ in range(2))
    tok, cu = i32([5, 17, 0]), i32([0, rows])
    ua, us = torch.rand(rows, generator=g).cuda(), torch.rand(1, generator=g).cuda()
    mem = torch.empty((rows - 1) * ld + 2 * V, device="cuda")
    far = [mem.as_strided((rows, V), (ld, 1), at) for at in (0, V)]
    far[0].copy_(p), far[1].copy_(q)
    for take in (0.0, 1.0):
        u = torch.full_like(ua, take)
        want = dsa.verify_draft(p, tok, cu, u, us, draft_probs=q, max_out=3)
        got = dsa.verify_draft(far[0], tok, cu, u, us, draft_probs=far[1], max_out=3)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---- streams and graphs ----------------------------------------------------------------


def test_two_calls_at_once_and_outputs_of_another_stream():
    """Calls of every operator on two streams at once give what each gives alone,
    and outputs cut for a stream are that stream's memory."""
    c = _chunk_case(64, 512, 64, [700, 90, 1300], [5, 1, 9], 64, seed=41)
    g = _cuda(c)
    ckw = dict(d_latent=512, d_rope=64, page_size=64, softmax_scale=c["scale"])
    q, k, gen = _qk_inputs(300, 64, 1, 576, torch.bfloat16, seed=42)
    pos = torch.randint(0, 90, (300,), generator=gen, dtype=I32).cuda()
    cs = torch.from_numpy(_tables(90, 64)).cuda()
    w = torch.ones(576, device="cuda")
    p, dq, tok, cu, ua, us = _verify_case(24, 6, 5003, True, seed=43)
    lay = _layout_case(40, 9, 500, 16, seed=44)
    li = [i32(x) for x in lay[:3]]
    lf, pages, none_used = i32(lay[4]), lay[5], i32([0])

    def calls(stream):
        table = torch.from_numpy(lay[3].copy()).cuda()
        r = [dsa.chunk_mla(g["q"], g["kv"], g["sc"], g["table"], g["req"], g["pos"], num_splits=S, stream=stream, **ckw)
             for S in (1, 3, 12)]
        r.append(dsa.qk_norm_rope(q, k, pos, cs, d_rope=64, q_weight=w, stream=stream))
        r.append(dsa.verify_draft(p, tok, cu, ua, us, draft_probs=dq, max_out=7, stream=stream)[:2])
        r.append(dsa.batch_layout(*li, table, lf, none_used, page_size=16, num_pages=pages, capacity=400, stream=stream))
        return [t for x in r for t in x] + [table]

    want = calls(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [calls(s) for s in streams]
        torch.cuda.synchronize()
        for rows in got:
            for x, y in zip(rows, want):
                assert torch.equal(x, y)
        del got, rows


def test_captured_norm_rope_and_verification_follow_their_inputs():
    T = 70
    q, k, gen = _qk_inputs(T, 4, 1, 576, torch.bfloat16, seed=51)
    cs = torch.from_numpy(_tables(64, 64)).cuda()
    w = (1 + 0.3 * torch.randn(576, generator=gen)).cuda()
    pos = torch.randint(0, 64, (T,), generator=gen, dtype=I32).cuda()
    slot = torch.arange(T, dtype=I32, device="cuda")
    kv, sc = torch.zeros(T, 576, dtype=torch.uint8, device="cuda"), torch.zeros(T, device="cuda")
    p, dq, tok, cu, ua, us = _verify_case(9, 4, 3001, True, seed=52)
    ctx = torch.arange(9, dtype=I32, device="cuda")
    qo = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    res = [torch.empty(9, 5, dtype=I32, device="cuda"), torch.empty(9, dtype=I32, device="cuda"),
           torch.empty(9, dtype=I32, device="cuda")]
    kw = dict(d_rope=64, q_weight=w, k_weight=w[:512], slot=slot)

    def norm(kv_, sc_, **o):
        return dsa.qk_norm_rope(q, k, pos, cs, kv=kv_, kv_scale=sc_, **kw, **o)[0]

    def verify(**o):
        return dsa.verify_draft(p, tok, cu, ua, us, draft_probs=dq, ctx_len=ctx, max_out=5, **o)

    norm(kv, sc), verify()  # loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm(kv, sc, q_out=qo)
        verify(tokens=res[0], num_out=res[1], ctx_out=res[2])
    for step in range(3):
        pos.copy_(torch.randint(0, 64, (T,), generator=gen, dtype=I32))
        q.normal_(), k.normal_()
        ua.uniform_(), us.uniform_()
        kv.zero_(), sc.zero_()
        graph.replay()
        kv2, sc2 = torch.zeros_like(kv), torch.zeros_like(sc)
        assert torch.equal(norm(kv2, sc2), qo)
        assert torch.equal(kv, kv2) and torch.equal(sc, sc2) and float(sc.min()) > 0
        for x, y in zip(verify(), res):
            assert torch.equal(x, y)


# ---- the binding's two ways to marshal a call ---------------------------------------


def _without_cpp(f):
    fast, dsa._fast = dsa._fast, None
    try:
        return f()
    finally:
        dsa._fast = fast


def test_cpp_marshalling_is_the_one_that_runs_and_agrees_with_python():
    assert dsa._fast is not None
    c, n, held, table, free, pages = _layout_case(9, 6, 100, 16, seed=11)
    p, q, tok, cu, ua, us = _verify_case(8, 5, 777, True, seed=6, pad_cols=3)
    ch = _cuda(_chunk_case(64, 512, 64, [300, 100], [3, 2], 64, seed=10))
    tiny = _cuda(_chunk_case(16, 64, 16, [500, 100], [1, 1], 16, seed=10))
    x, k, g = _qk_inputs(12, 6, 1, 576, torch.bfloat16, seed=2, pad=8)
    pos = torch.randint(0, 50, (12,), generator=g, dtype=I32).cuda()
    cs = torch.from_numpy(_tables(50, 64)).cuda()
    slot = torch.randperm(20, generator=g)[:12].to(I32).cuda()

    def layout():
        t = torch.from_numpy(table.copy()).cuda()
        return [*dsa.batch_layout(i32(c), i32(n), i32(held), t, i32(free), i32([0]), page_size=16, num_pages=pages,
                                  capacity=70), t]

    def rows():
        kv, sc = torch.zeros((20, 576), dtype=torch.uint8, device="cuda"), torch.zeros(20, device="cuda")
        a = dsa.qk_norm_rope(x, k, pos, cs, d_rope=64, slot=slot, kv=kv, kv_scale=sc)
        b = dsa.qk_norm_rope(x, k, pos, cs, d_rope=64, interleaved=False)
        assert a[1] is None
        return [a[0], kv, sc, *b]

    def attention():
        r = []
        for d, page, kw in ((ch, 64, dict(max_ctx=300)), (ch, 64, dict(num_splits=3)), (tiny, 16, {})):
            r += dsa.chunk_mla(d["q"], d["kv"], d["sc"], d["table"], d["req"], d["pos"], d_latent=d["dl"],
                               d_rope=d["dr"], page_size=page, softmax_scale=d["scale"], **kw)
        return r

    def verify():
        a = dsa.verify_draft(p, tok, cu, ua, us, draft_probs=q, max_out=6)
        assert a[2] is None
        return [*a[:2], *dsa.verify_draft(p, tok, cu, ua, us, max_out=6, ctx_len=tok[:8].contiguous())]

    for f in (layout, rows, attention, verify):
        a, b = f(), _without_cpp(f)
        torch.cuda.synchronize()
        for s, t in zip(a, b):
            assert s.dtype == t.dtype and s.shape == t.shape and torch.equal(s, t)


def test_calls_the_binding_refuses_both_ways():
    c, n, held, table, free, pages = _layout_case(9, 6, 100, 16, seed=11)
    a = (i32(c), i32(n), i32(held), torch.from_numpy(table).cuda(), i32(free), i32([0]))
    p, q, tok, cu, ua, us = _verify_case(8, 5, 777, True, seed=6)
    x, k, _ = _qk_inputs(12, 6, 1, 576, torch.bfloat16, seed=2, pad=8)
    pos, cs = i32([0] * 12), torch.from_numpy(_tables(50, 64)).cuda()
    ch = _cuda(_chunk_case(64, 512, 64, [300, 100], [3, 2], 64, seed=10))
    kw = dict(page_size=16, num_pages=pages, capacity=70)
    mla = (ch["q"], ch["kv"], ch["sc"], ch["table"], ch["req"], ch["pos"])
    mk = dict(d_latent=512, d_rope=64, page_size=64, softmax_scale=0.04)
    bad = [
        (ValueError, lambda: dsa.batch_layout(a[0].cpu(), *a[1:], **kw)),
        (TypeError, lambda: dsa.batch_layout(a[0].long(), *a[1:], **kw)),
        (ValueError, lambda: dsa.batch_layout(*a[:3], a[3].t(), *a[4:], **kw)),
        (ValueError, lambda: dsa.batch_layout(a[0], a[1][1:], *a[2:], **kw)),
        (ValueError, lambda: dsa.batch_layout(*a, **{**kw, "capacity": -1})),
        (dsa.DsaError, lambda: dsa.batch_layout(*a, **{**kw, "page_size": 0})),
        (dsa.DsaError, lambda: dsa.batch_layout(*a, **kw, out=dsa.BatchLayout(
            *[torch.empty(m, dtype=I32, device="cuda") for m in (10, 70, 70, 70)], a[0], torch.empty_like(a[0]),
            torch.empty_like(a[5])))),
        (ValueError, lambda: dsa.qk_norm_rope(x, k, pos[:5], cs, d_rope=64)),
        (ValueError, lambda: dsa.qk_norm_rope(x, k, pos, cs, d_rope=32)),
        (ValueError, lambda: dsa.qk_norm_rope(x, k[:4], pos, cs, d_rope=64)),
        (TypeError, lambda: dsa.qk_norm_rope(x.float(), k, pos, cs, d_rope=64)),
        (TypeError, lambda: dsa.qk_norm_rope(x, k.half(), pos, cs, d_rope=64)),
        (ValueError, lambda: dsa.qk_norm_rope(x.transpose(1, 2), None, pos, cs, d_rope=64)),
        (dsa.DsaError, lambda: dsa.qk_norm_rope(x, k, pos, cs, d_rope=64, q_weight=cs[0, :12].contiguous())),
        (dsa.DsaError, lambda: dsa.qk_norm_rope(x, k, pos, cs, d_rope=64, eps=-1.0)),
        (ValueError, lambda: dsa.chunk_mla(*mla[:5], mla[5][:2], **mk)),
        (ValueError, lambda: dsa.chunk_mla(*mla, **{**mk, "page_size": 7})),
        (dsa.DsaError, lambda: dsa.chunk_mla(*mla, **mk, num_splits=65)),
        (dsa.DsaError, lambda: dsa.chunk_mla(*mla, **mk, num_splits=0)),
        (dsa.DsaError, lambda: dsa.chunk_mla(*mla, **{**mk, "softmax_scale": float("inf")})),
        (TypeError, lambda: dsa.verify_draft(p.double(), tok, cu, ua, us, max_out=6)),
        (ValueError, lambda: dsa.verify_draft(p, tok, cu, ua, us, draft_probs=q[:, :5], max_out=6)),
        (ValueError, lambda: dsa.verify_draft(p, tok, cu, ua, us, max_out=0)),
        (ValueError, lambda: dsa.verify_draft(p, tok, cu[:4], ua, us, max_out=6)),
        (ValueError, lambda: dsa.verify_draft(p[:1].expand(p.shape), tok, cu, ua, us, max_out=6)),
        (TypeError, lambda: dsa.verify_draft(p, tok, cu, ua, us, max_out=6, dev_status=cs)),
    ]
    for i, (kind, f) in enumerate(bad):
        for way in (lambda f=f: f(), lambda f=f: _without_cpp(f)):
            with pytest.raises(kind):
                way()
                pytest.fail(f"case {i} was taken")


# ---- together ----------------------------------------------------------------------


def test_a_speculative_step_end_to_end():
    """Two verify steps of three requests: lengths -> layout -> norms, rotation
    and cache write -> attention over everything -> drafted tokens -> lengths,
    each stage against its definition on what the stage before produced."""
    H, dl, dr, page, R, n, V = 64, 512, 64, 16, 3, 4, 777
    d = dl + dr
    g = torch.Generator().manual_seed(77)
    pages, stride, cap = 60, 12, R * (n + 1) + 2
    free = torch.randperm(pages, generator=g).to(I32).cuda()
    table = torch.full((R, stride), -1, dtype=I32, device="cuda")
    kv = torch.full((pages * page, d), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes until written
    sc = torch.full((pages * page,), float("nan"), device="cuda")
    cs = _tables(stride * page, dr)
    csd = torch.from_numpy(cs).cuda()
    kw = (1 + 0.1 * torch.randn(dl, generator=g)).cuda()
    ctx, held, used = (torch.zeros(R, dtype=I32, device="cuda"), torch.zeros(R, dtype=I32, device="cuda"),
                       torch.zeros(1, dtype=I32, device="cuda"))
    st = torch.zeros(1, dtype=I32, device="cuda")
    for step, new in enumerate(([30, 17, 1], [n + 1, n + 1, 2], [n + 1, 1, n + 1])):
        cap_s = max(cap, sum(new))
        lay = dsa.batch_layout(ctx, i32(new), held, table, free, used, page_size=page, num_pages=pages, capacity=cap_s,
                               dev_status=st)
        q = torch.randn((cap_s, H, d), generator=g).to(torch.bfloat16).cuda()
        k = torch.randn((cap_s, 1, d), generator=g).to(torch.bfloat16).cuda()
        qo, _ = dsa.qk_norm_rope(q, k, lay.q_pos, csd, d_rope=dr, k_weight=kw, slot=lay.slot, kv=kv, kv_scale=sc,
                                 q_out=torch.zeros_like(q), dev_status=st)
        kws = dict(d_latent=dl, d_rope=dr, page_size=page, softmax_scale=d**-0.5, dev_status=st)
        out, lse = dsa.chunk_mla(qo, kv, sc, table, lay.q_req, lay.q_pos, **kws)
        torch.cuda.synchronize()
        pos = host(lay.q_pos)
        live = pos >= 0
        want = ref.norm_rope(host(k.double())[live], host(kw), pos[live], cs, dr, True, 1e-6)[:, 0]
        at = lay.slot[torch.from_numpy(live).cuda()].long()
        _check_codes(kv[at], sc[at], want)
        c = dict(q=qo.cpu(), kv=kv.cpu(), sc=sc.cpu(), table=table.cpu(), req=lay.q_req.cpu(), pos=lay.q_pos.cpu(), H=H,
                 dl=dl, dr=dr, page=page, scale=d**-0.5)
        _check_chunk(out, lse, _chunk_ref(c))
        # the step's "model": probabilities over V from the attention's output
        proj = torch.randn((H * dl, V), generator=g).cuda() * 0.2
        p = torch.softmax(out.float().view(cap_s, -1) @ proj, 1)
        dq = torch.softmax((p + 1e-6).log() + 0.5 * torch.randn((cap_s, V), generator=g).cuda(), 1)
        tok = torch.multinomial(dq.cpu(), 1, generator=g)[:, 0].to(I32).cuda()
        ua, us = torch.rand(cap_s, generator=g).cuda(), torch.rand(R, generator=g).cuda()
        before = ctx
        tokens, num, ctx = dsa.verify_draft(p, tok, lay.cu_q, ua, us, draft_probs=dq, ctx_len=before, max_out=max(new),
                                            dev_status=st)
        torch.cuda.synchronize()
        wt, wn, _ = ref.verify_draft(host(p), host(dq), host(tok), host(lay.cu_q), host(ua), host(us), max(new))
        assert np.array_equal(host(tokens), wt) and np.array_equal(host(num), wn)
        assert np.array_equal(host(ctx), host(before) + wn)
        held, used = lay.pages_held, lay.free_used
    assert int(st) == 0
