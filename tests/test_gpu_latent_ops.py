"""GPU tests of latent attention's other form and the products around it
(absorb_q, project_out, expand_kv, prompt_mla) against 64-bit definitions.

Tolerances, each from the arithmetic:
  products   half a bf16 step, 2^-8 of the value, plus the sum's additions: at most K of
      them, each off by at most one unit of 2^-23 of the largest partial sum, so
      (K + 2) 2^-23 sum |a b| (the scale's multiplication and the last rounding in the 2).
  attention  out: half a bf16 step, plus what the weights are off by.  A weight is
      rounded to bf16 (half a step, 2^-8); its logit to D = (K + 2) 2^-23 scale sum |q k|
      (largest over the keys) plus 2^-22 |z|, which moves a weight and the sum of weights by
      that much each; exponentials and the sum's additions 2^-21 + (n / 8) 2^-23; O's additions
      n 2^-23: all of A = sum_p softmax_p |v_p|.
      lse: D, 2^-21 + (n / 8) 2^-23 and 2^-22 of the value.
      The error's root mean square over a call: two independent roundings to bf16 (out, and
      weights), each at most 2^-8 / sqrt(3) where values spread evenly over a binade:
      3.2e-3 of the result's.
"""
import math

import pytest
import torch

import dsa_sparse_mla_topk_gb300 as dsa

pytestmark = pytest.mark.gpu
I32, BF16 = torch.int32, torch.bfloat16
LARGE = dict(heads=64, dn=128, dr=64, dv=128, dl=512)
SMALL = dict(heads=16, dn=32, dr=16, dv=32, dl=64)
ODD = dict(heads=3, dn=48, dr=16, dv=80, dl=208)
PLAIN = dict(heads=2, dn=112, dr=0, dv=16, dl=16)
SHAPES = [LARGE, SMALL, ODD, PLAIN]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dsa_sparse_mla_topk_gb300 import build
    build.build()
    dsa.load_library()


@pytest.fixture(params=["marshalled in C++", "marshalled in Python"])
def both_ways(request, monkeypatch):
    if request.param == "marshalled in Python":
        monkeypatch.setattr(dsa, "_fast", None)


def i32(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(shape, g, pad=0):
    """bf16 rows; pad > 0: the first columns of wider ones (strided)."""
    x = torch.randn((*shape[:-1], shape[-1] + pad), generator=g, device="cuda").to(BF16)
    return x[..., :shape[-1]]


def weight(c, g):
    return (torch.randn((c["heads"], c["dn"] + c["dv"], c["dl"]), generator=g, device="cuda") * c["dl"]**-0.5).to(BF16)


def near(got, want, bound):
    """Every element within its bound; what is not finite in want is the same in got."""
    assert got.shape == want.shape
    got, fine = got.double(), torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    odd = ~fine & ~torch.isnan(want)
    assert torch.equal(got[odd], want[odd])
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, float(over.max())


def near_product(got, a, b, k):
    """got bf16 = a b (per group, 64 bits)."""
    want = torch.matmul(a, b)
    near(got, want, 2.0**-8 * want.abs() + (k + 2) * 2.0**-23 * torch.matmul(a.abs(), b.abs()))


# ---- absorb_q, project_out -----------------------------------------------------------


def check_absorb(c, q, w, y):
    dn, dl = c["dn"], c["dl"]
    assert torch.equal(y[..., dl:].view(torch.int16), q[..., dn:].contiguous().view(torch.int16))  # the rotated part, bit for bit
    near_product(y[..., :dl].transpose(0, 1), q[..., :dn].double().transpose(0, 1), w[:, :dn].double(), dn)


def check_project(c, o, w, y):
    near_product(y.transpose(0, 1), o.double().transpose(0, 1), w[:, c["dn"]:].double().transpose(1, 2), c["dl"])


@pytest.mark.parametrize("c", SHAPES, ids=lambda c: f"{c['heads']}x{c['dn']}")
@pytest.mark.parametrize("n", [1, 2, 31, 127, 128, 129, 400, 1300])
@pytest.mark.parametrize("pad", [0, 24])
def test_products_match_the_definition(c, n, pad):
    g = gen(n + pad)
    w = weight(c, g)
    q, o = rows((n, c["heads"], c["dn"] + c["dr"]), g, pad), rows((n, c["heads"], c["dl"]), g, pad)
    check_absorb(c, q, w, dsa.absorb_q(q, w, d_rope=c["dr"]))
    check_project(c, o, w, dsa.project_out(o, w, d_nope=c["dn"]))


def test_products_head_major_rows_and_given_outputs(both_ways):
    """Rows stored head after head, expanded rows (a token stride of 0) and outputs of the caller's."""
    c, g, n = LARGE, gen(1), 150
    w = weight(c, g)
    q = rows((c["heads"], n, 192), g).transpose(0, 1)
    guard = torch.full((n + 2, 64, 576), 7.0, device="cuda", dtype=BF16)
    y = dsa.absorb_q(q, w, d_rope=64, q_out=guard[1:-1])
    assert y.data_ptr() == guard[1:].data_ptr() and bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all())
    check_absorb(c, q, w, y)
    o = rows((1, c["heads"], 512), g).expand(n, -1, -1)
    guard = torch.full((n + 2, 64, 128), 7.0, device="cuda", dtype=BF16)
    y = dsa.project_out(o, w, d_nope=128, out=guard[1:-1])
    assert bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all())
    check_project(c, o, w, y)
    assert dsa.absorb_q(q[:0], w, d_rope=64).shape == (0, 64, 576)
    assert dsa.project_out(o[:0], w, d_nope=128).shape == (0, 64, 128)


@pytest.mark.parametrize("c", [LARGE, ODD], ids=["64", "3"])
def test_products_rows_do_not_reach_each_other(c):
    g, n = gen(2), 300
    w = weight(c, g)
    q, o = rows((n, c["heads"], c["dn"] + c["dr"]), g), rows((n, c["heads"], c["dl"]), g)
    y, z = dsa.absorb_q(q, w, d_rope=c["dr"]), dsa.project_out(o, w, d_nope=c["dn"])
    bad = torch.arange(n, device="cuda") % 3 == 1
    q2, o2 = q.clone(), o.clone()
    q2[bad], o2[bad] = math.nan, math.inf
    y2, z2 = dsa.absorb_q(q2, w, d_rope=c["dr"]), dsa.project_out(o2, w, d_nope=c["dn"])
    assert torch.equal(y[~bad], y2[~bad]) and torch.equal(z[~bad], z2[~bad])
    assert bool(torch.isnan(y2[bad]).all())
    # a token's result does not depend on how many there are
    assert torch.equal(dsa.absorb_q(q[:5], w, d_rope=c["dr"]), y[:5])
    assert torch.equal(dsa.project_out(o[:5], w, d_nope=c["dn"]), z[:5])


def test_products_on_another_stream_and_captured():
    c, g, n = LARGE, gen(3), 40
    w, q, o = weight(c, g), rows((n, 64, 192), g), rows((n, 64, 512), g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, z = dsa.absorb_q(q, w, d_rope=64, stream=s), dsa.project_out(o, w, d_nope=128, stream=s)
    s.synchronize()
    check_absorb(c, q, w, y)
    check_project(c, o, w, z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = dsa.absorb_q(q, w, d_rope=64), dsa.project_out(o, w, d_nope=128)
    q.copy_(rows((n, 64, 192), g))
    o.copy_(rows((n, 64, 512), g))
    w.copy_(weight(c, g))
    graph.replay()
    torch.cuda.synchronize()
    check_absorb(c, q, w, y)
    check_project(c, o, w, z)


# ---- expand_kv -------------------------------------------------------------------------


def cache(c, R, ctx, page, g, slack=1):
    d, stride = c["dl"] + c["dr"], -(-ctx // page) + slack
    table = torch.randperm(R * stride, generator=g, device="cuda").to(I32).view(R, stride).contiguous()
    x = torch.randn((R * stride * page, d), generator=g, device="cuda")
    scale = x.abs().amax(1) / 448.0
    kv = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scale[::7] *= 2.0**-20
    scale[::11] = 0
    return kv, scale.contiguous(), table


def check_expand(c, kv, scale, table, lens, w, page, x):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    assert x.cu_k.tolist() == cu
    if cu[-1] == 0:
        return
    slot = torch.cat([table[r].long()[torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page
                      for r, n in enumerate(lens)])
    code, s = kv[slot].view(torch.float8_e4m3fn), scale[slot]
    n, dl = cu[-1], c["dl"]
    assert torch.equal(x.k_rope[:n].view(torch.int16),
                       (code[:, dl:].float() * s[:, None]).to(BF16).view(torch.int16))  # one product, one rounding: bit for bit
    a = code[:, :dl].double() * s.double()[:, None]
    near_product(x.kv[:n].flatten(1), a, w.double().flatten(0, 1).t(), dl)


def run_expand(c, kv, scale, table, lens, w, page, capacity, status=0):
    H, dw = c["heads"], c["dn"] + c["dv"]
    out = dsa.ExpandedKV(torch.full((capacity, H, dw), 7.0, device="cuda", dtype=BF16),
                         torch.full((capacity, c["dr"]), 7.0, device="cuda", dtype=BF16), i32([0] * (len(lens) + 1)))
    st = i32([0])
    x = dsa.expand_kv(kv, scale, table, i32(lens), w, d_rope=c["dr"], page_size=page, out=out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == status
    end = int(x.cu_k[-1])
    assert bool((x.kv[end:] == 7).all()) and bool((x.k_rope[end:] == 7).all())  # rows behind stay as they were
    return x


@pytest.mark.parametrize("c", SHAPES, ids=lambda c: f"{c['heads']}x{c['dn']}")
@pytest.mark.parametrize("lens,page", [([1], 1), ([0, 0], 16), ([128], 64), ([127, 0, 2], 48), ([129, 0, 130, 1], 7),
                                       ([700, 61], 128), ([0, 33, 0, 512, 5, 0], 64)])
@pytest.mark.parametrize("slack", [0, 200])
def test_expand_matches_the_definition(c, lens, page, slack):
    g = gen(sum(lens) + page)
    kv, scale, table = cache(c, len(lens), max(lens), page, g)
    w = weight(c, g)
    x = run_expand(c, kv, scale, table, lens, w, page, sum(lens) + slack)
    check_expand(c, kv, scale, table, lens, w, page, x)


def test_expand_many_requests_and_data_errors():
    c, g = SMALL, gen(5)
    kv, scale, table = cache(c, 8192, 3, 2, g)
    w = weight(c, g)
    lens = torch.randint(0, 4, (8192,), generator=g, device="cuda").tolist()
    check_expand(c, kv, scale, table, lens, w, 2, run_expand(c, kv, scale, table, lens, w, 2, sum(lens) + 3))
    # capacity: the requests up to the last one that fits
    cut = sum(lens[:5000]) - 1
    while lens[4999] == 0 or sum(lens[:5000]) <= cut:
        lens[4999] = 3
        cut = sum(lens[:5000]) - 1
    x = run_expand(c, kv, scale, table, lens, w, 2, cut, status=dsa.DEV_BAD_INDEX)
    fit = [n if r < 4999 else 0 for r, n in enumerate(lens)]
    check_expand(c, kv, scale, table, fit, w, 2, x)
    # lengths below zero and past the table's row give no rows, the others theirs
    row = table.shape[1] * 2
    lens = [3, -1, row, row + 1, 2, 2**31 - 1, 1]
    x = run_expand(c, kv, scale, table[:7].contiguous(), lens, w, 2, 40, status=dsa.DEV_BAD_INDEX | dsa.DEV_BAD_QPOS)
    check_expand(c, kv, scale, table, [3, 0, row, 0, 2, 0, 1], w, 2, x)
    # bad pages: rows of zeros
    t = table[:3].clone()
    t[0, 1], t[2, 0] = -1, kv.shape[0] // 2
    x = run_expand(c, kv, scale, t, [4, 2, 3], w, 2, 9, status=dsa.DEV_BAD_PAGE)
    assert x.cu_k.tolist() == [0, 4, 6, 9]
    for n in (2, 3, 6, 7):
        assert float(x.kv[n].abs().max()) == 0 and float(x.k_rope[n].abs().max()) == 0
    good = run_expand(c, kv, scale, table[:3].contiguous(), [4, 2, 3], w, 2, 9)
    for n in (0, 1, 4, 5, 8):
        assert torch.equal(x.kv[n], good.kv[n]) and torch.equal(x.k_rope[n], good.k_rope[n])
    assert run_expand(c, kv, scale, table[:2].contiguous(), [0, 0], w, 2, 0).cu_k.tolist() == [0, 0, 0]


def test_expand_codes_without_a_value_stay_in_their_row():
    c, g = LARGE, gen(6)
    kv, scale, table = cache(c, 1, 300, 64, g)
    w = weight(c, g)
    slot = lambda p: int(table[0, p // 64]) * 64 + p % 64  # noqa: E731
    want = run_expand(c, kv, scale, table, [300], w, 64, 300)
    kv[slot(100), 3] = 0x7F
    scale[slot(200)] = math.nan
    x = run_expand(c, kv, scale, table, [300], w, 64, 300)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[[100, 200]] = False
    assert torch.equal(x.kv[keep], want.kv[keep]) and bool(torch.isnan(x.kv[~keep]).all())


def test_expand_allocated_other_stream_and_captured(both_ways):
    c, g = LARGE, gen(7)
    kv, scale, table = cache(c, 3, 200, 64, g)
    w, lens = weight(c, g), i32([200, 3, 90])
    torch.cuda.synchronize()
    call = lambda **k: dsa.expand_kv(kv, scale, table, lens, w, d_rope=64, page_size=64, capacity=400, **k)  # noqa: E731
    check_expand(c, kv, scale, table, [200, 3, 90], w, 64, call())
    s = torch.cuda.Stream()
    ws = torch.empty(dsa.expand_kv_workspace_size(400, 512), dtype=torch.uint8, device="cuda")
    x = call(stream=s, workspace=ws)
    s.synchronize()
    check_expand(c, kv, scale, table, [200, 3, 90], w, 64, x)
    with pytest.raises(dsa.DsaError, match="workspace"):
        call(workspace=ws[:-16])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x = call()
    lens.copy_(i32([1, 199, 128]))
    graph.replay()
    torch.cuda.synchronize()
    check_expand(c, kv, scale, table, [1, 199, 128], w, 64, x)


# ---- prompt_mla --------------------------------------------------------------------------


def definition(c, q, kv, k_rope, cu_q, cu_k, pos, scale):
    """out, lse, and the bounds on both, in 64 bits.  cu_q, cu_k, pos: lists."""
    T, H, dn, dv = q.shape[0], c["heads"], c["dn"], c["dv"]
    K = dn + c["dr"]
    out = torch.zeros((T, H, dv), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(cu_q) - 1):
        for t0 in range(cu_q[r], cu_q[r + 1], 256):
            t1 = min(t0 + 256, cu_q[r + 1])
            last = torch.tensor(pos[t0:t1], device="cuda")
            n = int(last.max()) + 1
            if n <= 0:
                continue
            at = slice(cu_k[r], cu_k[r] + n)
            seen = (torch.arange(n, device="cuda")[None, :] <= last[:, None])[None]
            k = kv[at][..., :dn].double()
            if c["dr"]:
                k = torch.cat((k, k_rope[at].double()[:, None].expand(-1, H, -1)), -1)
            qq = q[t0:t1].double()
            z = torch.einsum("thd,khd->htk", qq, k) * scale
            d = torch.einsum("thd,khd->htk", qq.abs(), k.abs()) * scale * (K + 2) * 2.0**-23 + 2.0**-22 * z.abs()
            d = torch.where(seen & torch.isfinite(d), d, 0.0).amax(-1)
            z = torch.where(seen, z, -math.inf)
            live = last >= 0
            m = torch.logsumexp(z, -1)
            p = torch.where(seen, torch.softmax(z, -1), 0.0)  # (of logits so large that m + ln n is m, too)
            v = kv[at][..., dn:].double()
            # a value that a token does not see does not reach it
            vz, odd = torch.nan_to_num(v, 0.0, 0.0, 0.0), ~torch.isfinite(v)
            o = torch.einsum("htk,khd->thd", p, vz)
            if bool(odd.any()):
                hit = torch.einsum("htk,khd->thd", seen.expand(H, -1, -1).double(), odd.double()) > 0
                o = torch.where(hit, math.nan, o)
            A = torch.einsum("htk,khd->thd", p, vz.abs())
            sums = 2.0**-21 + n / 8 * 2.0**-23
            out[t0:t1] = torch.where(live[:, None, None], o, 0.0)
            lse[t0:t1] = torch.where(live[:, None], m.t(), -math.inf)
            b_out[t0:t1] = 2.0**-8 * o.abs() + A * (2.0**-8 + 2 * d.t()[..., None] + sums + n * 2.0**-23)
            b_lse[t0:t1] = d.t() + sums + 2.0**-22 * m.t().abs()
    return out, lse, b_out, b_lse


def check_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, scale, got, rms=True):
    out, lse = got
    w_out, w_lse, b_out, b_lse = definition(c, q, kv, k_rope, cu_q, cu_k, pos, scale)
    near(out, w_out, b_out)
    near(lse, w_lse, b_lse)
    fine = torch.isfinite(w_out)
    if rms and float(w_out[fine].norm()) > 0:
        assert float((out.double() - w_out)[fine].norm() / w_out[fine].norm()) <= 3.2e-3


def batch(c, lens, g, pad=0, extra=0, strided=0):
    """Requests of (new, ctx) tokens; `extra` padding tokens and rows."""
    cu_q, cu_k, pos = [0], [0], []
    for new, ctx in lens:
        cu_q.append(cu_q[-1] + new)
        cu_k.append(cu_k[-1] + ctx)
        pos += list(range(ctx - new, ctx))
    pos += [-1] * extra
    H, dn, dr, dv = c["heads"], c["dn"], c["dr"], c["dv"]
    q = rows((cu_q[-1] + extra, H, dn + dr), g, strided)
    kv, k_rope = rows((cu_k[-1] + extra, H, dn + dv), g, strided), rows((cu_k[-1] + extra, dr), g, strided)
    return q, kv, k_rope, cu_q, cu_k, pos


def run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, scale=None, status=0, **kw):
    scale = (c["dn"] + c["dr"])**-0.5 if scale is None else scale
    st = i32([0])
    got = dsa.prompt_mla(q, kv, k_rope if c["dr"] else None, i32(cu_q), i32(cu_k), i32(pos), d_nope=c["dn"],
                         softmax_scale=scale, dev_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == status
    return got


LENS = [[(1, 1)], [(1, 130)], [(2, 2), (1, 1)], [(127, 127)], [(128, 128)], [(129, 129)], [(255, 300)], [(256, 256), (1, 129)],
        [(257, 257)], [(300, 1000)], [(0, 5), (3, 3), (0, 0), (40, 200), (0, 1)], [(5, 640), (70, 70), (513, 513)]]


@pytest.mark.parametrize("c", SHAPES, ids=lambda c: f"{c['heads']}x{c['dn']}")
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_prompt_matches_the_definition(c, lens):
    g = gen(sum(a + b for a, b in lens))
    x = batch(c, lens, g, extra=3 if len(lens) > 1 else 0, strided=8 if len(lens) > 2 else 0)
    check_prompt(c, *x, (c["dn"] + c["dr"])**-0.5, run_prompt(c, *x))


@pytest.mark.parametrize("c", [LARGE, SMALL, ODD], ids=lambda c: f"{c['heads']}x{c['dn']}")
@pytest.mark.parametrize("splits", [2, 3, 8, 64])
def test_prompt_splits(c, splits):
    x = batch(c, [(5, 700), (130, 300), (1, 1), (3, 129)], gen(splits), extra=2)
    check_prompt(c, *x, (c["dn"] + c["dr"])**-0.5, run_prompt(c, *x, num_splits=splits))
    op, lp = dsa.prompt_mla_fwd(x[0], x[1], x[2], i32(x[3]), i32(x[4]), i32(x[5]), d_nope=c["dn"], softmax_scale=0.1,
                                num_splits=splits)
    assert op.shape == (splits, x[0].shape[0], c["heads"], c["dv"]) and lp.shape == op.shape[:3]
    assert float(op[:, -1].abs().max()) == 0 and float(lp[:, -1].max()) == -math.inf


def test_prompt_any_last_positions():
    """No mask, a limit for each token in no order, tokens that see nothing between others."""
    c, g = LARGE, gen(11)
    q, kv, k_rope, cu_q, cu_k, pos = batch(c, [(300, 500), (60, 70)], g)
    pos = torch.randint(-1, 500, (300,), generator=g, device="cuda").tolist() + [69] * 60
    pos[5:20] = [-1] * 15
    check_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, 192**-0.5, run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos))
    check_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, 192**-0.5, run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, num_splits=3))
    out, lse = run_prompt(c, q, kv, k_rope, cu_q, cu_k, [-1] * 360)  # requests that the layout refused
    assert float(out.abs().max()) == 0 and float(lse.max()) == -math.inf


@pytest.mark.parametrize("c", [LARGE, SMALL], ids=["64", "16"])
def test_prompt_logits_far_apart(c):
    """Peaked and growing logits (the running maximum moves), a scale of 0, and huge equal ones."""
    g, K = gen(12), c["dn"] + c["dr"]
    q, kv, k_rope, cu_q, cu_k, pos = batch(c, [(200, 600), (150, 150)], g)
    check_prompt(c, 6 * q, kv, k_rope, cu_q, cu_k, pos, K**-0.5, run_prompt(c, 6 * q, kv, k_rope, cu_q, cu_k, pos))
    grow = kv.clone()
    grow[..., :c["dn"]] = kv[..., :c["dn"]].abs() * (torch.arange(750, device="cuda") / 64)[:, None, None].to(BF16)
    up = q.abs()
    for s in (K**-0.5, 0.01):
        check_prompt(c, up, grow, k_rope, cu_q, cu_k, pos, s, run_prompt(c, up, grow, k_rope, cu_q, cu_k, pos, scale=s))
        check_prompt(c, -up, grow, k_rope, cu_q, cu_k, pos, s, run_prompt(c, -up, grow, k_rope, cu_q, cu_k, pos, scale=s))
    check_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, 0.0, run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, scale=0.0))
    big = torch.full_like(kv, 2.0**30)
    big[..., c["dn"]:] = kv[..., c["dn"]:]
    one = torch.zeros_like(q)
    one[..., 0] = 2.0**30
    check_prompt(c, one, big, k_rope, cu_q, cu_k, pos, 1.0, run_prompt(c, one, big, k_rope, cu_q, cu_k, pos, scale=1.0))
    check_prompt(c, -one, big, k_rope, cu_q, cu_k, pos, 1.0, run_prompt(c, -one, big, k_rope, cu_q, cu_k, pos, scale=1.0))


@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("splits", [1, 2])
def test_prompt_what_is_not_seen_does_not_reach_a_token(what, splits):
    c, g = LARGE, gen(13)
    q, kv, k_rope, cu_q, cu_k, pos = batch(c, [(150, 150), (20, 290), (3, 3)], g, extra=200)
    clean = run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, num_splits=splits)
    # behind the last request, in rows of no request's tokens, and at positions that only later tokens see
    kv2, rope2, q2 = kv.clone(), k_rope.clone(), q.clone()
    kv2[cu_k[-1]:], rope2[cu_k[-1]:], q2[cu_q[-1]:] = what, what, what
    kv2[60, :, 130] = what                    # a value, position 60 of request 0
    kv2[100] = what                           # key and value, position 100
    kv2[150 + 280, 5], rope2[150 + 284] = what, what
    got = run_prompt(c, q2, kv2, rope2, cu_q, cu_k, pos, num_splits=splits)
    # tokens before position 100 are as they were, but for the value's column
    col = torch.arange(128, device="cuda") != 2
    assert torch.equal(got[0][:60], clean[0][:60]) and torch.equal(got[1][:100], clean[1][:100])
    assert torch.equal(got[0][60:100][..., col], clean[0][60:100][..., col])
    assert not bool(torch.isfinite(got[0][60:150, :, 2]).any())
    assert not bool(torch.isfinite(got[0][100:150]).any()) and bool(torch.isnan(got[0][100:150]).all())
    assert bool(torch.isnan(got[1][100:150]).all())
    at = 150 + 10  # request 1's token of position 280
    assert torch.equal(got[0][150:at], clean[0][150:at]) and torch.equal(got[1][150:at], clean[1][150:at])
    other = torch.arange(64, device="cuda") != 5
    assert torch.equal(got[0][at:at + 4][:, other], clean[0][at:at + 4][:, other])
    assert bool(torch.isnan(got[0][at:at + 4, 5]).all()) and bool(torch.isnan(got[0][at + 4:170]).all())
    assert torch.equal(got[0][170:], clean[0][170:]) and torch.equal(got[1][170:], clean[1][170:])


def test_prompt_data_errors():
    c, g = SMALL, gen(14)
    q, kv, k_rope, cu_q, cu_k, pos = batch(c, [(30, 30), (30, 60), (30, 30)], g)
    good = run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos)

    def dead(got, a, b):
        assert float(got[0][a:b].abs().max()) == 0 and float(got[1][a:b].max()) == -math.inf

    def same(got, a, b):
        assert torch.equal(got[0][a:b], good[0][a:b]) and torch.equal(got[1][a:b], good[1][a:b])

    p = list(pos)
    p[3], p[40], p[41] = 30, -2, 60
    got = run_prompt(c, q, kv, k_rope, cu_q, cu_k, p, status=dsa.DEV_BAD_QPOS)
    for a, b in ((3, 4), (40, 42)):
        dead(got, a, b)
    for a, b in ((0, 3), (4, 40), (42, 90)):
        same(got, a, b)
    for bad in ([0, 30, 90, 121], [0, 30, 90, 2**31 - 1]):  # rows past the tensor
        got = run_prompt(c, q, kv, k_rope, cu_q, bad, pos, status=dsa.DEV_BAD_INDEX | dsa.DEV_BAD_QPOS)
        dead(got, 60, 90)
        same(got, 0, 60)
    got = run_prompt(c, q, kv, k_rope, cu_q, [0, -5, 90, 120], pos, status=dsa.DEV_BAD_INDEX | dsa.DEV_BAD_QPOS)
    dead(got, 0, 60)
    same(got, 60, 90)
    # a request whose token range is none: its tokens stay as they are
    out, lse = torch.full_like(good[0], 7.0), torch.full_like(good[1], 7.0)
    got = run_prompt(c, q, kv, k_rope, [0, 30, 60, 91], cu_k, pos, status=dsa.DEV_BAD_INDEX, buffers=dict(out=out, lse=lse))
    same(got, 0, 60)
    assert bool((out[60:] == 7).all()) and bool((lse[60:] == 7).all())
    # no requests at all: every token is padding
    out, lse = run_prompt(c, q, kv, k_rope, [0], [0], pos)
    dead((out, lse), 0, 90)
    # no rows
    out, lse = run_prompt(c, q, kv[:0], k_rope[:0], [0, 90], [0, 0], [-1] * 90)
    dead((out, lse), 0, 90)
    assert run_prompt(c, q[:0], kv, k_rope, [0, 0], [0, 5], [])[0].shape == (0, 16, 32)


def test_prompt_streams_graphs_and_outputs(both_ways):
    c, g = LARGE, gen(15)
    q, kv, k_rope, cu_q, cu_k, pos = batch(c, [(100, 300), (56, 56)], g, extra=100)
    args = (q, kv, k_rope)
    tq, tk, tp = i32(cu_q), i32(cu_k), i32(pos)
    torch.cuda.synchronize()
    call = lambda **k: dsa.prompt_mla(*args, tq, tk, tp, d_nope=128, softmax_scale=192**-0.5, **k)  # noqa: E731
    want = call()
    check_prompt(c, *args, cu_q, cu_k, pos, 192**-0.5, want)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = [call(stream=s) for s in streams for _ in range(3)]
    guard = torch.full((258, 64, 128), 7.0, device="cuda", dtype=BF16)
    with torch.cuda.stream(streams[0]):
        call(buffers=dict(out=guard[1:257]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(z, want[1]) for o, z in got)
    assert torch.equal(guard[1:257], want[0]) and bool((guard[0] == 7).all()) and bool((guard[257] == 7).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    lens = [(10, 40), (200, 316)]  # the graph follows its lengths
    _, _, _, cu_q, cu_k, pos = batch(c, lens, gen(1), extra=46)
    tq.copy_(i32(cu_q)), tk.copy_(i32(cu_k)), tp.copy_(i32(pos))
    q.copy_(rows((256, 64, 192), g))
    graph.replay()
    torch.cuda.synchronize()
    check_prompt(c, *args, cu_q, cu_k, pos, 192**-0.5, got)


def test_prompt_many_requests():
    c, g = SMALL, gen(16)
    lens = [(int(a), int(a + b)) for a, b in torch.randint(0, 4, (8192, 2), generator=torch.Generator().manual_seed(1)).tolist()]
    q, kv, k_rope, cu_q, cu_k, pos = batch(c, lens, g, extra=1000)
    out, lse = run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos)
    # every token on its own: its request's rows gathered, 7 at most
    t = torch.arange(cu_q[-1], device="cuda")
    r = torch.searchsorted(i32(cu_q)[1:], t.to(I32), right=True)
    last, j = i32(pos)[:cu_q[-1]], torch.arange(7, device="cuda")
    n = (i32(cu_k)[:-1][r][:, None] + j).clamp(max=kv.shape[0] - 1).long()
    k = torch.cat((kv[n][..., :32], k_rope[n][:, :, None].expand(-1, -1, 16, -1)), -1).double()
    z = torch.einsum("thd,tkhd->thk", q[t].double(), k) * 48**-0.5
    z = z.masked_fill((j[None] > last[:, None])[:, None], -math.inf)
    p = torch.softmax(z, -1)
    o = torch.einsum("thk,tkhd->thd", p, kv[n][..., 32:].double())
    A = torch.einsum("thk,tkhd->thd", p, kv[n][..., 32:].double().abs())
    near(out[:cu_q[-1]], o, 2.0**-8 * o.abs() + A * (2.0**-8 + 2.0**-12))
    near(lse[:cu_q[-1]], torch.logsumexp(z, -1), 2.0**-13)
    assert float(out[cu_q[-1]:].abs().max()) == 0 and float(lse[cu_q[-1]:].max()) == -math.inf


def test_prompt_rows_past_32_bit_offsets():
    """Keys and values of more than 2^31 elements (4.6 GB), the request at their end."""
    c, N = LARGE, 140_000
    g = gen(17)
    kv = torch.zeros((N, 64, 256), dtype=BF16, device="cuda")
    k_rope = torch.zeros((N, 64), dtype=BF16, device="cuda")
    new, ctx = 40, 260
    kv[N - ctx:] = rows((ctx, 64, 256), g)
    k_rope[N - ctx:] = rows((ctx, 64), g)
    q = rows((new + 1, 64, 192), g)
    pos = [7] + list(range(ctx - new, ctx))
    cu_q, cu_k = [0, 1, new + 1], [0, N - ctx, N]
    check_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, 192**-0.5, run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos))


# ---- together -------------------------------------------------------------------------------


def test_a_prompt_in_both_forms():
    """lengths -> layout -> norm, rotation and cache write -> attention in both forms, which agree."""
    c, P, dev = LARGE, 64, "cuda"
    g = gen(20)
    w = weight(c, g)
    pages, ctx, new = 40, [70, 0, 500], [33, 140, 1]
    table = torch.full((3, 12), -1, dtype=I32, device=dev)
    held = [-(-n // P) for n in ctx]
    table[0, :held[0]], table[2, :held[2]] = i32([3, 9]), i32([11, 4, 20, 5, 6, 7, 8, 1])
    free = i32([p for p in range(pages) if p not in (3, 9, 11, 4, 20, 5, 6, 7, 8, 1)])
    st = i32([0])
    lay = dsa.batch_layout(i32(ctx), i32(new), i32(held), table, free, i32([0]), page_size=P, num_pages=pages, capacity=180,
                           dev_status=st)
    kv = torch.randint(0, 120, (pages * P, 576), generator=g, dtype=torch.uint8, device=dev)
    sc = torch.rand(pages * P, generator=g, device=dev) * 0.01 + 0.001
    angle = torch.arange(600, device=dev)[:, None] * 10000.0**(-torch.arange(0, 64, 2, device=dev) / 64)[None, :]
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
    k_new, q = rows((180, 1, 576), g), rows((180, 64, 192), g)
    kw = 1 + 0.1 * torch.randn(512, generator=g, device=dev)
    dsa.qk_norm_rope(None, k_new, lay.q_pos, cos_sin, d_rope=64, k_weight=kw, slot=lay.slot, kv=kv, kv_scale=sc, dev_status=st)
    q, _ = dsa.qk_norm_rope(q, None, lay.q_pos, cos_sin, d_rope=64, q_out=torch.zeros_like(q), dev_status=st)
    scale = 192**-0.5
    # the absorbed form
    ql = dsa.absorb_q(q, w, d_rope=64)
    o, lse = dsa.chunk_mla(ql, kv, sc, table, lay.q_req, lay.q_pos, d_latent=512, d_rope=64, page_size=P, softmax_scale=scale,
                           max_ctx=512, dev_status=st)
    y = dsa.project_out(o, w, d_nope=128)
    # the expanded form
    x = dsa.expand_kv(kv, sc, table, lay.ctx_len, w, d_rope=64, page_size=P, capacity=800, dev_status=st)
    y2, lse2 = dsa.prompt_mla(q, x.kv, x.k_rope, lay.cu_q, x.cu_k, lay.q_pos, d_nope=128, softmax_scale=scale, dev_status=st)
    assert int(st) == 0
    # in 64 bits, from the cache
    slot = torch.cat([table[r].long()[torch.arange(n, device=dev) // P] * P + torch.arange(n, device=dev) % P
                      for r, n in enumerate(lay.ctx_len.tolist())])
    rows64 = kv[slot].view(torch.float8_e4m3fn).double() * sc[slot].double()[:, None]
    full = torch.einsum("nl,hdl->nhd", rows64[:, :512], w.double())
    want, want_lse, _, _ = definition(c, q, full, rows64[:, 512:], lay.cu_q.tolist(), x.cu_k.tolist(), lay.q_pos.tolist(), scale)
    n = int(lay.cu_q[-1])
    assert n == 174
    # roundings on the way, each 2^-8 / sqrt(3) of its values at most (root mean square).  Absorbed:
    # queries (they move logits: next), weights, latent outputs, outputs; expanded: keys, values, weights, outputs.
    # A logit's standard deviation s moves weights by s 2.25e-3: s < 4 here.
    assert float(want_lse[:n].abs().max()) < 30
    for a, b in ((y, lse), (y2, lse2)):
        rel = float((a[:n].double() - want[:n]).norm() / want[:n].norm())
        assert rel <= 2.25e-3 * math.sqrt(1 + 1 + 1 + 16), rel
        assert float(a[n:].abs().max()) == 0 and float(b[n:].max()) == -math.inf
        assert float((b[:n].double() - want_lse[:n]).abs().max()) <= 0.05


def test_calls_of_several_threads_and_graphs_at_once():
    """Host threads on streams of their own, and two captured steps replayed side by side: the same bits as alone."""
    import threading

    c, g = LARGE, gen(30)
    w = weight(c, g)
    q, o = rows((70, 64, 192), g), rows((70, 64, 512), g)
    kv, scale, table = cache(c, 2, 300, 64, g)
    lens = i32([300, 211])
    pq, _, _, cu_q, cu_k, pos = batch(c, [(40, 300), (30, 211)], g)
    tq, tp = i32(cu_q), i32(pos)

    def step():
        x = dsa.expand_kv(kv, scale, table, lens, w, d_rope=64, page_size=64, capacity=511)
        return (dsa.absorb_q(q, w, d_rope=64), dsa.project_out(o, w, d_nope=128), x.kv,
                *dsa.prompt_mla(pq, x.kv, x.k_rope, tq, x.cu_k, tp, d_nope=128, softmax_scale=0.07),
                *dsa.prompt_mla(pq, x.kv, x.k_rope, tq, x.cu_k, tp, d_nope=128, softmax_scale=0.07, num_splits=2))

    want = step()
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i] = step()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # pragma: no cover
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for r in got.values():
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, _, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_prompt_requests_of_every_length():
    """Queries from 1 to 300 behind contexts that end anywhere in a tile: one call, each request checked."""
    c, g = SMALL, gen(31)
    lens = [(n, n + (37 * n) % 290) for n in range(1, 301, 7)]
    x = batch(c, lens, g, extra=5)
    check_prompt(c, *x, 48**-0.5, run_prompt(c, *x))
    check_prompt(c, *x, 48**-0.5, run_prompt(c, *x, num_splits=5))
