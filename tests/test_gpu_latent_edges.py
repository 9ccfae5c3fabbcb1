"""GPU tests of latent attention's other form and the products around it at the
edges of what their calls allow."""
import math

import pytest
import torch

import dsa_sparse_mla_topk_gb300 as dsa
import test_gpu_latent_ops as ops
from test_gpu_latent_ops import BF16, LARGE, SMALL, both_ways, gen, i32, rows, weight  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dsa_sparse_mla_topk_gb300 import build
    build.build()
    dsa.load_library()


def shape(heads, dn=32, dr=16, dv=32, dl=64):
    return dict(heads=heads, dn=dn, dr=dr, dv=dv, dl=dl)


# ---- more than 64 heads ----------------------------------------------------------------


@pytest.mark.parametrize("c", [shape(65), shape(96, 128, 64, 128), shape(128, 128, 64, 128), shape(200, 48, 0, 80),
                               shape(1024, 16, 16, 16)], ids=lambda c: f"{c['heads']}x{c['dn']}")
@pytest.mark.parametrize("splits", [1, 2, 5, None])
def test_prompt_many_heads(c, splits, both_ways):  # noqa: F811
    """Heads past 64, in one share, in several, and in as many as the rule takes."""
    x = ops.batch(c, [(3, 700), (20, 150), (1, 1)], gen(c["heads"]), extra=2)
    scale = (c["dn"] + c["dr"])**-0.5
    ops.check_prompt(c, *x, scale, ops.run_prompt(c, *x, num_splits=splits))


def test_prompt_many_heads_shares_by_the_rule(both_ways):  # noqa: F811
    """A chunk whose number of shares the rule picks from a long context: 96 heads take more than one."""
    c, new, ctx = shape(96, 16, 0, 16), 256, 16_384
    assert dsa.pick_prompt_splits(new, 1, 96, ctx, num_sms=152) > 1
    x = ops.batch(c, [(new, ctx)], gen(3))
    ops.check_prompt(c, *x, 0.25, ops.run_prompt(c, *x))


@pytest.mark.parametrize("c", [shape(65, 48, 16, 80, 208), shape(128, 48, 16, 80, 208), shape(300, 48, 16, 80, 208),
                               shape(1, 16, 0, 16, 16), shape(1, 16, 64, 16, 512), shape(1, 128, 16, 112, 48)],
                         ids=lambda c: f"{c['heads']}x{c['dn']}x{c['dl']}")
def test_products_and_expansion_one_and_many_heads(c):
    g, n = gen(c["heads"]), 150
    w = weight(c, g)
    q, o = rows((n, c["heads"], c["dn"] + c["dr"]), g), rows((n, c["heads"], c["dl"]), g)
    ops.check_absorb(c, q, w, dsa.absorb_q(q, w, d_rope=c["dr"]))
    ops.check_project(c, o, w, dsa.project_out(o, w, d_nope=c["dn"]))
    kv, scale, table = ops.cache(c, 3, 200, 48, g)
    lens = [200, 0, 131]
    ops.check_expand(c, kv, scale, table, lens, w, 48, ops.run_expand(c, kv, scale, table, lens, w, 48, 340))


@pytest.mark.parametrize("heads,d_v", [(64, 512), (65, 128), (96, 80), (1024, 16), (1024, 128), (1000, 4)])
@pytest.mark.parametrize("splits", [1, 3, 64])
def test_combine_many_heads(heads, d_v, splits):
    """out = sum_s exp(lse_s - lse) o_s.  exp's argument is rounded by 2^-24 of |lse_s - lse| (below 40) and its
    own error is 2^-22; lse by 2^-22 of its value (below 30) and the splits' additions: a weight is off by (40 +
    120 + 4 + splits) 2^-24 of itself, the sum by the splits' additions more, and a rounding to bf16."""
    n, g = 3, gen(heads + splits)
    o = torch.randn((splits, n, heads, d_v), generator=g, device="cuda")
    l = torch.randn((splits, n, heads), generator=g, device="cuda") * 3
    l[splits // 2, 1, ::3] = -math.inf
    out, lse = dsa.combine(o, l)
    want = torch.logsumexp(l.double(), 0)
    w = torch.where(torch.isfinite(l), (l.double() - want).exp(), 0.0)
    off = (164 + splits) * 2.0**-24
    res = (w[..., None] * o.double()).sum(0)
    ops.near(out, res, 2.0**-8 * res.abs() + (off + (splits + 1) * 2.0**-24) * (w[..., None] * o.double().abs()).sum(0))
    ops.near(lse, want, 2.0**-22 * want.abs() + off)


# ---- values that are not finite ----------------------------------------------------------


@pytest.mark.parametrize("c", [LARGE, shape(5, 48, 16, 80), shape(3, 16, 0, 16), shape(2, 128, 64, 64)],
                         ids=lambda c: f"{c['heads']}x{c['dv']}")
@pytest.mark.parametrize("splits", [1, 3])
def test_prompt_bad_values_among_any_last_positions(c, splits):
    """A token that sees nothing makes every tile of its query tile one that is seen in part; bad values stand
    in some tiles, columns and heads, next to each other and far apart, and others read past them."""
    g = gen(c["heads"] + splits)
    q, kv, k_rope, cu_q, cu_k, pos = ops.batch(c, [(300, 1500), (130, 700), (5, 260)], g)
    r = torch.Generator().manual_seed(5)
    pos = [int(torch.randint(-1, n, (1,), generator=r)) for m, n in ((300, 1500), (130, 700), (5, 260)) for _ in range(m)]
    for t in (0, 140, 299, 300, 429, 434):
        pos[t] = -1
    pos[1], pos[141], pos[431] = 1499, 1499, 259
    H, dn, dv = c["heads"], c["dn"], c["dv"]
    for at, h, d, what in ((0, 0, 0, math.nan), (127, 1, dv - 1, math.inf), (128, 1, 3, -math.inf), (640, 0, 5, math.nan),
                           (641, 0, 5, math.nan), (300, 0, 5, math.inf), (1499, H - 1, dv // 2, math.nan),
                           (1500 + 699, 0, 8, math.inf), (1500 + 3, 1, 9, -math.nan), (2200 + 130, H - 1, 15, math.nan)):
        kv[at, h, dn + d] = what
    kv[900, H - 1, dn:] = math.nan
    ops.check_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, 0.1, ops.run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, scale=0.1,
                                                                            num_splits=splits))


@pytest.mark.parametrize("dv", [32, 128])
@pytest.mark.parametrize("at", [256, 384, 511, 640])
def test_prompt_bad_values_behind_what_half_the_tokens_see(dv, at):
    """The first 128 tokens end before a bad value that the next 128 see, in heads that take turns with heads whose first
    value is bad in every column: each token's results by what it sees alone."""
    c, g = shape(608, 32, 16, dv), gen(at + dv)
    q, kv, k_rope, cu_q, cu_k, pos = ops.batch(c, [(256, 700)], g)
    pos = [(7 * t) % 256 if t < 128 else 699 - t % 3 for t in range(256)]
    pos[9] = pos[140] = -1
    clean = ops.run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, num_splits=1)
    kv[0, ::2, 32:] = math.nan
    kv[at, 1::2, 32 + dv - 3] = math.inf
    dead = torch.tensor(pos, device="cuda") < 0
    for _ in range(20):
        out, lse = ops.run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos, num_splits=1)
        assert torch.equal(lse, clean[1])
        assert bool(torch.isnan(out[~dead][:, ::2]).all()) and torch.equal(out[dead], clean[0][dead])
        assert torch.equal(out[:128, 1::2], clean[0][:128, 1::2])
        col = torch.arange(dv, device="cuda") != dv - 3
        assert torch.equal(out[128:, 1::2][..., col], clean[0][128:, 1::2][..., col])
        assert bool(torch.isnan(out[128:, 1::2, dv - 3][~dead[128:]]).all())


@pytest.mark.parametrize("every", [False, True], ids=["two bad values", "bad values in every tile"])
def test_prompt_bad_values_in_a_context_of_millions_of_rows(every):
    """The work beside a tile's products is bounded for every tile, so that no wait of the call's runs out."""
    c, n, g = shape(1, 16, 0, 16), 1 << 24, gen(9)
    kv, q = rows((n, 1, 32), g), rows((4, 1, 16), g)
    kv[1000, 0, 16 + 3], kv[n - 3, 0, 16 + 7] = math.nan, math.inf
    if every:
        kv[1000:, 0, 16 + 3] = math.inf
        kv[5000::50, 0, 16 + 5] = math.nan
    pos = [-1, 999, n // 2, n - 1]
    ops.check_prompt(c, q, kv, None, [0, 4], [0, n], pos, 0.25,
                     ops.run_prompt(c, q, kv, None, [0, 4], [0, n], pos, scale=0.25, num_splits=1), rms=False)


# ---- scales --------------------------------------------------------------------------------


@pytest.mark.parametrize("c", [LARGE, SMALL], ids=["64", "16"])
@pytest.mark.parametrize("scale", [0.0, 2.0**-140, 2.0**-126, 2.0**-124, 3e-37, 2.0**-118])
@pytest.mark.parametrize("splits", [1, 3])
def test_prompt_small_scales_of_large_logits(c, scale, splits):
    """Sums up to 2^126 under scales down to 0: the logits are what their product is."""
    q, kv, k_rope, cu_q, cu_k, pos = ops.batch(c, [(140, 400), (30, 30)], gen(21))
    one = torch.zeros_like(q)
    one[..., 0] = q[..., 0].clamp(-1, 1) * 2.0**63
    kv[..., 0] = kv[..., 0].clamp(-1, 1) * 2.0**63
    ops.check_prompt(c, one, kv, k_rope, cu_q, cu_k, pos, scale, ops.run_prompt(c, one, kv, k_rope, cu_q, cu_k, pos, scale=scale,
                                                                                num_splits=splits))


# ---- data errors ---------------------------------------------------------------------------


@pytest.mark.parametrize("bad", [0, 1, 37, 199])
@pytest.mark.parametrize("busy", [False, True], ids=["alone", "beside others"])
def test_prompt_ranges_that_are_none_are_told(bad, busy):
    """A request whose token range goes down or past the tokens, wherever it stands and whichever CTAs run first:
    told, its tokens left alone, the others' results as without it."""
    c, R, g = SMALL, 200, gen(7)
    q, kv, k_rope, cu_q, cu_k, pos = ops.batch(c, [(300, 330)] * R, g)
    want = ops.run_prompt(c, q, kv, k_rope, cu_q, cu_k, pos)
    cut = list(cu_q)
    cut[bad + 1] = len(pos) + 1 if bad == R - 1 else 300 * (bad + 2) + 5  # too high here, and so down at the next
    other = torch.cuda.Stream()
    for _ in range(5):
        out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
        torch.cuda.synchronize()
        if busy:
            with torch.cuda.stream(other):
                for _ in range(3):
                    dsa.prompt_mla(q, kv, k_rope, i32(cu_q), i32(cu_k), i32(pos), d_nope=32, softmax_scale=0.1)
        st = i32([0])
        dsa.prompt_mla(q, kv, k_rope, i32(cut), i32(cu_k), i32(pos), d_nope=32, softmax_scale=48**-0.5, dev_status=st,
                       buffers=dict(out=out, lse=lse))
        torch.cuda.synchronize()
        # (the request before the one that goes down takes tokens that are the next one's: past their contexts)
        assert int(st) & dsa.DEV_BAD_INDEX
        good = torch.ones(len(pos), dtype=torch.bool, device="cuda")
        good[300 * bad:300 * (bad + 2) + 5] = False
        assert torch.equal(out[good], want[0][good]) and torch.equal(lse[good], want[1][good])
        if bad == R - 1:
            assert bool((out[300 * bad:] == 7).all()) and bool((lse[300 * bad:] == 7).all())


# ---- the largest sizes ---------------------------------------------------------------------


@pytest.mark.parametrize("op", ["absorb", "project"])
@pytest.mark.parametrize("n", [2**31 - 1, 2**31 - 128, 2**31 - 255])
def test_products_of_the_most_tokens(op, n):
    """One head of 16 values and as many tokens as there may be: overlapping rows (a token stride of 8) of 32 GiB,
    outputs of 64 GiB.  All written; the first, the last and some between against 64 bits."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GiB of free memory")
    g = gen(3)
    x = torch.empty(8 * n + 8, dtype=BF16, device="cuda").normal_(generator=g).as_strided((n, 1, 16), (8, 16, 1))
    w = weight(shape(1, 16, 0, 16, 16), g)
    y = torch.full((n, 1, 16), math.nan, dtype=BF16, device="cuda")
    st = i32([0])
    if op == "absorb":
        dsa.absorb_q(x, w, d_rope=0, q_out=y, dev_status=st)
    else:
        dsa.project_out(x, w, d_nope=16, out=y, dev_status=st)
    assert int(st) == 0
    b = w[0, :16].double() if op == "absorb" else w[0, 16:].double().t()
    for at in (0, 2**30 - 500, 2**31 - 2**20 - 77, n - 1000):
        ops.near_product(y[at:at + 1000, 0], x[at:at + 1000, 0].double(), b, 16)
    for at in range(0, n, 2**27):
        assert not bool(torch.isnan(y[at:at + 2**27]).any()), at
    del x, y
    torch.cuda.empty_cache()


def test_products_results_past_32_bit_offsets():
    """Results of more than 2^31 values: the first rows, those around 2^31 values, the last."""
    c, g = LARGE, gen(40)
    w = weight(c, g)
    n = 2**31 // (64 * 576) + 300
    q = rows((n, 64, 192), g)
    y = dsa.absorb_q(q, w, d_rope=64)
    assert y.numel() > 2**31
    for at in (0, n - 400, n - 150):
        ops.check_absorb(c, q[at:at + 150], w, y[at:at + 150])
    del q, y
    n = 2**31 // (64 * 128) + 300
    o = rows((n, 64, 512), g)
    y = dsa.project_out(o, w, d_nope=128)
    assert y.numel() > 2**31
    for at in (0, n - 400, n - 150):
        ops.check_project(c, o[at:at + 150], w, y[at:at + 150])
    del o, y
    torch.cuda.empty_cache()


def test_expand_results_past_32_bit_offsets():
    c, g, P = LARGE, gen(41), 64
    n = 2**31 // (64 * 256) + 300
    kv, scale, table = ops.cache(c, 2, n, P, g)
    w = weight(c, g)
    x = ops.run_expand(c, kv, scale, table, [n, 77], w, P, n + 100)
    assert x.cu_k.tolist() == [0, n, n + 77] and x.kv[:n].numel() > 2**31
    for r, at, m in ((0, 0, 150), (0, n - 400, 400), (1, 0, 77)):
        p = torch.arange(at, at + m, device="cuda")
        slot = table[r].long()[p // P] * P + p % P
        a = kv[slot].view(torch.float8_e4m3fn).double() * scale[slot].double()[:, None]
        out = slice(n * r + at, n * r + at + m)
        ops.near_product(x.kv[out].flatten(1), a[:, :512], w.double().flatten(0, 1).t(), 512)
        assert torch.equal(x.k_rope[out], a[:, 512:].float().to(BF16))
    del x
    torch.cuda.empty_cache()


# ---- workspaces ------------------------------------------------------------------------------


@pytest.mark.parametrize("c", ops.SHAPES, ids=lambda c: f"{c['heads']}x{c['dn']}")
def test_expand_whatever_the_workspace_holds(c, both_ways):  # noqa: F811
    """What a tile's rows past the last one read of the workspace (NaN here, and infinite scales) reaches nothing."""
    g, lens = gen(42), [100, 0, 133]
    kv, scale, table = ops.cache(c, 3, 140, 48, g)
    w = weight(c, g)
    want = ops.run_expand(c, kv, scale, table, lens, w, 48, 700)
    for fill in (0xff, 0x7f):  # NaN in both types; 0x7f7f, the largest finite values
        ws = torch.full((dsa.expand_kv_workspace_size(700, c["dl"]),), fill, dtype=torch.uint8, device="cuda")
        out = dsa.ExpandedKV(torch.full_like(want.kv, 7.0), torch.full_like(want.k_rope, 7.0), i32([0] * 4))
        x = dsa.expand_kv(kv, scale, table, i32(lens), w, d_rope=c["dr"], page_size=48, out=out, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(x, want))
    ops.check_expand(c, kv, scale, table, lens, w, 48, want)
