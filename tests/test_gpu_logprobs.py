"""GPU tests of token_logprobs against its definition in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, half an fp32 step of the value): d = z - m
is rounded once (u |d|), e^d is off by u |d| plus 2^-22 (the exponential's argument, its scale
to base 2: 2 u |d|, and its own error) of itself; a sum by (vocab / 256 + 64) u of its
terms' (256 partial sums at least, then tree and cluster); log1p by 2^-22 of
itself.  So, with S = 1 + rest:
  lse - m   is off by E = sum_{j != a} e^d (3 u |d| + 2^-22 + (vocab / 256 + 64) u) / S + 2^-22 log S,
  logprob   by E + 2 u |d_t| + u |logprob|,
  entropy   by E + sum e^d |d| (4 u |d| + 2^-22 + (vocab / 256 + 65) u) / S + entropy (E + 2^-22)."""
import math

import numpy as np
import pytest
import torch

import dsa_sparse_mla_topk_gb300 as dsa

pytestmark = pytest.mark.gpu
I32 = torch.int32
U = 2.0**-24


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


def logits(shape, dtype, seed, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * spread).to(dtype)


def check(z, tok, top, got, what=""):
    """Every row of z (no NaN, no +inf) and tok."""
    z = z.double()
    R, V = z.shape
    m = z.amax(1, keepdim=True)
    d = torch.where(z == -math.inf, -math.inf, z - torch.where(m == -math.inf, 0.0, m))
    e = d.exp()
    none = m[:, 0] == -math.inf
    at = z.argmax(1, keepdim=True)
    e1 = e.scatter(1, at, 0.0)
    dd = torch.where(d == -math.inf, 0.0, d)
    rest = e1.sum(1)
    S = 1 + rest
    adds = (V / 256 + 64) * U
    E = (e1 * (3 * U * dd.abs() + 2.0**-22 + adds)).sum(1) / S + 2.0**-22 * rest.log1p()
    lp = d - rest.log1p()[:, None]
    t = tok.long().clamp(min=0)[:, None]
    want = torch.where((tok < 0) | none, -math.inf, lp.gather(1, t)[:, 0])
    bound = E + 2 * U * dd.gather(1, t)[:, 0].abs() + U * want.abs()
    off = lambda a, b: torch.where(torch.isfinite(b), (a.double() - b).abs(), torch.where(a.double() == b, 0.0, math.inf))  # noqa: E731
    assert bool((off(got.logprob, want) <= bound).all()), (what, off(got.logprob, want), bound)
    ent = torch.where(none, 0.0, rest.log1p() - (e * dd).sum(1) / S)
    bound = E + (e * dd.abs() * (4 * U * dd.abs() + 2.0**-22 + adds + U)).sum(1) / S + ent * (E + 2.0**-22)
    assert bool((off(got.entropy, ent) <= bound).all()), (what, off(got.entropy, ent), bound)
    zt = z.gather(1, t)
    col = torch.arange(V, device="cuda")[None]
    rank = torch.where(tok < 0, -1, ((z > zt) | ((z == zt) & (col < t))).sum(1))
    assert torch.equal(got.rank.long(), rank), what
    assert got.top_ids.shape == got.top_logprobs.shape == (R, top)
    if not top:
        return
    k = min(top, V)
    val, ids = torch.sort(z, dim=1, descending=True, stable=True)
    val, ids = val[:, :k], torch.where(val[:, :k] == -math.inf, -1, ids[:, :k])
    full = torch.full((R, top), -1, dtype=torch.long, device="cuda")
    full[:, :k] = ids
    assert torch.equal(got.top_ids.long(), full), what
    want = torch.where(full < 0, -math.inf, lp.gather(1, full.clamp(min=0)))
    bound = E[:, None] + 2 * U * dd.gather(1, full.clamp(min=0)).abs() + U * want.abs()
    assert bool((off(got.top_logprobs, want) <= bound).all()), what


def run(z, tok, top, status=0, **kw):
    st = i32([0])
    got = dsa.token_logprobs(z, tok, top=top, dev_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st) == status
    return got


def some(R, V, seed=0):
    return torch.randint(0, V, (R,), generator=torch.Generator().manual_seed(seed), dtype=I32).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 64, 257, 1000, 4097, 32003, 50257, 131072, 262147])
@pytest.mark.parametrize("R,top", [(1, 0), (5, 20), (40, 1), (3, 64)])
def test_logprobs_match_the_definition(dtype, V, R, top):
    z, tok = logits((R, V), dtype, V + R), some(R, V)
    tok[0] = V - 1
    check(z, tok, top, run(z, tok, top))


@pytest.mark.parametrize("R", [200, 700, 1500])
def test_logprobs_many_rows(R):
    z, tok = logits((R, 5003), torch.bfloat16, R), some(R, 5003)
    check(z, tok, 8, run(z, tok, 8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,top", [(1, 3), (9, 20), (515, 64), (2049, 64), (8200, 1), (32003, 20), (70001, 0)])
def test_logprobs_more_rows_than_run_at_once(dtype, V, top):
    R = 1400
    z, tok = logits((R, V), dtype, V), some(R, V)
    z[5], z[-1, V // 2:] = 1.5, -math.inf
    z[7] = -math.inf
    tok[::9] = V - 1
    check(z, tok, top, run(z, tok, top))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [300, 8200, 140003])
def test_logprobs_shapes_of_rows(dtype, V):
    """Ties everywhere, all equal, ascending, descending, blocks of large ones, a sure token, masks, signed zeros."""
    j = torch.arange(V, device="cuda")
    z = logits((12, V), torch.float32, V)
    z[0] = (z[0]).round()
    z[1] = 2.5
    z[2] = j / V * 20
    z[3] = -j / V * 20
    z[4] = torch.where((j > V // 2) & (j <= V // 2 + 150), 9.0 + (j % 3) * 0.5, -3.0)
    z[5] = -40.0
    z[5, V // 3] = 20.0
    z[6, V // 7:] = -math.inf
    z[7] = -math.inf
    z[7, [3, V - 1]] = 1.5
    z[8] = -math.inf
    z[9] = torch.where(j % 2 == 0, 0.0, -0.0)
    z[10] = -60000.0 + (j % 5) * 1000.0
    z[11] = torch.where(j % 37 == 1, 60000.0, -60000.0)
    z = z.to(dtype)
    for seed, top in ((1, 5), (2, 64), (3, 0)):
        tok = some(12, V, seed)
        tok[5] = V // 3 if seed < 3 else 0
        tok[7], tok[8] = (V - 1, 4) if seed == 1 else (0, V - 1)
        tok[11] = 1
        check(z, tok, top, run(z, tok, top), f"top {top}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_logprobs_strides_and_unaligned_rows(dtype):
    for V, ld, at in ((1000, 1003, 1), (4096, 4160, 0), (30001, 30002, 3), (129, 131, 5), (65536, 65544, 8)):
        wide = logits((6, ld), dtype, V)
        wide = torch.cat((wide.flatten(), wide[0]))
        z = wide.as_strided((6, V), (ld, 1), at)
        # what lies beside a row does not belong to it
        keep = z.clone()
        wide.fill_(math.inf)
        z.copy_(keep)
        tok = some(6, V)
        check(keep, tok, 10, run(z, tok, 10))


def test_logprobs_odd_rows_and_tokens():
    z, tok = logits((8, 3000), torch.float32, 4), some(8, 3000)
    want = run(z, tok, 4)
    z[1, 17], z[2, 2999], z[3, 5], z[5] = math.nan, math.inf, -math.nan, math.nan
    tok2 = tok.clone()
    tok2[6], tok2[7] = -1, 3000
    got = run(z, tok2, 4, status=dsa.DEV_BAD_INDEX)
    for r in (0, 4):
        assert all(torch.equal(a[r], b[r]) for a, b in zip(got, want))
    for r in (1, 2, 3, 5):
        assert math.isnan(got.logprob[r]) and math.isnan(got.entropy[r]) and bool(torch.isnan(got.top_logprobs[r]).all())
        assert -1 <= int(got.top_ids[r].min()) and int(got.top_ids[r].max()) < 3000 and 0 <= int(got.rank[r]) < 3000
    assert got.top_ids[2, 0] == 2999
    for r in (6, 7):
        assert got.rank[r] == -1 and got.logprob[r] == -math.inf
        assert torch.equal(got.top_ids[r], want.top_ids[r]) and got.entropy[r] == want.entropy[r]
    assert torch.equal(got.top_logprobs[6:], want.top_logprobs[6:])


def test_logprobs_a_row_alone_gives_what_it_gives_in_a_batch():
    z, tok = logits((300, 32003), torch.bfloat16, 5), some(300, 32003)
    whole = run(z, tok, 6)
    again = run(z, tok, 6)
    assert all(torch.equal(a, b) for a, b in zip(whole, again))
    one = run(z[7:8], tok[7:8], 6)
    assert torch.equal(one.rank, whole.rank[7:8]) and torch.equal(one.top_ids, whole.top_ids[7:8])
    check(z[7:8], tok[7:8], 6, one)


def test_logprobs_outputs_streams_and_graphs(both_ways):
    z, tok = logits((9, 50001), torch.float16, 6), some(9, 50001)
    torch.cuda.synchronize()
    want = run(z, tok, 5)
    check(z, tok, 5, want)
    guard = [torch.full((11, *t.shape[1:]), 7, dtype=t.dtype, device="cuda") for t in want]
    out = dsa.TokenLogprobs(*(t[1:10] for t in guard))
    got = run(z, tok, 5, out=out)
    assert all(torch.equal(a, b) and a.data_ptr() == o.data_ptr() for a, b, o in zip(got, want, out))
    assert all(bool((t[0] == 7).all()) and bool((t[10] == 7).all()) for t in guard)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    many = [dsa.token_logprobs(z, tok, top=5, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for m in many for a, b in zip(m, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dsa.token_logprobs(z, tok, top=5)
    z.copy_(logits((9, 50001), torch.float16, 7))
    tok.copy_(some(9, 50001, 8))
    graph.replay()
    torch.cuda.synchronize()
    check(z, tok, 5, got)
    empty = run(z[:0], tok[:0], 3)
    assert empty.logprob.shape == (0,) and empty.top_ids.shape == (0, 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
def test_logprobs_of_a_very_long_row(dtype):
    """Thousands of turns a thread: counts of the columns before the token are carried over in between."""
    V = 70_000_003
    z = logits((2, V), dtype, 7)
    at = [int(torch.sort(r.float()).indices[k]) for r, k in zip(z, (10, V // 2))]  # a token almost all come before, one in the middle
    check(z, i32(at), 20, run(z, i32(at), 20))


def test_logprobs_rows_past_32_bit_offsets():
    big = torch.empty((2, 2**31 + 8), dtype=torch.bfloat16, device="cuda")
    z = big[:, :5000]
    z.copy_(logits((2, 5000), torch.bfloat16, 9))
    tok = some(2, 5000)
    check(z, tok, 3, run(z, tok, 3))


def test_logprobs_of_a_verified_step():
    """Drafts verified against the target's rows, then the taken tokens' log probabilities from the logits."""
    R, n, V = 6, 4, 3001
    z = logits((R * n, V), torch.float32, 10, spread=1.0)
    p = torch.softmax(z, 1)
    cu = torch.arange(0, R * n + 1, n, dtype=I32, device="cuda")
    drafts = p.argmax(1).to(I32)
    u = torch.rand(R * n, generator=torch.Generator().manual_seed(3)).cuda()
    tokens, num, _ = dsa.verify_draft(p, drafts, cu, 0.002 * u, u[:R].contiguous(), max_out=n)
    got = run(z, tokens.flatten(), 2)
    i = torch.arange(n, device="cuda")[None] < num[:, None]
    flat = tokens.flatten()
    check(z, flat, 2, got)
    assert torch.equal(torch.isfinite(got.logprob).view(R, n), i)
    live = flat >= 0
    probs = p[live, flat[live].long()]
    assert float((got.logprob[live].exp() - probs).abs().max()) <= 2.0**-18
    assert int(num.min()) >= 1 and bool((got.top_ids[:, 0] == drafts).all())
    assert np.isfinite(got.entropy.cpu().numpy()).all()
