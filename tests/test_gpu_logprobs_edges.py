"""GPU tests of token_logprobs: what a row's results depend on, and its sums in rows
of very many values."""
import math

import pytest
import torch

from test_gpu_logprobs import U, check, logits, run, some

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import dsa_sparse_mla_topk_gb300 as dsa
    from dsa_sparse_mla_topk_gb300 import build
    build.build()
    dsa.load_library()


@DTYPES
@pytest.mark.parametrize("V", [515, 32003])
def test_logprobs_depend_on_the_row_and_on_how_many_there_are(dtype, V):
    """The same row among 1 to 700: rank and ids bit for bit, the rest within the sums' bounds; among as many rows of
    other values bit for bit."""
    z, tok = logits((700, V), dtype, 1), some(700, V)
    z[:, V - 7:] = -math.inf
    alone = run(z[:1], tok[:1], 7)
    check(z[:1], tok[:1], 7, alone)
    for n in (2, 19, 20, 38, 77, 153, 305, 700):
        got = run(z[:n], tok[:n], 7)
        check(z[:1], tok[:1], 7, type(got)(*(t[:1] for t in got)), n)
        assert torch.equal(got.rank[:1], alone.rank) and torch.equal(got.top_ids[:1], alone.top_ids)
        other = z[:n].clone()
        other[1:] = logits((n - 1, V), dtype, n, spread=9.0)
        other[n - 1] = math.nan
        again = run(other, tok[:n], 7)
        assert all(torch.equal(a[0], b[0]) for a, b in zip(got, again)), n


@DTYPES
@pytest.mark.parametrize("R,V,parts", [(2, 70_000_003, 8192), (160, 2_000_003, 1024), (310, 1_000_003, 512)],
                         ids=["clusters", "512 threads", "256 threads"])
def test_logprobs_sums_of_very_long_rows(dtype, R, V, parts):
    """logprob and entropy within the bounds of test_gpu_logprobs' head, with the sums' additions as the call makes them:
    a row's values go to `parts` sums in turn (two a thread: eight CTAs of 512 threads a row for few
    rows, one of 512 up to 304 rows, one of 256 past that), so that one has V / parts terms."""
    z, tok = logits((R, V), dtype, R), some(R, V)
    got = run(z, tok, 0)
    adds = (V / parts + 64) * U
    for r in range(0, R, 16 if R > 2 else 1):
        x = z[r].double()
        at = int(x.argmax())
        d = x - x[at]
        e = d.exp()
        entropy_terms = (e * d.abs()).sum()
        entropy_off = (e * d.abs() * (4 * U * d.abs() + 2.0**-22 + adds + U)).sum()
        e[at] = 0
        rest = e.sum()
        S = 1 + rest
        E = (e * (3 * U * d.abs() + 2.0**-22 + adds)).sum() / S + 2.0**-22 * rest.log1p()
        dt = d[int(tok[r])]
        lp = dt - rest.log1p()
        assert abs(float(got.logprob[r]) - float(lp)) <= float(E + 2 * U * dt.abs() + U * lp.abs())
        ent = rest.log1p() + entropy_terms / S
        assert abs(float(got.entropy[r]) - float(ent)) <= float(E + entropy_off / S + ent * (E + 2.0**-22))
