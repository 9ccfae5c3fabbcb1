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
