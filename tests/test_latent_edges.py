"""CPU tests of the latent products, the expanded form's attention and the tokens' log
probabilities at the edges of their arguments."""
import ctypes

import pytest

import dsa_sparse_mla_topk_gb300 as dsa
from test_latent_args import A, _prompt, lib, no_device_only  # noqa: F401


@no_device_only
@pytest.mark.parametrize("heads", [1, 64, 65, 96, 128, 1000, 1024, 1025])
@pytest.mark.parametrize("d_v", [16, 48, 80, 128])
def test_combine_takes_the_heads_that_prompt_attention_takes(lib, heads, d_v):  # noqa: F811
    """A split prompt call ends in a Combine: every shape of the one is one of the other's."""
    far = [ctypes.c_void_p(x << 44) for x in range(1, 10)]
    ok = heads <= 1024
    # (no tokens: nothing is launched, the sizes are checked)
    assert lib.dsa_combine(far[0], far[1], 2, 0, heads, d_v, far[2], far[3], None) == (0 if ok else 1)
    prompt = lib.dsa_prompt_mla_fwd(far[0], heads * (d_v + 16), d_v + 16, far[1], heads * 2 * d_v, 2 * d_v, 100, far[2], 16,
                                    far[3], far[4], far[5], 1, 0, heads, d_v, 16, d_v, 0.1, 2, None, None, far[6], far[7],
                                    None, None)
    assert prompt == (0 if ok else 2)
    if heads == 128:
        assert dsa.pick_prompt_splits(1024, 1, heads, 16384, num_sms=152) > 1


@no_device_only
def test_combine_keeps_its_limit_for_wider_values(lib):  # noqa: F811
    assert lib.dsa_combine(A(0), A(1), 2, 0, 64, 512, A(2), A(3), None) == 0
    assert lib.dsa_combine(A(0), A(1), 2, 0, 65, 132, A(2), A(3), None) == 1
    assert lib.dsa_combine(A(0), A(1), 2, 0, 0, 128, A(2), A(3), None) == 1


@no_device_only
@pytest.mark.parametrize("scale,expect", [(2.0**127, 0), (2.0**127 * (1 + 2.0**-23), 1), (3e38, 1), (float("inf"), 1), (0.0, 0),
                                          (-0.0, 0), (-1e-45, 1)])
def test_prompt_scales_whose_logits_to_base_2_are_finite(lib, scale, expect):  # noqa: F811
    """Past 2^127 log2 e times the scale is infinite, and a sum of 0 times that no number."""
    if expect == 0:  # (nothing is launched without tokens, but the scale is looked at first)
        assert _prompt(lib, scale=scale, n=0) == 0
    else:
        assert _prompt(lib, scale=scale, n=0) == _prompt(lib, scale=scale) == expect
