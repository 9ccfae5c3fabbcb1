"""Refusals of the latent products, the expanded form's attention and the tokens' log
probabilities: the C ABI's argument checks (no device needed: fake addresses
that no check reads) and the binding's."""
import ctypes

import pytest
import torch

import dsa_sparse_mla_topk_gb300 as dsa
from dsa_sparse_mla_topk_gb300 import build as dsa_build


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load_library()


no_device_only = pytest.mark.skipif(torch.cuda.is_available(),
                                    reason="fake device addresses are only used where no CUDA device is present")
VP = ctypes.c_void_p


def A(i):  # distinct 16-byte aligned addresses, far apart
    return VP(0x100000000 * (i + 1))


def M(i, by=4):  # the same, not aligned
    return VP(0x100000000 * (i + 1) + by)


def _absorb(lib, **over):
    a = dict(q=A(0), ts=64 * 192, hs=192, w=A(1), n=4, H=64, dn=128, dr=64, dv=128, dl=512, y=A(2), st=None, s=None)
    a.update(over)
    return lib.dsa_absorb_q(*a.values())


def _project(lib, **over):
    a = dict(o=A(0), ts=64 * 512, hs=512, w=A(1), n=4, H=64, dn=128, dv=128, dl=512, y=A(2), st=None, s=None)
    a.update(over)
    return lib.dsa_project_out(*a.values())


SIZES = [(dict(n=-1), 1), (dict(n=0), 0), (dict(H=0), 1), (dict(H=1025), 2), (dict(n=1 << 27), 2), (dict(dn=8), 2),
         (dict(dn=136), 2), (dict(dn=144), 2), (dict(dv=0), 2), (dict(dv=144), 2), (dict(dl=520), 2), (dict(dl=528), 2),
         (dict(w=None), 1), (dict(w=M(1)), 1), (dict(y=None), 1), (dict(y=M(2)), 1), (dict(ts=4), 1), (dict(hs=12), 1),
         (dict(ts=-8), 1), (dict(ts=1 << 36), 1), (dict(y=A(1)), 1)]


@no_device_only
@pytest.mark.parametrize("over,expect", SIZES + [(dict(q=None), 1), (dict(q=M(0)), 1), (dict(dr=8), 2), (dict(dr=80), 2),
                                                 (dict(dr=-16), 2), (dict(y=A(0)), 1)])
def test_absorb_argument_checks(lib, over, expect):
    assert _absorb(lib, **over) == expect


@no_device_only
@pytest.mark.parametrize("over,expect", SIZES + [(dict(o=None), 1), (dict(o=M(0)), 1), (dict(y=VP(0x100000000 + 1024)), 1)])
def test_project_argument_checks(lib, over, expect):
    assert _project(lib, **over) == expect


def _expand(lib, **over):
    a = dict(kv=A(0), sc=A(1), np=32, bt=A(2), R=4, bs=8, ctx=A(3), w=A(4), H=64, dl=512, dr=64, dkv=256, P=64, cap=256,
             out=A(5), rope=A(6), cu=A(7), ws=A(8), wb=1 << 20, st=None, s=None)
    a.update(over)
    return lib.dsa_expand_kv(*a.values())


@no_device_only
@pytest.mark.parametrize("over,expect", [
    (dict(R=0), 1), (dict(R=8193), 2), (dict(bs=0), 1), (dict(P=0), 1), (dict(np=0), 1), (dict(np=1 << 30), 2),
    (dict(cap=-1), 1), (dict(cap=(1 << 30) + 1, wb=1 << 50), 2), (dict(H=0), 1), (dict(H=2000), 2), (dict(dl=40), 2),
    (dict(dl=528), 2), (dict(dr=8), 2), (dict(dr=80), 2), (dict(dkv=16), 2), (dict(dkv=272), 2), (dict(dkv=40), 2),
    (dict(kv=None), 1), (dict(kv=M(0)), 1), (dict(sc=None), 1), (dict(bt=None), 1), (dict(ctx=None), 1), (dict(w=None), 1),
    (dict(w=M(4)), 1), (dict(out=None), 1), (dict(out=M(5)), 1), (dict(rope=None), 1), (dict(rope=M(6)), 1),
    (dict(cu=None), 1), (dict(ws=None), 1), (dict(ws=M(8)), 1), (dict(wb=256 * 512 * 2), 3),
    (dict(out=A(0)), 1), (dict(rope=A(5)), 1), (dict(cu=A(3)), 1), (dict(ws=A(4)), 1), (dict(ws=A(5)), 1), (dict(cu=A(8)), 1),
])
def test_expand_argument_checks(lib, over, expect):
    assert _expand(lib, **over) == expect


def test_expand_workspace_size(lib):
    size = dsa.expand_kv_workspace_size
    assert size(0, 512) == 0 and size(256, 512) >= 256 * (1024 + 4)
    assert size(1 << 30, 512) >= (1 << 30) * 1028  # past 32 bits
    assert all(size(n + 1, 64) >= size(n, 64) for n in range(1, 300))


def _prompt(lib, **over):
    a = dict(q=A(0), qt=64 * 192, qh=192, kv=A(1), kt=64 * 256, kh=256, N=100, rope=A(2), rs=64, cuq=A(3), cuk=A(4),
             pos=A(5), R=2, n=8, H=64, dn=128, dr=64, dv=128, scale=0.07, S=1, out=A(6), lse=A(7), op=None, lp=None, st=None,
             s=None)
    a.update(over)
    return lib.dsa_prompt_mla_fwd(*a.values())


@no_device_only
@pytest.mark.parametrize("over,expect", [
    (dict(n=-1), 1), (dict(n=0), 0), (dict(N=-1), 1), (dict(R=-1), 1), (dict(R=8193), 2), (dict(n=(1 << 30) + 1), 2),
    (dict(N=(1 << 26) + 1), 2), (dict(N=1 << 26, kt=(1 << 36) - 8), 1), (dict(S=0), 1), (dict(S=65), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(scale=-0.1), 1), (dict(H=0), 1), (dict(H=1025), 2), (dict(dn=8), 2), (dict(dn=144), 2), (dict(dr=72), 2),
    (dict(dv=8), 2), (dict(dv=256), 2), (dict(q=None), 1), (dict(q=M(0)), 1), (dict(qt=4), 1), (dict(qh=-8), 1),
    (dict(kv=None), 1), (dict(kv=M(1)), 1), (dict(kt=4), 1), (dict(kh=12), 1), (dict(rope=None), 1), (dict(rope=M(2)), 1),
    (dict(rs=4), 1), (dict(rs=-8), 1), (dict(cuq=None), 1), (dict(cuk=None), 1), (dict(pos=None), 1), (dict(out=None), 1),
    (dict(out=M(6)), 1), (dict(S=2), 1), (dict(S=2, op=A(8)), 1), (dict(S=2, op=M(8), lp=A(9)), 1),
    (dict(out=A(0)), 1), (dict(out=A(1)), 1), (dict(lse=A(5)), 1), (dict(lse=A(6)), 1), (dict(out=A(2)), 1),
    (dict(S=2, op=A(8), lp=A(8)), 1), (dict(S=2, op=A(1), lp=A(9)), 1),
])
def test_prompt_argument_checks(lib, over, expect):
    assert _prompt(lib, **over) == expect


def _logprobs(lib, **over):
    a = dict(z=A(0), ld=1000, n=4, V=1000, dt=2, tok=A(1), top=5, lp=A(2), ent=A(3), rank=A(4), ids=A(5), tlp=A(6), st=None,
             s=None)
    a.update(over)
    return lib.dsa_token_logprobs(*a.values())


@no_device_only
@pytest.mark.parametrize("over,expect", [
    (dict(n=-1), 1), (dict(n=0), 0), (dict(V=0), 1), (dict(ld=999), 1), (dict(dt=3), 1), (dict(dt=-1), 1), (dict(top=-1), 1),
    (dict(top=65), 2), (dict(n=(1 << 24) + 1), 2), (dict(V=(1 << 30) + 1, ld=1 << 31), 2), (dict(ld=1 << 62), 1),
    (dict(z=None), 1), (dict(z=M(0, 2)), 1), (dict(z=M(0, 1), dt=0), 1), (dict(tok=None), 1), (dict(lp=None), 1),
    (dict(ent=None), 1), (dict(rank=None), 1), (dict(ids=None), 1), (dict(tlp=None), 1),
    (dict(lp=A(0)), 1), (dict(ent=A(2)), 1), (dict(rank=A(1)), 1), (dict(ids=A(4)), 1), (dict(tlp=A(5)), 1),
])
def test_logprobs_argument_checks(lib, over, expect):
    assert _logprobs(lib, **over) == expect


def test_binding_rejects_what_is_not_documented(lib):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    w = bf(2, 64, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.absorb_q(bf(1, 2, 48), w, d_rope=16)
    with pytest.raises(TypeError, match="bfloat16"):
        dsa.absorb_q(torch.zeros(1, 2, 48), w, d_rope=16)
    with pytest.raises(TypeError, match="Tensor"):
        dsa.project_out(None, w, d_nope=32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.project_out(bf(1, 2, 64), w, d_nope=32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.expand_kv(torch.zeros(64, 80, dtype=torch.uint8), torch.zeros(64), i(1, 1), i(1), w, d_rope=16, page_size=64,
                      capacity=4)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.prompt_mla(bf(1, 2, 48), bf(1, 2, 64), bf(1, 16), i(2), i(2), i(1), d_nope=32, softmax_scale=1.0)
    with pytest.raises(TypeError, match="logits"):
        dsa.token_logprobs(torch.zeros(1, 4, dtype=torch.float64), i(1))
    with pytest.raises(ValueError, match="CUDA"):
        dsa.token_logprobs(torch.zeros(1, 4), i(1))


def test_prompt_split_rule(lib):
    """The rule on 152 SMs: shares while the tiles leave SMs idle and a share outweighs its part of the Combine."""
    pick = lambda n, R, H, ctx: dsa.pick_prompt_splits(n, R, H, ctx, num_sms=152)  # noqa: E731
    assert pick(1, 1, 64, 512) == 1 and pick(1, 1, 64, 1024) == 2 and pick(1, 1, 64, 16384) == 2
    assert pick(256, 1, 64, 16384) == 2 and pick(300, 1, 64, 16384) == 1 and pick(128, 2, 64, 8192) == 1
    assert pick(3, 3, 64, 8192) == 3 and pick(1024, 1, 64, 16384) == 1 and pick(16384, 8, 64, 3048) == 1
    assert pick(1, 1, 16, 16384) == 8 and pick(0, 1, 64, 100) == pick(1, 0, 64, 100) == 1
    for n in (1, 5, 300, 1 << 30):
        for R in (1, 7, 8192):
            for ctx in (1, 127, 129, 5000, 1 << 20, 2**31 - 1):
                assert 1 <= pick(n, R, 64, ctx) <= min(8, -(-ctx // 128))
