"""Refusals of the serving step's operators: the C ABI's argument checks (no
device needed: fake addresses that no check reads) and the binding's."""
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
    return VP(0x1000000 * (i + 1))


MISALIGNED = VP(0x1000004)


def _layout(lib, **over):
    a = dict(ctx=A(0), new=A(1), held=A(2), R=4, bt=A(3), bs=8, free=A(4), nf=16, used=A(5), P=64, np=32, cap=64,
             cu=A(6), req=A(7), pos=A(8), slot=A(9), co=A(10), ho=A(11), uo=A(12), st=None, s=None)
    a.update(over)
    return lib.dsa_batch_layout(*a.values())


@no_device_only
@pytest.mark.parametrize("over,expect", [
    (dict(R=0), 1), (dict(R=-1), 1), (dict(R=8193), 2), (dict(bs=0), 1), (dict(nf=-1), 1), (dict(P=0), 1),
    (dict(np=0), 1), (dict(np=1 << 30), 2), (dict(cap=-1), 1),
    (dict(ctx=None), 1), (dict(new=None), 1), (dict(held=None), 1), (dict(bt=None), 1), (dict(free=None), 1),
    (dict(used=None), 1), (dict(cu=None), 1), (dict(req=None), 1), (dict(pos=None), 1), (dict(slot=None), 1),
    (dict(co=None), 1), (dict(ho=None), 1), (dict(uo=None), 1),
    # outputs over inputs: another CTA may still read them
    (dict(co=A(0)), 1), (dict(ho=A(2)), 1), (dict(uo=A(5)), 1), (dict(cu=A(1)), 1), (dict(slot=A(0)), 1),
])
def test_batch_layout_argument_checks(lib, over, expect):
    assert _layout(lib, **over) == expect


def _norm(lib, **over):
    a = dict(q=A(0), qt=64 * 576, qh=576, nq=64, qw=A(1), qn=576, qo=A(2), k=A(3), kt=576, kh=576, nk=1, kw=A(4), kn=512,
             ko=None, T=4, d=576, rope=64, dt=0, pos=A(5), cs=A(6), mp=100, eps=1e-6, il=1, slot=A(7), kv=A(8), sc=A(9),
             ns=64, st=None, s=None)
    a.update(over)
    return lib.dsa_qk_norm_rope(*a.values())


@no_device_only
@pytest.mark.parametrize("over,expect", [
    (dict(T=-1), 1), (dict(d=0), 1), (dict(d=580), 1), (dict(d=1032), 1), (dict(rope=8), 1), (dict(rope=-16), 1),
    (dict(rope=592), 1), (dict(dt=2), 1), (dict(il=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(nq=-1), 1), (dict(qn=4), 1), (dict(qn=584), 1), (dict(qw=None), 1), (dict(qw=MISALIGNED), 1),
    (dict(q=None), 1), (dict(q=MISALIGNED), 1), (dict(qt=4), 1), (dict(qh=4), 1), (dict(qt=-8), 1), (dict(qo=None), 1),
    (dict(qo=MISALIGNED), 1), (dict(qo=A(0), qt=64 * 576 + 8), 1), (dict(k=None), 1),
    (dict(pos=None), 1), (dict(cs=None), 1), (dict(cs=MISALIGNED), 1), (dict(mp=0), 1),
    (dict(slot=None), 1), (dict(kv=None), 1), (dict(sc=None), 1), (dict(kv=MISALIGNED), 1), (dict(ns=0), 1),
    (dict(nk=2, kh=576, kt=1152), 1), (dict(slot=None, kv=None, sc=None), 1),  # no cache and no k_out
    (dict(T=1 << 30), 2), (dict(T=0), 0), (dict(nq=0, nk=0, slot=None, kv=None, sc=None), 0),
])
def test_norm_rope_argument_checks(lib, over, expect):
    assert _norm(lib, **over) == expect


def _chunk(lib, **over):
    a = dict(q=A(0), kv=A(1), sc=A(2), np=4, bt=A(3), R=1, bs=4, req=A(4), pos=A(5), n=1, H=64, dl=512, dr=64, P=64,
             scale=0.04, S=1, out=A(6), lse=A(7), op=None, lp=None, st=None, s=None)
    a.update(over)
    return lib.dsa_chunk_mla_fwd(*a.values())


@no_device_only
@pytest.mark.parametrize("over,expect", [
    (dict(H=32), 2), (dict(dl=256), 2), (dict(dr=32), 2), (dict(P=0), 1), (dict(n=-1), 1), (dict(S=0), 1),
    (dict(S=65), 1), (dict(S=9), 1), (dict(S=4, op=A(8)), 1), (dict(S=4, out=None), 1), (dict(q=None), 1), (dict(kv=None), 1), (dict(sc=None), 1), (dict(bt=None), 1), (dict(req=None), 1),
    (dict(pos=None), 1), (dict(out=None), 1), (dict(q=MISALIGNED), 1), (dict(kv=MISALIGNED), 1),
    (dict(out=MISALIGNED), 1), (dict(scale=float("inf")), 1), (dict(S=4, lp=A(8)), 1),
    (dict(S=4, op=MISALIGNED, lp=A(8)), 1), (dict(np=0), 1), (dict(np=1 << 26), 2), (dict(R=0), 1), (dict(n=0), 0),
])
def test_chunk_argument_checks(lib, over, expect):
    assert _chunk(lib, **over) == expect


def _verify(lib, **over):
    a = dict(p=A(0), ld=100, rows=8, V=100, q=A(1), ldq=100, tok=A(2), ua=A(3), us=A(4), cu=A(5), R=2, mo=4, ctx=A(6),
             out=A(7), num=A(8), co=A(9), st=None, s=None)
    a.update(over)
    return lib.dsa_verify_draft(*a.values())


@no_device_only
@pytest.mark.parametrize("over,expect", [
    (dict(rows=-1), 1), (dict(V=0), 1), (dict(R=-1), 1), (dict(mo=0), 1), (dict(ld=99), 1), (dict(ldq=99), 1),
    (dict(ctx=None), 1), (dict(co=None), 1), (dict(us=None), 1), (dict(cu=None), 1), (dict(out=None), 1),
    (dict(num=None), 1), (dict(p=None), 1), (dict(tok=None), 1), (dict(ua=None), 1), (dict(R=(1 << 24) + 1), 2),
    (dict(V=(1 << 30) + 1, ld=1 << 31, ldq=1 << 31), 2),
    (dict(R=0), 0),
])
def test_verify_argument_checks(lib, over, expect):
    assert _verify(lib, **over) == expect


@no_device_only
def test_outputs_over_inputs_are_refused(lib):
    """Another CTA may still read what an output would replace."""
    def at(base, off):
        return VP(base.value + off)
    # new pages are read from free_pages and old ones from block_table while tokens are written
    assert _layout(lib, slot=A(4)) == 1
    assert _layout(lib, pos=at(A(3), 16)) == 1
    # rows: 4 tokens of 64 x 576, token stride twice that
    wide = dict(qt=2 * 64 * 576)
    last = 2 * (3 * 2 * 64 * 576 + 64 * 576)  # bytes from the first to behind the last value
    assert _norm(lib, qo=at(A(0), last - 16), **wide) == 1
    assert _norm(lib, qo=A(3)) == 1
    assert _norm(lib, ko=at(A(0), 32)) == 1
    assert _norm(lib, ko=at(A(2), 2 * 4 * 64 * 576 - 16)) == 1
    q_bytes = 2 * 64 * 576
    assert _chunk(lib, out=A(0)) == 1
    assert _chunk(lib, out=at(A(0), q_bytes - 16)) == 1
    assert _chunk(lib, S=2, op=at(A(0), -(2 * 4 * 64 * 512) + 16), lp=A(8)) == 1
    assert _chunk(lib, S=2, out=A(0)) == 1  # merged by the call
    for k in ("out", "num", "co"):
        for x in (2, 3, 4, 5):
            assert _verify(lib, **{k: A(x)}) == 1, (k, x)
    assert _verify(lib, out=A(6)) == 1
    assert _verify(lib, num=A(6)) == 1
    assert _verify(lib, co=at(A(6), 4)) == 1


def test_chunk_split_rule(lib):
    """The rule on 152 SMs: no split once the tokens fill the GPU or the context is
    a few tiles; clusters that run in one wave when half the rows are padding; many
    splits for one long context."""
    pick = lambda n, ctx, H=64: dsa.pick_chunk_splits(n, H, 512 if H == 64 else 64, 64 if H == 64 else 16, ctx, 152)  # noqa: E731
    assert pick(1024, 16384) == pick(256, 8192) == pick(152, 1024) == 1
    # a full batch and a half full one count the same: 128 tokens of 4,096 positions
    # take 66 and 63 us in one share, 82 and 43 in two; 48 tokens 44 and 41 us in two, 54 and 27 in five
    assert pick(128, 4096) == pick(152, 16384) == 2 and pick(48, 4096) == 5
    assert pick(1, 1) == pick(1, 64) == pick(1, 256) == 1
    assert pick(1, 65536) >= 32
    assert pick(32, 8192) == 4 and pick(32, 1024) == 4 and pick(24, 4096) == 5
    assert pick(2, 512, 16) == 2 and pick(128, 1024, 16) == 1 and pick(1, 4096, 16) == 8 and pick(107, 12733, 16) == 5
    for n in (1, 3, 15, 16, 23, 24, 36, 37, 76, 77, 200):
        for ctx in (1, 63, 64, 65, 1000, 5000, 100000):
            s = pick(n, ctx)
            assert 1 <= s <= min(64, -(-ctx // 64))
            if 2 <= s <= 8 and ctx <= 1000:
                assert n <= 2 * {2: 76, 3: 46, 4: 36, 5: 28, 6: 23, 7: 15, 8: 15}[s]
    assert dsa.pick_chunk_splits(4, 32, 512, 64, 2048, 152) == 1  # unsupported heads
    assert dsa.pick_chunk_splits(0, 64, 512, 64, 2048, 152) == 1


def test_binding_rejects_cpu_tensors_and_types(lib):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        dsa.batch_layout(i(2), i(2), i(2), i(2, 4), i(8), i(1), page_size=16, num_pages=8, capacity=4)
    with pytest.raises(TypeError):
        dsa.batch_layout(torch.zeros(2), i(2), i(2), i(2, 4), i(8), i(1), page_size=16, num_pages=8, capacity=4)
    b = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.qk_norm_rope(b, None, i(2), torch.zeros(4, 16), d_rope=16)
    with pytest.raises(TypeError):
        dsa.qk_norm_rope(b.float(), None, i(2), torch.zeros(4, 16), d_rope=16)
    with pytest.raises(ValueError):
        dsa.qk_norm_rope(None, None, None, None, d_rope=0)
    with pytest.raises(ValueError):
        dsa.chunk_mla(torch.zeros(1, 16, 80, dtype=torch.bfloat16), torch.zeros(16, 80, dtype=torch.uint8),
                      torch.zeros(16), i(1, 1), i(1), i(1), d_latent=64, d_rope=16, page_size=16, softmax_scale=0.1)
    with pytest.raises(ValueError):
        dsa.verify_draft(torch.zeros(2, 8), i(2), i(2), torch.zeros(2), torch.zeros(1), max_out=2)
    with pytest.raises(TypeError):
        dsa.verify_draft(torch.zeros(2, 8).double(), i(2), i(2), torch.zeros(2), torch.zeros(1), max_out=2)
