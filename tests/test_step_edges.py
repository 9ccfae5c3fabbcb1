"""CPU tests of the serving step's calls at the edges of their arguments: sizes
whose counters would wrap, overlaps, errors left behind, the binding's loading."""
import ctypes

import pytest
import torch

import dsa_sparse_mla_topk_gb300 as dsa
from dsa_sparse_mla_topk_gb300 import build as dsa_build
from test_step_args import A, _chunk, _layout, _norm, _verify, lib, no_device_only  # noqa: F401


@no_device_only
@pytest.mark.parametrize("cap,expect", [((1 << 30) + 1, 2), ((1 << 31) - 4, 2), ((1 << 31) - 1, 2)])
def test_layout_capacity_that_its_counters_cannot_hold(lib, cap, expect):  # noqa: F811
    """Four tokens past, or one past, a capacity near 2^31 is a negative number: the
    last 16-byte store would go past the arrays."""
    far = [ctypes.c_void_p(x << 36) for x in range(1, 4)]
    assert _layout(lib, cap=cap, req=far[0], pos=far[1], slot=far[2]) == expect


@no_device_only
@pytest.mark.parametrize("over", [dict(mo=(1 << 30) + 1), dict(mo=(1 << 31) - 1), dict(rows=(1 << 30) + 1),
                                  dict(rows=(1 << 31) - 1)])
def test_verify_sizes_that_its_counters_cannot_hold(lib, over):  # noqa: F811
    """Rows and outputs are counted 32 or a block of threads ahead: near 2^31 the count
    would turn negative and the loop would go on."""
    far = {k: ctypes.c_void_p(x << 44) for x, k in enumerate(("p", "q", "tok", "ua", "us", "cu", "ctx", "out", "num", "co"), 1)}
    assert _verify(lib, **far, **over) == 2


def at(base, off):
    return ctypes.c_void_p(base.value + off)


@no_device_only
def test_layout_table_over_its_inputs_and_outputs_over_each_other(lib):  # noqa: F811
    """The block table is written: it may not lie over the lengths or the free list."""
    table = 4 * 4 * 8  # its bytes
    for x in (0, 1, 2, 4, 5):  # lengths, held pages, free_pages, free_used
        assert _layout(lib, bt=A(x)) == 1, x
        assert _layout(lib, bt=at(A(x), -table + 4)) == 1, x
        assert _layout(lib, bt=at(A(x), -table)) == 4, x  # next to it (4: no device to launch on)
    outs = dict(cu=4 * 5, req=4 * 64, pos=4 * 64, slot=4 * 64, co=16, ho=16, uo=4)
    for a, n in outs.items():
        for b in outs:
            if a < b:
                assert _layout(lib, **{a: A(20), b: at(A(20), n - 4)}) == 1, (a, b)
                assert _layout(lib, **{a: A(20), b: at(A(20), n)}) == 4, (a, b)


@no_device_only
def test_outputs_over_any_input_or_each_other(lib):  # noqa: F811
    """Not over the queries alone: other CTAs still read positions, tables, weights,
    probabilities and cache rows while the first results are written."""
    # 4 = taken, but no device to launch on
    for x in (1, 4, 5, 6, 7):  # weights, positions, cos_sin, slots under the rows and the cache that are written
        for k in ("qo", "kv", "sc"):
            assert _norm(lib, **{k: A(x)}) == 1, (k, x)
    assert _norm(lib, kv=A(0)) == 1 and _norm(lib, kv=A(3)) == 1 and _norm(lib, sc=A(3)) == 1
    assert _norm(lib, kv=A(2)) == 1 and _norm(lib, sc=A(8)) == 1
    assert _norm(lib, qo=A(0)) == 4 and _norm(lib, ko=A(3)) == 4 and _norm(lib) == 4  # in place; apart
    for k in ("out", "lse"):
        for x in range(6):
            assert _chunk(lib, **{k: A(x)}) == 1, (k, x)
    assert _chunk(lib, lse=at(A(6), 2 * 64 * 512 - 4)) == 1 and _chunk(lib, lse=at(A(6), 2 * 64 * 512)) == 4
    part = dict(S=2, op=A(20), lp=A(21))
    assert _chunk(lib, **part) == 4 and _chunk(lib, **{**part, "lp": A(1)}) == 1
    assert _chunk(lib, **{**part, "op": A(3)}) == 1 and _chunk(lib, **{**part, "lp": A(20)}) == 1
    assert _chunk(lib, **part, out=A(0), lse=A(0)) == 4  # not written
    for k in ("out", "num", "co"):
        for x in (0, 1):
            assert _verify(lib, **{k: at(A(x), 4 * (7 * 100 + 96))}) == 1, (k, x)
            assert _verify(lib, **{k: at(A(x), 4 * (7 * 100 + 100))}) == 4, (k, x)
    assert _verify(lib, out=A(20), num=at(A(20), 28)) == 1 and _verify(lib, num=A(20), co=A(20)) == 1
    assert _verify(lib, co=A(6)) == 4  # the lengths in place


def _verify_req(lib, **over):  # noqa: F811
    a = dict(p=A(0), ld=100, rows=8, V=100, q=A(1), ldq=100, tok=A(2), ua=A(3), us=A(4), cu=A(5), req=A(10), R=2, mo=4,
             ctx=A(6), out=A(7), num=A(8), co=A(9), st=None, s=None)
    a.update(over)
    return lib.dsa_verify_draft_req(*a.values())


@no_device_only
def test_verification_with_the_requests_of_its_rows(lib):  # noqa: F811
    """The checks of dsa_verify_draft, and the rows' requests are an input like any other."""
    assert _verify_req(lib) == 4 and _verify_req(lib, req=None) == 4 and _verify_req(lib, R=0) == 0
    for k in ("out", "num", "co"):
        assert _verify_req(lib, **{k: A(10)}) == 1, k
        assert _verify_req(lib, **{k: at(A(10), 4 * 8 - 4)}) == 1, k
    assert _verify_req(lib, rows=-1) == 1 and _verify_req(lib, V=0) == 1 and _verify_req(lib, us=None) == 1


def test_split_rule_of_batches_whose_live_tokens_are_known(lib):  # noqa: F811
    """A full batch is not split for the sake of padding that it does not have, and a
    padded one is split like the small batch that it is."""
    pick = lambda n, live, ctx, H=64: dsa.pick_chunk_splits(  # noqa: E731
        n, H, 512 if H == 64 else 64, 64 if H == 64 else 16, ctx, 152, live=live)
    assert pick(128, None, 4096) == 2 and pick(128, 128, 4096) == 1 and pick(128, 72, 4096) == 2
    assert pick(48, None, 4096) == 5 and pick(48, 48, 4096) < 5 and pick(48, 27, 4096) == 5
    assert pick(152, 152, 16384) == 1
    for n, live, ctx in ((128, 20, 4096), (64, 64, 8192), (1000, 18, 5000), (7, 7, 100)):
        for H in (16, 64):
            assert pick(n, live, ctx, H) == pick(live, live, ctx, H)  # padding costs nothing
    # but to the Combine, which more than 8 splits need and which takes every token
    assert pick(3, 3, 5000) > 8 >= pick(1000, 3, 5000)
    assert pick(128, 0, 4096) == pick(128, 1, 4096) and pick(5, 99, 4096) == pick(5, 5, 4096)


# ---- the binding's C++ marshalling ---------------------------------------------------


def test_a_marshalling_module_that_cannot_be_loaded_is_left_alone(lib, tmp_path, monkeypatch):  # noqa: F811
    """Another Python's module, or a broken file, is no reason for every call to raise."""
    bad = tmp_path / "_marshal.so"
    bad.write_bytes(b"not a library")
    monkeypatch.setattr(dsa, "MARSHAL_PATH", str(bad))
    with pytest.warns(UserWarning, match="marshalled in Python"):
        assert dsa._load_marshal(lib) is None
    monkeypatch.setattr(dsa, "MARSHAL_PATH", str(tmp_path / "none.so"))
    assert dsa._load_marshal(lib) is None


def test_a_marshalling_module_of_another_library_version_is_left_alone(lib):  # noqa: F811
    class Other:
        def __getattr__(self, name):
            return (lambda: 1) if name == "dsa_version" else getattr(lib, name)
    if dsa._load_marshal(lib) is None:
        pytest.skip("not built here")
    with pytest.warns(UserWarning, match="another version"):
        assert dsa._load_marshal(Other()) is None


def test_a_marshalling_source_that_does_not_compile_stops_no_build(tmp_path, monkeypatch):
    """The build goes on without the module, and a module of other sources does not stay behind."""
    src, out = tmp_path / "marshal.cpp", tmp_path / "_marshal.so"
    src.write_text("this is not C++\n")
    out.write_bytes(b"older")
    monkeypatch.setattr(dsa_build, "MARSHAL_SRC", str(src))
    monkeypatch.setattr(dsa_build, "marshal_path", lambda: str(out))
    with pytest.warns(UserWarning, match="g\\+\\+ failed"):
        assert dsa_build.build_marshal(force=True) is None
    assert not list(tmp_path.glob("*.so*"))


def test_the_modules_name_holds_both_versions():
    import sysconfig
    assert dsa.MARSHAL_PATH == dsa_build.marshal_path()
    assert torch.__version__ in dsa.MARSHAL_PATH and sysconfig.get_config_var("SOABI") in dsa.MARSHAL_PATH
