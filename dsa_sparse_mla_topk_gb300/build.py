"""Build the CUDA library in-tree: csrc/*.cu (+ host-only csrc/*.cpp) -> libdsa.so (sm_103a only).

Each translation unit is compiled in parallel with nvcc, then linked into one
shared library with a plain C ABI (include/dsa.h).  The library links the
shared CUDA runtime so that it shares the process's runtime with PyTorch.

csrc/python/marshal.cpp, the Python binding's argument marshalling, is compiled
beside it with g++ against the installed PyTorch -> _marshal.<its version>.<Python's ABI>.so.  It
holds no kernels; without it (no Python or PyTorch headers, or they do not compile) the binding
marshals in Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdsa.so")
MARSHAL_SRC = os.path.join(CSRC, "python", "marshal.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdsa.so")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                   "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr", *extra]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "dsa.h"), __file__]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def marshal_path() -> str:
    import sysconfig

    import torch

    return os.path.join(PKG, f"_marshal.{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def build_marshal(force: bool = False) -> str | None:
    """The marshalling module for the PyTorch and the Python in use; None where it cannot be
    built (headers missing, a compiler error, which is warned of), and no older one stays."""
    import sysconfig

    import torch

    lib = marshal_path()
    deps = (MARSHAL_SRC, os.path.join(INCLUDE, "dsa.h"), __file__)
    if not force and os.path.exists(lib) and all(os.path.getmtime(d) <= os.path.getmtime(lib) for d in deps):
        return lib
    inc, cxx = sysconfig.get_paths()["include"], shutil.which("g++")
    root = os.path.dirname(torch.__file__)
    tinc, tlib = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    if not cxx or not all(os.path.exists(p) for p in (os.path.join(inc, "Python.h"), os.path.join(tinc, "ATen"),
                                                      os.path.join(cuda, "cuda_runtime_api.h"))):
        _remove(lib)
        return None
    tmp = lib + f".{os.getpid()}.tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", tinc, "-I",
           os.path.join(tinc, "torch", "csrc", "api", "include"), "-I", inc, "-I", cuda, MARSHAL_SRC, "-o", tmp,
           "-L", tlib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        _remove(tmp)
        _remove(lib)
        warnings.warn(f"g++ failed for {MARSHAL_SRC}, calls are marshalled in Python:\n{r.stderr}")
        return None
    os.replace(tmp, lib)
    return lib


def _remove(path: str) -> None:
    if os.path.exists(path):
        os.remove(path)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    with cf.ThreadPoolExecutor(max_workers=1) as ex:  # beside the CUDA sources
        marshal = ex.submit(build_marshal, force)
        lib = _build_library(force, verbose, ptxas_info)
        marshal.result()
    return lib


def _build_library(force: bool, verbose: bool, ptxas_info: bool) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        cmd = [cc, *_flags(extra), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose or ptxas_info:
        for _, err in results:
            if err:
                sys.stderr.write(err)
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
