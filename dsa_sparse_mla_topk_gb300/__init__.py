"""GB300 (sm_103a) DSA sparse-MLA library: Python binding of the C ABI.

The three calls of the path -- ``topk_select``, ``sparse_mla_fwd`` and
``combine`` -- marshal torch tensors (device memory, the current CUDA stream)
into the C ABI declared in ``include/dsa.h`` and run entirely in the
library's CUDA kernels.  ``batch_layout``, ``qk_norm_rope``, ``chunk_mla`` and
``verify_draft`` are the rest of a serving step around them; ``absorb_q`` and
``project_out`` the products before and after attention in the cache's latent
space, ``expand_kv`` and ``prompt_mla`` the form with every head's own keys and
values, and ``token_logprobs`` the log probabilities of a step's tokens.  There
is no CPU or PyTorch fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import sysconfig
import threading
import warnings
from typing import NamedTuple

import torch

__all__ = ["DsaError", "load_library", "topk_select", "sparse_mla_fwd", "combine", "sparse_mla_topk",
           "topk_sparse_mla_fwd", "two_kernel_path_supported", "sparse_mla_topk_fused", "fused_path_supported",
           "kv_write",
           "PrefixCache", "BatchLayout", "batch_layout", "qk_norm_rope", "chunk_mla_fwd", "chunk_mla", "verify_draft",
           "absorb_q", "project_out", "ExpandedKV", "expand_kv", "expand_kv_workspace_size", "prompt_mla_fwd", "prompt_mla",
           "pick_prompt_splits",
           "TokenLogprobs", "token_logprobs",
           "kv_tile_count", "kv_tile_size", "pick_num_splits", "pick_chunk_splits", "status_string", "EXPORTED_SYMBOLS",
           "DEV_BAD_QPOS", "DEV_BAD_INDEX", "DEV_BAD_PAGE", "DEV_TIMEOUT", "DEV_NO_PAGES"]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa.so")

DEV_BAD_QPOS, DEV_BAD_INDEX, DEV_BAD_PAGE, DEV_TIMEOUT, DEV_NO_PAGES = 1, 2, 4, 8, 16

# Every symbol include/dsa.h declares.
EXPORTED_SYMBOLS = ("dsa_status_string", "dsa_version", "dsa_topk_select", "dsa_topk_workspace_size",
                    "dsa_sparse_mla_fwd", "dsa_sparse_mla_workspace_size", "dsa_sparse_mla_fwd_noalloc",
                    "dsa_sparse_mla_topk_fwd", "dsa_sparse_mla_topk_max_k", "dsa_topk_sparse_mla_fwd",
                    "dsa_combine", "dsa_kv_write", "dsa_batch_layout", "dsa_qk_norm_rope", "dsa_chunk_mla_fwd",
                    "dsa_verify_draft", "dsa_verify_draft_req", "dsa_absorb_q", "dsa_project_out", "dsa_expand_kv",
                    "dsa_expand_kv_workspace_size", "dsa_prompt_mla_fwd", "dsa_prompt_pick_num_splits", "dsa_token_logprobs", "dsa_prefix_cache_create", "dsa_prefix_cache_destroy",
                    "dsa_prefix_cache_acquire", "dsa_prefix_cache_release", "dsa_prefix_cache_stats",
                    "dsa_kv_tile_count", "dsa_kv_tile_size", "dsa_pick_num_splits",
                    "dsa_chunk_pick_num_splits", "dsa_chunk_pick_num_splits_live")

_lock = threading.Lock()
_lib = None
_fast = None  # the C++ marshalling module, bound to the loaded library


class DsaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} (status {status})")
        self.status = status


def load_library(path: str | None = None):
    """Load libdsa.so (built by ``__graft_entry__.build()`` or
    ``python -m dsa_sparse_mla_topk_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build the CUDA library first "
                               "(python -m dsa_sparse_mla_topk_gb300.build)")
        lib = ctypes.CDLL(p)
        i32, i64, vp, f32, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
        lib.dsa_status_string.argtypes = [i32]
        lib.dsa_status_string.restype = ctypes.c_char_p
        lib.dsa_version.argtypes = []
        lib.dsa_version.restype = i32
        lib.dsa_topk_select.argtypes = [vp, i64, vp, i32, i32, vp, vp, sz, vp, vp]
        lib.dsa_topk_select.restype = i32
        lib.dsa_topk_workspace_size.argtypes = [i32, i64, i32]
        lib.dsa_topk_workspace_size.restype = sz
        lib.dsa_sparse_mla_fwd.argtypes = [vp, vp, vp, i64, vp, i32, i32, vp, vp, i32, i32, i32, i32, i32, i32,
                                           f32, i32, vp, vp, vp, vp, vp, sz, vp, vp]
        lib.dsa_sparse_mla_fwd_noalloc.argtypes = [vp, vp, vp, i64, vp, i32, i32, vp, vp, i32, i32, i32, i32, i32,
                                                   i32, f32, i32, vp, vp, vp, vp, vp, vp]
        lib.dsa_sparse_mla_fwd_noalloc.restype = i32
        lib.dsa_sparse_mla_topk_fwd.argtypes = [vp, i64, vp, i32, vp, vp, vp, vp, i64, vp, i32, i32, vp, i32, i32, i32,
                                                i32, i32, f32, vp, vp, vp, sz, vp, vp]
        lib.dsa_sparse_mla_topk_fwd.restype = i32
        lib.dsa_topk_sparse_mla_fwd.argtypes = [vp, i64, vp, i32, vp, vp, vp, vp, i64, vp, i32, i32, vp, i32, i32,
                                                i32, i32, i32, f32, i32, vp, vp, vp, vp, vp, sz, vp, vp]
        lib.dsa_topk_sparse_mla_fwd.restype = i32
        lib.dsa_sparse_mla_topk_max_k.argtypes = []
        lib.dsa_sparse_mla_topk_max_k.restype = i32
        lib.dsa_sparse_mla_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.dsa_sparse_mla_workspace_size.restype = sz
        lib.dsa_sparse_mla_fwd.restype = i32
        lib.dsa_combine.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp]
        lib.dsa_combine.restype = i32
        lib.dsa_kv_write.argtypes = [vp, i32, i32, vp, vp, vp, i32, i32, i32, i64, vp, vp, vp, vp]
        lib.dsa_kv_write.restype = i32
        lib.dsa_batch_layout.argtypes = [vp, vp, vp, i32, vp, i32, vp, i32, vp, i32, i64, i32, vp, vp, vp, vp, vp, vp,
                                         vp, vp, vp]
        lib.dsa_batch_layout.restype = i32
        lib.dsa_qk_norm_rope.argtypes = [vp, i64, i64, i32, vp, i32, vp, vp, i64, i64, i32, vp, i32, vp, i32, i32, i32,
                                         i32, vp, vp, i32, f32, i32, vp, vp, vp, i64, vp, vp]
        lib.dsa_qk_norm_rope.restype = i32
        lib.dsa_chunk_mla_fwd.argtypes = [vp, vp, vp, i64, vp, i32, i32, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp,
                                          vp, vp, vp, vp, vp]
        lib.dsa_chunk_mla_fwd.restype = i32
        lib.dsa_verify_draft.argtypes = [vp, i64, i32, i32, vp, i64, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp]
        lib.dsa_verify_draft.restype = i32
        lib.dsa_verify_draft_req.argtypes = [vp, i64, i32, i32, vp, i64, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp,
                                             vp]
        lib.dsa_verify_draft_req.restype = i32
        lib.dsa_absorb_q.argtypes = [vp, i64, i64, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp]
        lib.dsa_absorb_q.restype = i32
        lib.dsa_project_out.argtypes = [vp, i64, i64, vp, i32, i32, i32, i32, i32, vp, vp, vp]
        lib.dsa_project_out.restype = i32
        lib.dsa_expand_kv.argtypes = [vp, vp, i64, vp, i32, i32, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp,
                                      vp, sz, vp, vp]
        lib.dsa_expand_kv.restype = i32
        lib.dsa_expand_kv_workspace_size.argtypes = [i32, i32]
        lib.dsa_expand_kv_workspace_size.restype = sz
        lib.dsa_prompt_mla_fwd.argtypes = [vp, i64, i64, vp, i64, i64, i32, vp, i64, vp, vp, vp, i32, i32, i32, i32, i32,
                                           i32, f32, i32, vp, vp, vp, vp, vp, vp]
        lib.dsa_prompt_mla_fwd.restype = i32
        lib.dsa_prompt_pick_num_splits.argtypes = [i32, i32, i32, i32, i32]
        lib.dsa_prompt_pick_num_splits.restype = i32
        lib.dsa_token_logprobs.argtypes = [vp, i64, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp]
        lib.dsa_token_logprobs.restype = i32
        lib.dsa_prefix_cache_create.argtypes = [i32, i32]
        lib.dsa_prefix_cache_create.restype = vp
        lib.dsa_prefix_cache_destroy.argtypes = [vp]
        lib.dsa_prefix_cache_destroy.restype = None
        lib.dsa_prefix_cache_acquire.argtypes = [vp, vp, i64, vp, i32, vp, vp]
        lib.dsa_prefix_cache_acquire.restype = i32
        lib.dsa_prefix_cache_release.argtypes = [vp, vp, i32]
        lib.dsa_prefix_cache_release.restype = i32
        lib.dsa_prefix_cache_stats.argtypes = [vp, vp, vp, vp]
        lib.dsa_prefix_cache_stats.restype = i32
        lib.dsa_kv_tile_count.argtypes = [i32, i32]
        lib.dsa_kv_tile_count.restype = i32
        lib.dsa_kv_tile_size.argtypes = [i32, i32, i32]
        lib.dsa_kv_tile_size.restype = i32
        lib.dsa_pick_num_splits.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.dsa_pick_num_splits.restype = i32
        lib.dsa_chunk_pick_num_splits.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.dsa_chunk_pick_num_splits.restype = i32
        lib.dsa_chunk_pick_num_splits_live.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        lib.dsa_chunk_pick_num_splits_live.restype = i32
        global _fast
        _fast = _load_marshal(lib)
        _lib = lib
        return lib


# csrc/python/marshal.cpp as built for this PyTorch and this Python
MARSHAL_PATH = os.path.join(_PKG, f"_marshal.{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def _load_marshal(lib):
    """The C++ marshalling bound to ``lib``'s entry points; None where there is none
    for this PyTorch, this Python and this library, and Python marshals."""
    if not os.path.exists(MARSHAL_PATH):
        return None
    from importlib.machinery import ExtensionFileLoader
    from importlib.util import module_from_spec, spec_from_loader

    loader = ExtensionFileLoader("_marshal", MARSHAL_PATH)
    try:
        m = module_from_spec(spec_from_loader("_marshal", loader))
        loader.exec_module(m)
    except (ImportError, OSError) as e:
        warnings.warn(f"{MARSHAL_PATH} cannot be loaded ({e}): calls are marshalled in Python")
        return None
    if getattr(m, "header_version", 0) != lib.dsa_version():
        warnings.warn(f"{MARSHAL_PATH} was built for another version of the library: calls are marshalled in Python")
        return None
    m.bind(*(ctypes.cast(f, ctypes.c_void_p).value
             for f in (lib.dsa_batch_layout, lib.dsa_qk_norm_rope, lib.dsa_chunk_mla_fwd, lib.dsa_combine,
                       lib.dsa_chunk_pick_num_splits, lib.dsa_verify_draft_req, lib.dsa_absorb_q, lib.dsa_project_out,
                       lib.dsa_expand_kv, lib.dsa_expand_kv_workspace_size, lib.dsa_prompt_mla_fwd,
                       lib.dsa_prompt_pick_num_splits, lib.dsa_token_logprobs)))
    return m


def status_string(status: int) -> str:
    return load_library().dsa_status_string(int(status)).decode()


def kv_tile_count(width: int, tile: int) -> int:
    return load_library().dsa_kv_tile_count(int(width), int(tile))


def kv_tile_size(heads: int, d_latent: int, d_rope: int) -> int:
    return load_library().dsa_kv_tile_size(heads, d_latent, d_rope)


def pick_num_splits(num_q: int, heads: int, d_latent: int, d_rope: int, k: int, num_sms: int = 0) -> int:
    return load_library().dsa_pick_num_splits(num_q, heads, d_latent, d_rope, k, num_sms)


def pick_chunk_splits(num_q: int, heads: int, d_latent: int, d_rope: int, max_ctx: int, num_sms: int = 0,
                      live: int | None = None) -> int:
    """KV splits chunk_mla takes for contexts of about max_ctx positions; ``live``:
    about how many of the tokens are no padding (None: unknown)."""
    lib, ctx = load_library(), max(1, min(max_ctx, 2**31 - 1))
    if live is None:
        return lib.dsa_chunk_pick_num_splits(num_q, heads, d_latent, d_rope, ctx, num_sms)
    return lib.dsa_chunk_pick_num_splits_live(num_q, max(0, min(live, num_q)), heads, d_latent, d_rope, ctx, num_sms)


def _p(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle without a Stream object (2.8 us less per call on a
# Grace host), where this torch has the call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _check(t: torch.Tensor, name: str, dtype, ndim: int | None = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _call(fn: str, *args):
    st = getattr(load_library(), fn)(*args)
    if st != 0:
        raise DsaError(fn, st)


def topk_select(scores: torch.Tensor, q_pos: torch.Tensor, k: int, idx: torch.Tensor | None = None,
                dev_status: torch.Tensor | None = None, stream=None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """int32 [num_q, k] causal top-k positions (ascending, -1 padded).
    ``workspace`` (uint8, at least ``topk_workspace_size`` bytes) is allocated
    when the sliced path for rows longer than 65,536 positions applies and
    none is given; an empty tensor selects the in-place path instead."""
    _check(scores, "scores", torch.float32, 2)
    _check(q_pos, "q_pos", torch.int32, 1)
    num_q, ld = scores.shape
    if idx is None:
        idx = torch.empty((num_q, k), dtype=torch.int32, device=scores.device)
    _check(idx, "idx", torch.int32, 2)
    ws_bytes = topk_workspace_size(num_q, ld, k)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=scores.device)
    _call("dsa_topk_select", _p(scores), ld, _p(q_pos), num_q, k, _p(idx), _p(workspace),
          0 if workspace is None else workspace.numel(), _p(dev_status), _stream(stream))
    return idx


def sparse_mla_workspace_size(num_q: int, heads: int, d_latent: int, d_rope: int, k: int) -> int:
    return load_library().dsa_sparse_mla_workspace_size(num_q, heads, d_latent, d_rope, k)


def sparse_mla_fwd(q, kv, kv_scale, block_table, q_req, idx, *, d_latent: int, d_rope: int, page_size: int,
                   softmax_scale: float, num_splits: int = 1, out=None, lse=None, o_part=None, lse_part=None,
                   workspace=None, dev_status=None, stream=None):
    """Partial step.  num_splits == 1: returns (out bf16, lse fp32).
    num_splits > 1: returns (o_part fp32 [S, ...], lse_part fp32 [S, ...])."""
    _check(q, "q", torch.bfloat16, 3)
    _check(kv, "kv", torch.uint8, 2)
    _check(kv_scale, "kv_scale", torch.float32, 1)
    _check(block_table, "block_table", torch.int32, 2)
    _check(q_req, "q_req", torch.int32, 1)
    _check(idx, "idx", torch.int32, 2)
    num_q, H, dqk = q.shape
    if dqk != d_latent + d_rope or kv.shape[1] != dqk or kv.shape[0] % page_size:
        raise ValueError("q / kv row sizes do not match d_latent + d_rope, or kv is not whole pages")
    dev = q.device
    if num_splits == 1:
        if out is None:
            out = torch.empty((num_q, H, d_latent), dtype=torch.bfloat16, device=dev)
        if lse is None:
            lse = torch.empty((num_q, H), dtype=torch.float32, device=dev)
    else:
        if o_part is None:
            o_part = torch.empty((num_splits, num_q, H, d_latent), dtype=torch.float32, device=dev)
        if lse_part is None:
            lse_part = torch.empty((num_splits, num_q, H), dtype=torch.float32, device=dev)
    ws_bytes = sparse_mla_workspace_size(num_q, H, d_latent, d_rope, idx.shape[1])
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _call("dsa_sparse_mla_fwd", _p(q), _p(kv), _p(kv_scale), kv.shape[0] // page_size, _p(block_table),
          block_table.shape[0], block_table.shape[1], _p(q_req), _p(idx), num_q, H, d_latent, d_rope, page_size,
          idx.shape[1], float(softmax_scale), num_splits, _p(out) if num_splits == 1 else None,
          _p(lse) if num_splits == 1 else None, _p(o_part) if num_splits > 1 else None,
          _p(lse_part) if num_splits > 1 else None, _p(workspace) if ws_bytes else None, ws_bytes,
          _p(dev_status), _stream(stream))
    return (out, lse) if num_splits == 1 else (o_part, lse_part)


def sparse_mla_fwd_noalloc(q, kv, kv_scale, block_table, q_req, idx, out, lse, *, d_latent: int, d_rope: int,
                           page_size: int, softmax_scale: float, dev_status=None, stream=None):
    """Partial step without a workspace (no device allocation inside the
    library call): scratch comes from a fixed array in the library; the
    caller provides out / lse.  See include/dsa.h for its limits."""
    for t, name, dt in ((q, "q", torch.bfloat16), (kv, "kv", torch.uint8), (kv_scale, "kv_scale", torch.float32),
                        (block_table, "block_table", torch.int32), (q_req, "q_req", torch.int32),
                        (idx, "idx", torch.int32), (out, "out", torch.bfloat16), (lse, "lse", torch.float32)):
        _check(t, name, dt)
    num_q, H, _ = q.shape
    _call("dsa_sparse_mla_fwd_noalloc", _p(q), _p(kv), _p(kv_scale), kv.shape[0] // page_size, _p(block_table),
          block_table.shape[0], block_table.shape[1], _p(q_req), _p(idx), num_q, H, d_latent, d_rope, page_size,
          idx.shape[1], float(softmax_scale), 1, _p(out), _p(lse), None, None, _p(dev_status), _stream(stream))
    return out, lse


def combine(o_part: torch.Tensor, lse_part: torch.Tensor, out=None, lse=None, stream=None):
    """Combine step: (out bf16 [num_q, H, dv], lse fp32 [num_q, H])."""
    _check(o_part, "o_part", torch.float32, 4)
    _check(lse_part, "lse_part", torch.float32, 3)
    S, num_q, H, dv = o_part.shape
    if out is None:
        out = torch.empty((num_q, H, dv), dtype=torch.bfloat16, device=o_part.device)
    if lse is None:
        lse = torch.empty((num_q, H), dtype=torch.float32, device=o_part.device)
    _call("dsa_combine", _p(o_part), _p(lse_part), S, num_q, H, dv, _p(out), _p(lse), _stream(stream))
    return out, lse


def topk_workspace_size(num_q: int, ld: int, k: int) -> int:
    """Workspace bytes dsa_topk_select can use (0 when no workspace applies)."""
    return int(load_library().dsa_topk_workspace_size(num_q, ld, k))


def kv_write(rows: torch.Tensor, req: torch.Tensor, pos: torch.Tensor, block_table: torch.Tensor,
             kv: torch.Tensor, kv_scale: torch.Tensor, *, page_size: int, dev_status=None, stream=None):
    """Quantise bf16 rows [n, d_qk] to FP8 E4M3 with one fp32 scale per token
    and store them, in place, into the paged cache ``kv`` (uint8 [slots, d_qk])
    and ``kv_scale`` (fp32 [slots]) at each row's (request, position) slot."""
    _check(rows, "rows", torch.bfloat16, 2)
    _check(req, "req", torch.int32, 1)
    _check(pos, "pos", torch.int32, 1)
    _check(block_table, "block_table", torch.int32, 2)
    _check(kv, "kv", torch.uint8, 2)
    _check(kv_scale, "kv_scale", torch.float32, 1)
    n, d = rows.shape
    if req.shape != (n,) or pos.shape != (n,) or kv.shape[1] != d or kv.shape[0] != kv_scale.shape[0]:
        raise ValueError("inconsistent shapes")
    if kv.shape[0] % page_size:
        raise ValueError("kv rows must be a whole number of pages")
    _call("dsa_kv_write", _p(rows), n, d, _p(req), _p(pos), _p(block_table), block_table.shape[0],
          block_table.shape[1], page_size, kv.shape[0] // page_size, _p(kv), _p(kv_scale), _p(dev_status),
          _stream(stream))
    return kv, kv_scale


class PrefixCache:
    """KV-only prefix-sharing page allocator (host side): requests sharing
    whole-page prefixes get the same page ids; see dsa_prefix_cache_* in
    include/dsa.h."""

    def __init__(self, page_size: int, num_pages: int):
        self._lib = load_library()
        self.page_size, self.num_pages = page_size, num_pages
        self._h = self._lib.dsa_prefix_cache_create(page_size, num_pages)
        if not self._h:
            raise DsaError("dsa_prefix_cache_create", 1)

    def acquire(self, tokens):
        """int32 page ids of a request's tokens, and how many of the leading
        ones were already cached (their KV rows need not be written)."""
        import numpy as np
        t = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        n_pages = (len(t) + self.page_size - 1) // self.page_size
        bt = np.empty(max(1, n_pages), dtype=np.int32)
        np_out, ns_out = ctypes.c_int32(0), ctypes.c_int32(0)
        st = self._lib.dsa_prefix_cache_acquire(self._h, t.ctypes.data_as(ctypes.c_void_p), len(t),
                                                bt.ctypes.data_as(ctypes.c_void_p), n_pages, ctypes.byref(np_out),
                                                ctypes.byref(ns_out))
        if st != 0:
            raise DsaError("dsa_prefix_cache_acquire", st)
        return bt[:np_out.value].copy(), ns_out.value

    def release(self, block_table):
        import numpy as np
        bt = np.ascontiguousarray(np.asarray(block_table, dtype=np.int32))
        st = self._lib.dsa_prefix_cache_release(self._h, bt.ctypes.data_as(ctypes.c_void_p), len(bt))
        if st != 0:
            raise DsaError("dsa_prefix_cache_release", st)

    def stats(self):
        """(pages referenced by live requests, pages cached, pages free)."""
        a, b, c = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int32(0)
        self._lib.dsa_prefix_cache_stats(self._h, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c))
        return a.value, b.value, c.value

    def close(self):
        if self._h:
            self._lib.dsa_prefix_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def sparse_mla_topk_fused(q, kv, kv_scale, block_table, q_req, q_pos, scores, k: int, *, d_latent: int,
                          d_rope: int, page_size: int, softmax_scale: float, idx=None, out=None, lse=None,
                          workspace=None, dev_status=None, stream=None):
    """Top-k and the Partial step (one KV split) in one kernel call
    (dsa_sparse_mla_topk_fwd); same results as topk_select followed by
    sparse_mla_fwd.  Returns (out, lse, idx)."""
    for t, name, dt in ((q, "q", torch.bfloat16), (kv, "kv", torch.uint8), (kv_scale, "kv_scale", torch.float32),
                        (block_table, "block_table", torch.int32), (q_req, "q_req", torch.int32),
                        (q_pos, "q_pos", torch.int32), (scores, "scores", torch.float32)):
        _check(t, name, dt)
    num_q, H, dqk = q.shape
    if dqk != d_latent + d_rope or kv.shape[1] != dqk or kv.shape[0] % page_size:
        raise ValueError("q / kv row sizes do not match d_latent + d_rope, or kv is not whole pages")
    dev = q.device
    if idx is None:
        idx = torch.empty((num_q, k), dtype=torch.int32, device=dev)
    if out is None:
        out = torch.empty((num_q, H, d_latent), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((num_q, H), dtype=torch.float32, device=dev)
    ws_bytes = sparse_mla_workspace_size(num_q, H, d_latent, d_rope, k)
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _call("dsa_sparse_mla_topk_fwd", _p(scores), scores.shape[1], _p(q_pos), k, _p(idx), _p(q), _p(kv),
          _p(kv_scale), kv.shape[0] // page_size, _p(block_table), block_table.shape[0], block_table.shape[1],
          _p(q_req), num_q, H, d_latent, d_rope, page_size, float(softmax_scale), _p(out), _p(lse),
          _p(workspace) if ws_bytes else None, ws_bytes, _p(dev_status), _stream(stream))
    return out, lse, idx


def two_kernel_path_supported(heads: int, d_latent: int, d_rope: int, ld: int) -> bool:
    """Whether topk_sparse_mla_fwd takes this shape: the tensor-core head
    shape and rows of at most 65,536 positions (any k, any KV split)."""
    return (heads, d_latent, d_rope) == (64, 512, 64) and ld <= 65536


def topk_sparse_mla_fwd(q, kv, kv_scale, block_table, q_req, q_pos, scores, k: int, *, d_latent: int, d_rope: int,
                        page_size: int, softmax_scale: float, num_splits: int = 1, idx=None, out=None, lse=None,
                        o_part=None, lse_part=None, workspace=None, dev_status=None, stream=None):
    """topk_select followed by sparse_mla_fwd as two kernels, the top-k also
    looking up each selected position's page and scale
    (dsa_topk_sparse_mla_fwd); bit for bit the results of the two calls.
    Returns (out, lse, idx), or (o_part, lse_part, idx) when num_splits > 1."""
    for t, name, dt in ((q, "q", torch.bfloat16), (kv, "kv", torch.uint8), (kv_scale, "kv_scale", torch.float32),
                        (block_table, "block_table", torch.int32), (q_req, "q_req", torch.int32),
                        (q_pos, "q_pos", torch.int32), (scores, "scores", torch.float32)):
        _check(t, name, dt)
    num_q, H, dqk = q.shape
    if dqk != d_latent + d_rope or kv.shape[1] != dqk or kv.shape[0] % page_size:
        raise ValueError("q / kv row sizes do not match d_latent + d_rope, or kv is not whole pages")
    dev = q.device
    if idx is None:
        idx = torch.empty((num_q, k), dtype=torch.int32, device=dev)
    if num_splits == 1:
        if out is None:
            out = torch.empty((num_q, H, d_latent), dtype=torch.bfloat16, device=dev)
        if lse is None:
            lse = torch.empty((num_q, H), dtype=torch.float32, device=dev)
    else:
        if o_part is None:
            o_part = torch.empty((num_splits, num_q, H, d_latent), dtype=torch.float32, device=dev)
        if lse_part is None:
            lse_part = torch.empty((num_splits, num_q, H), dtype=torch.float32, device=dev)
    ws_bytes = sparse_mla_workspace_size(num_q, H, d_latent, d_rope, k)
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _call("dsa_topk_sparse_mla_fwd", _p(scores), scores.shape[1], _p(q_pos), k, _p(idx), _p(q), _p(kv),
          _p(kv_scale), kv.shape[0] // page_size, _p(block_table), block_table.shape[0], block_table.shape[1],
          _p(q_req), num_q, H, d_latent, d_rope, page_size, float(softmax_scale), num_splits,
          _p(out) if num_splits == 1 else None, _p(lse) if num_splits == 1 else None,
          _p(o_part) if num_splits > 1 else None, _p(lse_part) if num_splits > 1 else None,
          _p(workspace) if ws_bytes else None, ws_bytes, _p(dev_status), _stream(stream))
    return (out, lse, idx) if num_splits == 1 else (o_part, lse_part, idx)


def fused_path_supported(num_q: int, heads: int, d_latent: int, d_rope: int, ld: int, k: int,
                         num_splits: int) -> bool:
    """Whether the single-kernel path (dsa_sparse_mla_topk_fwd: the row's top-k,
    the page lookup and the Partial in one CTA per query token) can run this
    shape: the tensor-core head shape, one KV split, rows of at most 65,536
    positions and k within the kernel's limit.

    sparse_mla_topk does not pick it by itself: measured on GB300, the separate
    calls are faster at every decode batch tried (8 to 128 requests of a 64K
    context, and the 8-token verify and prefill shapes): the single kernel's
    selection and tile loop run a little slower, and it cannot split the KV
    range, which the small batches need."""
    del num_q
    if (heads, d_latent, d_rope) != (64, 512, 64) or num_splits != 1 or ld > 65536:
        return False
    return k <= load_library().dsa_sparse_mla_topk_max_k()


def sparse_mla_topk(q, kv, kv_scale, block_table, q_req, q_pos, scores, k: int, *, d_latent: int, d_rope: int,
                    page_size: int, softmax_scale: float, num_splits: int | None = None, buffers: dict | None = None,
                    dev_status=None, stream=None, fused: bool | None = None):
    """One pass of the whole path: top-k -> Partial -> Combine (when split).
    ``buffers`` (optional) holds preallocated idx / out / lse / o_part /
    lse_part / workspace tensors.  ``fused``: True runs top-k and the Partial
    step in one kernel (dsa_sparse_mla_topk_fwd, where fused_path_supported);
    False or None, the faster path: where two_kernel_path_supported, the top-k
    with the page lookup and then the attention kernel
    (dsa_topk_sparse_mla_fwd), else topk_select and sparse_mla_fwd.  The
    results are the same every way.  Returns (out, lse, idx)."""
    b = buffers or {}
    num_q, H, _ = q.shape
    if num_splits is None:
        num_splits = pick_num_splits(num_q, H, d_latent, d_rope, k)
    if fused:
        if num_splits != 1:
            raise ValueError("the fused path has one KV split")
        return sparse_mla_topk_fused(q, kv, kv_scale, block_table, q_req, q_pos, scores, k, d_latent=d_latent,
                                     d_rope=d_rope, page_size=page_size, softmax_scale=softmax_scale,
                                     idx=b.get("idx"), out=b.get("out"), lse=b.get("lse"),
                                     workspace=b.get("workspace"), dev_status=dev_status, stream=stream)
    if two_kernel_path_supported(H, d_latent, d_rope, scores.shape[1]):
        r = topk_sparse_mla_fwd(q, kv, kv_scale, block_table, q_req, q_pos, scores, k, d_latent=d_latent,
                                d_rope=d_rope, page_size=page_size, softmax_scale=softmax_scale,
                                num_splits=num_splits, idx=b.get("idx"), out=b.get("out"), lse=b.get("lse"),
                                o_part=b.get("o_part"), lse_part=b.get("lse_part"), workspace=b.get("workspace"),
                                dev_status=dev_status, stream=stream)
        if num_splits == 1:
            return r
        out, lse = combine(r[0], r[1], out=b.get("out"), lse=b.get("lse"), stream=stream)
        return out, lse, r[2]
    idx = topk_select(scores, q_pos, k, idx=b.get("idx"), dev_status=dev_status, stream=stream,
                      workspace=b.get("topk_workspace"))
    if num_splits == 1:
        out, lse = sparse_mla_fwd(q, kv, kv_scale, block_table, q_req, idx, d_latent=d_latent, d_rope=d_rope,
                                  page_size=page_size, softmax_scale=softmax_scale, num_splits=1, out=b.get("out"),
                                  lse=b.get("lse"), workspace=b.get("workspace"), dev_status=dev_status,
                                  stream=stream)
        return out, lse, idx
    op, lp = sparse_mla_fwd(q, kv, kv_scale, block_table, q_req, idx, d_latent=d_latent, d_rope=d_rope,
                            page_size=page_size, softmax_scale=softmax_scale, num_splits=num_splits,
                            o_part=b.get("o_part"), lse_part=b.get("lse_part"), workspace=b.get("workspace"),
                            dev_status=dev_status, stream=stream)
    out, lse = combine(op, lp, out=b.get("out"), lse=b.get("lse"), stream=stream)
    return out, lse, idx


# ---- the rest of a serving step --------------------------------------------------
#
# These calls are a few microseconds of GPU work in a decode step, so the host's
# time matters.  An ordinary call (documented tensors, outputs allocated here, the
# current device and stream) goes through the C++ marshalling; it takes nothing
# else, and what it does not take is checked, explained or run by the code here.

_I32, _F32, _BF16, _U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8


def _need(t, name: str, dtype, ndim: int, dev: int):
    """A contiguous CUDA tensor of this type and rank on device ``dev``."""
    try:
        if t.dtype is dtype and t.get_device() == dev >= 0 and t.dim() == ndim and t.is_contiguous():
            return
    except AttributeError:
        pass
    _check(t, name, dtype, ndim)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


def _need_rows(t, name: str, dtype, ndim: int, dev: int):
    """As _need, but only the last dimension has to be contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor" + (f" on cuda:{dev}, got {t.device}" if dev >= 0 else ""))
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")


def _need_shape(t, name: str, shape: tuple):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _strides(t):
    """Token and head strides of rows [tokens, heads, d]; 0 where only one is there."""
    return t.stride(0) if t.shape[0] > 1 else 0, t.stride(1) if t.shape[1] > 1 else 0


def _ptr(t):
    return None if t is None else t.data_ptr()


def _done(fn: str, r):
    """What the C++ marshalling returned: outputs, or a status that is an error."""
    if type(r) is int:
        raise DsaError(fn, r)
    return r


def _run(dev: int, stream, fn: str, *args):
    """Calls ``fn`` with the tensors' device current, on its current stream when
    none is given."""
    lib = _lib or load_library()
    if dev == torch.cuda.current_device():
        st = getattr(lib, fn)(*args, _stream(stream))
    else:
        with torch.cuda.device(dev):
            st = getattr(lib, fn)(*args, _stream(stream))
    if st != 0:
        raise DsaError(fn, st)


def _empty(shape, dtype, like, stream):
    """An output on ``like``'s device, from the memory of the stream that writes it:
    what was there before on another stream may still be in use."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _status_ptr(dev_status, dev: int):
    if dev_status is None:
        return None
    _need(dev_status, "dev_status", _I32, dev_status.dim(), dev)
    if dev_status.numel() < 1:
        raise ValueError("dev_status needs one element")
    return dev_status.data_ptr()


def _device_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t.get_device()


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether the spans of memory from the first to the last element overlap."""
    def span(t):
        n = 1 + sum((s - 1) * st for s, st in zip(t.shape, t.stride()))
        return t.data_ptr(), t.data_ptr() + n * t.element_size()
    if a.numel() == 0 or b.numel() == 0:
        return False
    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


class BatchLayout(NamedTuple):
    """What batch_layout writes (int32 tensors): token ranges cu_q [num_req +
    1]; request, position and cache slot of every token, -1 padded [capacity];
    the requests' lengths and pages after the step [num_req]; the count of
    free-list pages taken [1]."""
    cu_q: torch.Tensor
    q_req: torch.Tensor
    q_pos: torch.Tensor
    slot: torch.Tensor
    ctx_len: torch.Tensor
    pages_held: torch.Tensor
    free_used: torch.Tensor


def batch_layout(ctx_len: torch.Tensor, new_len: torch.Tensor, pages_held: torch.Tensor, block_table: torch.Tensor,
                 free_pages: torch.Tensor, free_used: torch.Tensor, *, page_size: int, num_pages: int, capacity: int,
                 out: BatchLayout | None = None, dev_status=None, stream=None) -> BatchLayout:
    """A step's token ranges, slot map and grown block tables from the
    requests' lengths (dsa_batch_layout): ``block_table`` gets the new pages in
    place, everything else is returned.  ``out`` (a BatchLayout of
    preallocated tensors, not the inputs) is written when given; else the
    outputs share one allocation, but what the next step keeps (cu_q, lengths,
    pages, free_used) has another one where the token arrays are over 64 KB."""
    if out is None and stream is None and _fast is not None:
        r = _fast.batch_layout(ctx_len, new_len, pages_held, block_table, free_pages, free_used, page_size, num_pages,
                               capacity, dev_status)
        if r is not None:
            return BatchLayout._make(_done("dsa_batch_layout", r))
    dev = _device_of(ctx_len, "ctx_len")
    _need(ctx_len, "ctx_len", _I32, 1, dev)
    _need(new_len, "new_len", _I32, 1, dev)
    _need(pages_held, "pages_held", _I32, 1, dev)
    _need(block_table, "block_table", _I32, 2, dev)
    _need(free_pages, "free_pages", _I32, 1, dev)
    _need(free_used, "free_used", _I32, 1, dev)
    R = ctx_len.shape[0]
    if new_len.shape[0] != R or pages_held.shape[0] != R or block_table.shape[0] != R or free_used.shape[0] != 1:
        raise ValueError("inconsistent shapes")
    if capacity < 0:
        raise ValueError("capacity must not be negative")
    if out is None:
        # the token arrays first, a multiple of 16 bytes apart; the requests' state, which the
        # next step keeps, apart from token arrays of more than 64 KB
        cap, words = (capacity + 3) & -4, 3 * R + 2
        if 12 * cap > 64 * 1024:
            buf, state = _empty(3 * cap, _I32, ctx_len, stream), _empty(words, _I32, ctx_len, stream)
        else:
            buf = _empty(3 * cap + words, _I32, ctx_len, stream)
            state = buf[3 * cap:]
        q_req, q_pos, slot = buf[:cap], buf[cap:2 * cap], buf[2 * cap:3 * cap]
        if cap != capacity:
            q_req, q_pos, slot = q_req[:capacity], q_pos[:capacity], slot[:capacity]
        out = BatchLayout(cu_q=state[:R + 1], q_req=q_req, q_pos=q_pos, slot=slot, ctx_len=state[R + 1:2 * R + 1],
                          pages_held=state[2 * R + 1:3 * R + 1], free_used=state[3 * R + 1:])
        p, c = buf.data_ptr(), state.data_ptr()
        ptrs = (c, p, p + 4 * cap, p + 8 * cap, c + 4 * R + 4, c + 8 * R + 4, c + 12 * R + 4)
    else:
        for x, name, n in zip(out, BatchLayout._fields, (R + 1, capacity, capacity, capacity, R, R, 1)):
            _need(x, "out." + name, _I32, 1, dev)
            _need_shape(x, "out." + name, (n,))
        ptrs = [x.data_ptr() for x in out]
    _run(dev, stream, "dsa_batch_layout", ctx_len.data_ptr(), new_len.data_ptr(), pages_held.data_ptr(), R,
         block_table.data_ptr(), block_table.shape[1], free_pages.data_ptr(), free_pages.shape[0], free_used.data_ptr(),
         page_size, num_pages, capacity, *ptrs, _status_ptr(dev_status, dev))
    return out


_ROW_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, pos: torch.Tensor | None,
                 cos_sin: torch.Tensor | None, *, d_rope: int, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = True,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                 slot: torch.Tensor | None = None, kv: torch.Tensor | None = None,
                 kv_scale: torch.Tensor | None = None, dev_status=None, stream=None):
    """Norm of each head's leading ``len(weight)`` values and rotation of its
    last ``d_rope`` values for query and key rows [tokens, heads, d] (bf16 or
    fp16, any token and head strides that are multiples of 8), in one pass
    (dsa_qk_norm_rope).  With ``slot`` / ``kv`` / ``kv_scale`` the single key
    head goes into the FP8 cache.  Returns (q_out, k_out); a side that is
    None, or keys that only go into the cache, give None.  Tokens with pos =
    -1 are left as they were."""
    some = q if q is not None else k
    if q_out is None and k_out is None and stream is None and _fast is not None:
        r = _fast.qk_norm_rope(q, k, pos, cos_sin, d_rope, q_weight, k_weight, eps, interleaved, slot, kv, kv_scale,
                               dev_status)
        if r is not None:
            return _done("dsa_qk_norm_rope", r)
    if some is None:
        raise ValueError("q or k must be given")
    dev = _device_of(some, "q or k")
    dtype = some.dtype
    code = _ROW_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"rows must be bfloat16 or float16, got {dtype}")
    qh = kh = qn = kn = qst = qsh = kst = ksh = slots = 0
    qp = kp = qwp = kwp = qop = kop = None
    if some.dim() != 3:
        raise ValueError("rows must be [tokens, heads, d]")
    n, _, d = some.shape
    cache = slot is not None or kv is not None or kv_scale is not None
    given = q_out is not None or k_out is not None
    if q is not None:
        _need_rows(q, "q", dtype, 3, dev)
        qp, qh = q.data_ptr(), q.shape[1]
        qst, qsh = _strides(q)
        if q_out is None:
            q_out = _empty(q.shape, dtype, q, stream)
        else:
            _need(q_out, "q_out", dtype, 3, dev)
            _need_shape(q_out, "q_out", q.shape)
        qop = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        _need_rows(k, "k", dtype, 3, dev)
        if k.shape[0] != n or k.shape[2] != d:
            raise ValueError("q and k must have the same tokens and row sizes")
        kp, kh = k.data_ptr(), k.shape[1]
        kst, ksh = _strides(k)
        if k_out is not None:
            _need(k_out, "k_out", dtype, 3, dev)
            _need_shape(k_out, "k_out", k.shape)
        elif not cache:
            k_out = _empty(k.shape, dtype, k, stream)
        kop = None if k_out is None else k_out.data_ptr()
    elif k_out is not None or cache:
        raise ValueError("k_out or a cache write without k")
    if q_weight is not None:
        _need(q_weight, "q_weight", _F32, 1, dev)
        qwp, qn = q_weight.data_ptr(), q_weight.shape[0]
    if k_weight is not None:
        _need(k_weight, "k_weight", _F32, 1, dev)
        kwp, kn = k_weight.data_ptr(), k_weight.shape[0]
    max_pos = 0
    if cos_sin is not None:
        _need(cos_sin, "cos_sin", _F32, 2, dev)
        max_pos = cos_sin.shape[0]
    if pos is not None:
        _need(pos, "pos", _I32, 1, dev)
    if d_rope and (pos is None or cos_sin is None or cos_sin.shape[1] != d_rope):
        raise ValueError("a rotation needs pos and cos_sin [max_pos, d_rope]")
    if pos is not None and pos.shape[0] != n:
        raise ValueError("pos must have one entry per token")
    if cache:
        if slot is None or kv is None or kv_scale is None:
            raise ValueError("the cache write needs slot, kv and kv_scale")
        _need(slot, "slot", _I32, 1, dev)
        _need(kv, "kv", _U8, 2, dev)
        _need(kv_scale, "kv_scale", _F32, 1, dev)
        slots = kv.shape[0]
        if slot.shape[0] != n or kv.shape[1] != d or kv_scale.shape[0] != slots:
            raise ValueError("slot must be [tokens], kv [slots, d] and kv_scale [slots]")
    if given:
        for o, own, name in ((q_out, q, "q_out"), (k_out, k, "k_out")):
            for x in (q, k):
                if o is not None and x is not None and _overlap(o, x) and not (
                        x is own and o.data_ptr() == x.data_ptr() and x.is_contiguous()):
                    raise ValueError(f"{name} overlaps an input (in place needs its own, contiguous)")
    _run(dev, stream, "dsa_qk_norm_rope", qp, qst, qsh, qh, qwp, qn, qop, kp, kst, ksh, kh, kwp, kn, kop, n, d, d_rope,
         code, _ptr(pos), _ptr(cos_sin), max_pos, float(eps), 1 if interleaved else 0, _ptr(slot), _ptr(kv), _ptr(kv_scale),
         slots, _status_ptr(dev_status, dev))
    return q_out, k_out


def chunk_mla_fwd(q, kv, kv_scale, block_table, q_req, q_pos, *, d_latent: int, d_rope: int, page_size: int,
                  softmax_scale: float, num_splits: int = 1, merge: bool = False, out=None, lse=None, o_part=None,
                  lse_part=None, dev_status=None, stream=None):
    """Attention of each token to all positions 0..q_pos of its request
    (dsa_chunk_mla_fwd).  num_splits == 1, or ``merge`` with at most 8 splits:
    returns (out bf16, lse fp32).  Else returns (o_part fp32 [S, ...],
    lse_part fp32 [S, ...]) for combine."""
    dev = _device_of(q, "q")
    _need(q, "q", _BF16, 3, dev)
    _need(kv, "kv", _U8, 2, dev)
    _need(kv_scale, "kv_scale", _F32, 1, dev)
    _need(block_table, "block_table", _I32, 2, dev)
    _need(q_req, "q_req", _I32, 1, dev)
    _need(q_pos, "q_pos", _I32, 1, dev)
    num_q, H, dqk = q.shape
    slots = kv.shape[0]
    if dqk != d_latent + d_rope or kv.shape[1] != dqk or page_size <= 0 or slots % page_size:
        raise ValueError("q / kv row sizes do not match d_latent + d_rope, or kv is not whole pages")
    if q_req.shape[0] != num_q or q_pos.shape[0] != num_q or kv_scale.shape[0] != slots:
        raise ValueError("inconsistent shapes")
    op = lp = oo = ll = None
    whole = num_splits == 1 or merge
    if whole:
        if out is None:
            out = _empty((num_q, H, d_latent), _BF16, q, stream)
        else:
            _need(out, "out", _BF16, 3, dev)
            _need_shape(out, "out", (num_q, H, d_latent))
        if lse is None:
            lse = _empty((num_q, H), _F32, q, stream)
        else:
            _need(lse, "lse", _F32, 2, dev)
            _need_shape(lse, "lse", (num_q, H))
        oo, ll = out.data_ptr(), lse.data_ptr()
    else:
        if o_part is None:
            o_part = _empty((num_splits, num_q, H, d_latent), _F32, q, stream)
        else:
            _need(o_part, "o_part", _F32, 4, dev)
            _need_shape(o_part, "o_part", (num_splits, num_q, H, d_latent))
        if lse_part is None:
            lse_part = _empty((num_splits, num_q, H), _F32, q, stream)
        else:
            _need(lse_part, "lse_part", _F32, 3, dev)
            _need_shape(lse_part, "lse_part", (num_splits, num_q, H))
        op, lp = o_part.data_ptr(), lse_part.data_ptr()
    _run(dev, stream, "dsa_chunk_mla_fwd", q.data_ptr(), kv.data_ptr(), kv_scale.data_ptr(), slots // page_size,
         block_table.data_ptr(), block_table.shape[0], block_table.shape[1], q_req.data_ptr(), q_pos.data_ptr(), num_q,
         H, d_latent, d_rope, page_size, float(softmax_scale), num_splits, oo, ll, op, lp, _status_ptr(dev_status, dev))
    return (out, lse) if whole else (o_part, lse_part)


def chunk_mla(q, kv, kv_scale, block_table, q_req, q_pos, *, d_latent: int, d_rope: int, page_size: int,
              softmax_scale: float, max_ctx: int | None = None, live: int | None = None, num_splits: int | None = None,
              buffers: dict | None = None, dev_status=None, stream=None):
    """The whole pass over every visible position: chunk_mla_fwd, merging its
    splits or, with more than 8 or where ``buffers`` holds partials, followed by
    combine.  ``max_ctx`` (default: the block table's width) is about the
    longest context and ``live`` (default: unknown, the batch may be half padding)
    about how many of the tokens are live, from which the number of KV splits is
    picked when ``num_splits`` is None; the result is right for any value.  ``buffers``
    (optional) holds preallocated out / lse / o_part / lse_part tensors.
    Returns (out, lse), which share one allocation unless given (clone lse to
    keep it alone)."""
    b = buffers or {}
    if num_splits is None and max_ctx is None:
        max_ctx = block_table.shape[1] * page_size
    if num_splits is None and live is not None:
        num_splits = pick_chunk_splits(q.shape[0], q.shape[1], d_latent, d_rope, max_ctx, live=live)
    if not b and stream is None and _fast is not None and num_splits != 0:
        r = _fast.chunk_mla(q, kv, kv_scale, block_table, q_req, q_pos, d_latent, d_rope, page_size, softmax_scale,
                            max_ctx or 1, num_splits or 0, dev_status)
        if r is not None:
            return _done("dsa_chunk_mla_fwd", r)
    num_q, H, _ = q.shape
    if num_splits is None:
        num_splits = pick_chunk_splits(num_q, H, d_latent, d_rope, max_ctx)
    out, lse = b.get("out"), b.get("lse")
    merge = 1 < num_splits <= 8 and b.get("o_part") is None and b.get("lse_part") is None
    if num_splits == 1 or merge or num_q == 0:
        return chunk_mla_fwd(q, kv, kv_scale, block_table, q_req, q_pos, d_latent=d_latent, d_rope=d_rope,
                             page_size=page_size, softmax_scale=softmax_scale, num_splits=num_splits if merge else 1,
                             merge=merge, out=out, lse=lse, dev_status=dev_status, stream=stream)
    op, lp = chunk_mla_fwd(q, kv, kv_scale, block_table, q_req, q_pos, d_latent=d_latent, d_rope=d_rope,
                           page_size=page_size, softmax_scale=softmax_scale, num_splits=num_splits,
                           o_part=b.get("o_part"), lse_part=b.get("lse_part"), dev_status=dev_status, stream=stream)
    dev = q.get_device()
    if out is None:
        out = _empty((num_q, H, d_latent), _BF16, q, stream)
    else:
        _need(out, "out", _BF16, 3, dev)
        _need_shape(out, "out", (num_q, H, d_latent))
    if lse is None:
        lse = _empty((num_q, H), _F32, q, stream)
    else:
        _need(lse, "lse", _F32, 2, dev)
        _need_shape(lse, "lse", (num_q, H))
    _run(dev, stream, "dsa_combine", op.data_ptr(), lp.data_ptr(), num_splits, num_q, H, d_latent, out.data_ptr(),
         lse.data_ptr())
    return out, lse


def verify_draft(target_probs: torch.Tensor, draft_tokens: torch.Tensor, cu_rows: torch.Tensor,
                 u_accept: torch.Tensor, u_sample: torch.Tensor, *, draft_probs: torch.Tensor | None = None,
                 ctx_len: torch.Tensor | None = None, q_req: torch.Tensor | None = None, max_out: int, tokens: torch.Tensor | None = None,
                 num_out: torch.Tensor | None = None, ctx_out: torch.Tensor | None = None, dev_status=None, stream=None):
    """Verification of drafted tokens against the target's probabilities from
    given random numbers (dsa_verify_draft_req).  ``cu_rows`` and ``q_req`` are
    batch_layout's: a request that it refused gets no tokens (without q_req
    its rows would be verified like any others).  Returns (tokens int32
    [num_req, max_out], -1 padded; num_out int32 [num_req]; ctx_out = ctx_len +
    num_out, or None without ctx_len); they share one allocation of max_out + 2
    words a request unless given."""
    if tokens is None and num_out is None and ctx_out is None and stream is None and _fast is not None:
        r = _fast.verify_draft(target_probs, draft_tokens, cu_rows, u_accept, u_sample, draft_probs, ctx_len, q_req,
                               max_out, dev_status)
        if r is not None:
            return _done("dsa_verify_draft_req", r)
    dev = _device_of(target_probs, "target_probs")
    _need_rows(target_probs, "target_probs", _F32, 2, dev)
    rows, vocab = target_probs.shape
    ld = ldd = vocab
    if rows > 1:
        ld = target_probs.stride(0)
    if draft_probs is not None:
        _need_rows(draft_probs, "draft_probs", _F32, 2, dev)
        _need_shape(draft_probs, "draft_probs", target_probs.shape)
        if rows > 1:
            ldd = draft_probs.stride(0)
    if ld < vocab or ldd < vocab:
        raise ValueError("rows of probabilities must not overlap")
    _need(draft_tokens, "draft_tokens", _I32, 1, dev)
    _need(cu_rows, "cu_rows", _I32, 1, dev)
    _need(u_accept, "u_accept", _F32, 1, dev)
    _need(u_sample, "u_sample", _F32, 1, dev)
    R = u_sample.shape[0]
    if cu_rows.shape[0] != R + 1 or draft_tokens.shape[0] != rows or u_accept.shape[0] != rows:
        raise ValueError("inconsistent shapes")
    if max_out < 1:
        raise ValueError("max_out must be positive")
    if q_req is not None:
        _need(q_req, "q_req", _I32, 1, dev)
        if q_req.shape[0] < rows:
            raise ValueError("q_req must have an entry for every row")
    if tokens is None:
        tokens = _empty((R, max_out), _I32, target_probs, stream)
    else:
        _need(tokens, "tokens", _I32, 2, dev)
        _need_shape(tokens, "tokens", (R, max_out))
    if num_out is None:
        num_out = _empty(R, _I32, target_probs, stream)
    else:
        _need(num_out, "num_out", _I32, 1, dev)
        _need_shape(num_out, "num_out", (R,))
    if ctx_len is None:
        if ctx_out is not None:
            raise ValueError("ctx_out needs ctx_len")
    else:
        _need(ctx_len, "ctx_len", _I32, 1, dev)
        _need_shape(ctx_len, "ctx_len", (R,))
        if ctx_out is None:
            ctx_out = _empty(R, _I32, target_probs, stream)
        else:
            _need(ctx_out, "ctx_out", _I32, 1, dev)
            _need_shape(ctx_out, "ctx_out", (R,))
    _run(dev, stream, "dsa_verify_draft_req", target_probs.data_ptr(), ld, rows, vocab, _ptr(draft_probs), ldd,
         draft_tokens.data_ptr(), u_accept.data_ptr(), u_sample.data_ptr(), cu_rows.data_ptr(), _ptr(q_req), R,
         max_out, _ptr(ctx_len), tokens.data_ptr(), num_out.data_ptr(), _ptr(ctx_out), _status_ptr(dev_status, dev))
    return tokens, num_out, ctx_out


# ---- latent attention's other form, and the products around both -------------------


def _given(t, name: str, dtype, shape: tuple, like, stream):
    """The caller's contiguous output of this type and shape, or a fresh one."""
    if t is None:
        return _empty(shape, dtype, like, stream)
    _need(t, name, dtype, len(shape), like.get_device())
    _need_shape(t, name, shape)
    return t


def absorb_q(q: torch.Tensor, w_kv: torch.Tensor, *, d_rope: int, q_out: torch.Tensor | None = None,
             dev_status=None, stream=None) -> torch.Tensor:
    """Queries in the cache's latent space (dsa_absorb_q): q bf16 [tokens, heads,
    d_nope + d_rope] (any token and head strides that are multiples of 8) and the
    up-projection w_kv bf16 [heads, d_nope + d_v, d_latent] of every head's keys
    and values give bf16 [tokens, heads, d_latent + d_rope], the queries of
    chunk_mla and sparse_mla_topk; the rotated part stays as it is."""
    if q_out is None and stream is None and _fast is not None:
        r = _fast.absorb_q(q, w_kv, d_rope, dev_status)
        if r is not None:
            return _done("dsa_absorb_q", r)
    dev = _device_of(q, "q")
    _need_rows(q, "q", _BF16, 3, dev)
    _need(w_kv, "w_kv", _BF16, 3, dev)
    n, H, d = q.shape
    if w_kv.shape[0] != H:
        raise ValueError("q and w_kv must have the same heads")
    _, dw, dl = w_kv.shape
    q_out = _given(q_out, "q_out", _BF16, (n, H, dl + d_rope), q, stream)
    ts, hs = _strides(q)
    _run(dev, stream, "dsa_absorb_q", q.data_ptr(), ts, hs, w_kv.data_ptr(), n, H, d - d_rope, d_rope, dw - (d - d_rope),
         dl, q_out.data_ptr(), _status_ptr(dev_status, dev))
    return q_out


def project_out(o: torch.Tensor, w_kv: torch.Tensor, *, d_nope: int, out: torch.Tensor | None = None,
                dev_status=None, stream=None) -> torch.Tensor:
    """Attention's latent outputs o bf16 [tokens, heads, d_latent] (strides as for
    absorb_q) to every head's values, bf16 [tokens, heads, d_v] (dsa_project_out)."""
    if out is None and stream is None and _fast is not None:
        r = _fast.project_out(o, w_kv, d_nope, dev_status)
        if r is not None:
            return _done("dsa_project_out", r)
    dev = _device_of(o, "o")
    _need_rows(o, "o", _BF16, 3, dev)
    _need(w_kv, "w_kv", _BF16, 3, dev)
    n, H, dl = o.shape
    if w_kv.shape[0] != H or w_kv.shape[2] != dl:
        raise ValueError("o and w_kv must have the same heads and latent width")
    dv = w_kv.shape[1] - d_nope
    if dv <= 0:
        raise ValueError("d_nope leaves no values in w_kv")
    out = _given(out, "out", _BF16, (n, H, dv), o, stream)
    ts, hs = _strides(o)
    _run(dev, stream, "dsa_project_out", o.data_ptr(), ts, hs, w_kv.data_ptr(), n, H, d_nope, dv, dl, out.data_ptr(),
         _status_ptr(dev_status, dev))
    return out


class ExpandedKV(NamedTuple):
    """What expand_kv writes: every head's key and value of each row, kv bf16
    [capacity, heads, d_nope + d_v]; the rotated part of the keys, which all heads
    share, k_rope bf16 [capacity, d_rope]; the requests' row ranges cu_k int32
    [num_req + 1]."""
    kv: torch.Tensor
    k_rope: torch.Tensor
    cu_k: torch.Tensor


def expand_kv_workspace_size(capacity: int, d_latent: int) -> int:
    return int(load_library().dsa_expand_kv_workspace_size(capacity, d_latent))


def expand_kv(kv: torch.Tensor, kv_scale: torch.Tensor, block_table: torch.Tensor, ctx_len: torch.Tensor,
              w_kv: torch.Tensor, *, d_rope: int, page_size: int, capacity: int | None = None,
              out: ExpandedKV | None = None, workspace: torch.Tensor | None = None, dev_status=None,
              stream=None) -> ExpandedKV:
    """Keys and values of every head for the cached rows of each request, packed
    one request after another (dsa_expand_kv), from the paged FP8 cache and the
    up-projection w_kv bf16 [heads, d_nope + d_v, d_latent].  ``capacity`` is the
    number of rows to make room for, or ``out`` (an ExpandedKV) holds them; rows
    behind the last request are left as they were.  ``workspace`` (uint8,
    expand_kv_workspace_size bytes) is allocated when none is given."""
    if out is not None and capacity is None and workspace is None and stream is None and _fast is not None:
        r = _fast.expand_kv(kv, kv_scale, block_table, ctx_len, w_kv, d_rope, page_size, *out, dev_status)
        if r is not None:
            if r:
                raise DsaError("dsa_expand_kv", r)
            return out
    dev = _device_of(kv, "kv")
    _need(kv, "kv", _U8, 2, dev)
    _need(kv_scale, "kv_scale", _F32, 1, dev)
    _need(block_table, "block_table", _I32, 2, dev)
    _need(ctx_len, "ctx_len", _I32, 1, dev)
    _need(w_kv, "w_kv", _BF16, 3, dev)
    R, (H, dw, dl), slots = ctx_len.shape[0], w_kv.shape, kv.shape[0]
    if page_size <= 0 or slots % page_size or kv_scale.shape[0] != slots or kv.shape[1] != dl + d_rope:
        raise ValueError("kv must be whole pages of rows of w_kv's latent width + d_rope, kv_scale one value a row")
    if block_table.shape[0] != R:
        raise ValueError("block_table must have a row for every request")
    if (capacity is None) == (out is None):
        raise ValueError("give capacity or out")
    if out is None:
        if capacity < 0:
            raise ValueError("capacity must not be negative")
        out = ExpandedKV(_empty((capacity, H, dw), _BF16, kv, stream), _empty((capacity, d_rope), _BF16, kv, stream),
                         _empty(R + 1, _I32, kv, stream))
    else:
        capacity = out.kv.shape[0]
        for t, name, dt, shape in zip(out, ExpandedKV._fields, (_BF16, _BF16, _I32),
                                      ((capacity, H, dw), (capacity, d_rope), (R + 1,))):
            _given(t, "out." + name, dt, shape, kv, stream)
    ws = expand_kv_workspace_size(capacity, dl)
    if workspace is None:
        workspace = _empty(ws, _U8, kv, stream)
    else:
        _need(workspace, "workspace", _U8, 1, dev)
    _run(dev, stream, "dsa_expand_kv", kv.data_ptr(), kv_scale.data_ptr(), slots // page_size, block_table.data_ptr(), R,
         block_table.shape[1], ctx_len.data_ptr(), w_kv.data_ptr(), H, dl, d_rope, dw, page_size, capacity,
         out.kv.data_ptr(), out.k_rope.data_ptr() if d_rope else None, out.cu_k.data_ptr(), workspace.data_ptr(),
         workspace.numel(), _status_ptr(dev_status, dev))
    return out


def prompt_mla_fwd(q: torch.Tensor, kv: torch.Tensor, k_rope: torch.Tensor | None, cu_q: torch.Tensor,
                   cu_k: torch.Tensor, q_pos: torch.Tensor, *, d_nope: int, softmax_scale: float, num_splits: int = 1,
                   out=None, lse=None, o_part=None, lse_part=None, dev_status=None, stream=None):
    """Attention over every head's own keys and values (dsa_prompt_mla_fwd).
    num_splits == 1: returns (out bf16, lse fp32); else (o_part fp32 [S, ...],
    lse_part fp32 [S, ...]) for combine."""
    dev = _device_of(q, "q")
    _need_rows(q, "q", _BF16, 3, dev)
    _need_rows(kv, "kv", _BF16, 3, dev)
    for t, name in ((cu_q, "cu_q"), (cu_k, "cu_k"), (q_pos, "q_pos")):
        _need(t, name, _I32, 1, dev)
    (n, H, dqk), N = q.shape, kv.shape[0]
    dr, dv = dqk - d_nope, kv.shape[2] - d_nope
    if kv.shape[1] != H or dr < 0 or dv <= 0:
        raise ValueError("q and kv must have the same heads, with d_nope values of each head's key in front")
    if dr > 0:
        _need_rows(k_rope, "k_rope", _BF16, 2, dev)
        _need_shape(k_rope, "k_rope", (N, dr))
    if cu_q.shape[0] < 1 or cu_k.shape != cu_q.shape or q_pos.shape[0] != n:
        raise ValueError("cu_q and cu_k must have one entry more than there are requests, q_pos one for each token")
    if num_splits == 1:
        out = _given(out, "out", _BF16, (n, H, dv), q, stream)
        lse = _given(lse, "lse", _F32, (n, H), q, stream)
        ptrs = (out.data_ptr(), lse.data_ptr(), None, None)
    else:
        o_part = _given(o_part, "o_part", _F32, (num_splits, n, H, dv), q, stream)
        lse_part = _given(lse_part, "lse_part", _F32, (num_splits, n, H), q, stream)
        ptrs = (None, None, o_part.data_ptr(), lse_part.data_ptr())
    (qt, qh), (kt, kh) = _strides(q), _strides(kv)
    _run(dev, stream, "dsa_prompt_mla_fwd", q.data_ptr(), qt, qh, kv.data_ptr(), kt, kh, N,
         k_rope.data_ptr() if dr else None, k_rope.stride(0) if dr and N > 1 else 0, cu_q.data_ptr(), cu_k.data_ptr(),
         q_pos.data_ptr(), cu_q.shape[0] - 1, n, H, d_nope, dr, dv, float(softmax_scale), num_splits, *ptrs,
         _status_ptr(dev_status, dev))
    return (out, lse) if num_splits == 1 else (o_part, lse_part)


def pick_prompt_splits(num_tokens: int, num_req: int, heads: int, max_ctx: int, num_sms: int = 0) -> int:
    """Shares of the rows that prompt_mla takes for contexts of about max_ctx positions."""
    return load_library().dsa_prompt_pick_num_splits(num_tokens, num_req, heads, max(1, min(max_ctx, 2**31 - 1)), num_sms)


def prompt_mla(q: torch.Tensor, kv: torch.Tensor, k_rope: torch.Tensor | None, cu_q: torch.Tensor, cu_k: torch.Tensor,
               q_pos: torch.Tensor, *, d_nope: int, softmax_scale: float, max_ctx: int | None = None,
               num_splits: int | None = None, buffers: dict | None = None, dev_status=None, stream=None):
    """Attention of new tokens q bf16 [tokens, heads, d_nope + d_rope] over every
    head's own keys and values, kv bf16 [rows, heads, d_nope + d_v] and the shared
    rotated part k_rope bf16 [rows, d_rope] (expand_kv's, or a prompt's own
    projections; any strides that are multiples of 8): token t of request r, cu_q[r] <=
    t < cu_q[r + 1], attends to rows cu_k[r] .. cu_k[r] + q_pos[t].  ``cu_q`` and
    ``q_pos`` are batch_layout's; padding and q_pos = -1 give 0.  ``max_ctx``
    (default: the rows a request on average) is about the longest context, from which
    the number of shares of the rows is picked when ``num_splits`` is None; the
    result is right for any value.  Give it where ``kv`` has room for more rows than
    the requests have: rows that no request has count in the default.  ``buffers`` (optional) holds preallocated out / lse /
    o_part / lse_part tensors.  Returns (out bf16 [tokens, heads, d_v], lse fp32 [tokens,
    heads]), which share one allocation unless given (clone lse to keep it alone)."""
    b = buffers or {}
    if not b and stream is None and _fast is not None and num_splits != 0:
        r = _fast.prompt_mla(q, kv, k_rope, cu_q, cu_k, q_pos, d_nope, softmax_scale, max_ctx or 0, num_splits or 0,
                             dev_status)
        if r is not None:
            return _done("dsa_prompt_mla_fwd", r)
    _need_rows(q, "q", _BF16, 3, _device_of(q, "q"))
    S = num_splits
    if S is None:
        R = max(1, cu_q.shape[0] - 1)
        S = pick_prompt_splits(q.shape[0], R, q.shape[1], kv.shape[0] // R if max_ctx is None else max_ctx)
    r = prompt_mla_fwd(q, kv, k_rope, cu_q, cu_k, q_pos, d_nope=d_nope, softmax_scale=softmax_scale, num_splits=S,
                       out=b.get("out") if S == 1 else None, lse=b.get("lse") if S == 1 else None, o_part=b.get("o_part"),
                       lse_part=b.get("lse_part"), dev_status=dev_status, stream=stream)
    if S == 1:
        return r
    n, H, dv = r[0].shape[1:]
    out = _given(b.get("out"), "out", _BF16, (n, H, dv), q, stream)
    lse = _given(b.get("lse"), "lse", _F32, (n, H), q, stream)
    if n:
        _run(q.get_device(), stream, "dsa_combine", r[0].data_ptr(), r[1].data_ptr(), S, n, H, dv, out.data_ptr(),
             lse.data_ptr())
    return out, lse


class TokenLogprobs(NamedTuple):
    """What token_logprobs writes: logprob and entropy fp32 [rows], rank int32
    [rows], and the alternatives top_ids int32 and top_logprobs fp32 [rows, top]."""
    logprob: torch.Tensor
    entropy: torch.Tensor
    rank: torch.Tensor
    top_ids: torch.Tensor
    top_logprobs: torch.Tensor


_LOGIT_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, *, top: int = 0, out: TokenLogprobs | None = None,
                   dev_status=None, stream=None) -> TokenLogprobs:
    """Log probabilities of ``tokens`` int32 [rows] (-1: none) under the rows of
    ``logits`` [rows, vocab] (fp32, bf16 or fp16, any row stride; -inf: masked), with
    the rows' entropies, the tokens' ranks and the ``top`` most probable
    alternatives, ties to the lower id (dsa_token_logprobs).  ``out`` (a
    TokenLogprobs of preallocated tensors) is written when given; else the outputs
    share one allocation."""
    if out is None and stream is None and _fast is not None:
        r = _fast.token_logprobs(logits, tokens, top, dev_status)
        if r is not None:
            return TokenLogprobs._make(_done("dsa_token_logprobs", r))
    dev = _device_of(logits, "logits")
    code = _LOGIT_DTYPES.get(logits.dtype)
    if code is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
    _need_rows(logits, "logits", logits.dtype, 2, dev)
    _need(tokens, "tokens", _I32, 1, dev)
    rows, vocab = logits.shape
    if tokens.shape[0] != rows:
        raise ValueError("tokens must have one entry per row")
    if top < 0:
        raise ValueError("top must not be negative")
    ld = logits.stride(0) if rows > 1 else vocab
    if ld < vocab:
        raise ValueError("rows of logits must not overlap")
    shapes = ((rows,), (rows,), (rows,), (rows, top), (rows, top))
    out = TokenLogprobs(*(_given(t, "out." + name, dt, shape, logits, stream) for t, name, dt, shape in
                          zip(out or (None,) * 5, TokenLogprobs._fields, (_F32, _F32, _I32, _I32, _F32), shapes)))
    _run(dev, stream, "dsa_token_logprobs", logits.data_ptr(), ld, rows, vocab, code, tokens.data_ptr(), top,
         out.logprob.data_ptr(), out.entropy.data_ptr(), out.rank.data_ptr(), out.top_ids.data_ptr() if top else None,
         out.top_logprobs.data_ptr() if top else None, _status_ptr(dev_status, dev))
    return out
