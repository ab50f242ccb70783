"""Loads libseqattn.so (built in-tree by sequence_attn_fwd_gb300.build) via ctypes.

The library must exist: there is no fallback implementation. Import fails
with a message naming the build command when it is missing.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libseqattn.so")

# Every function the public header include/seqattn.h declares.
EXPORTS = ["attn_fwd", "attn_partial", "lse_merge", "attn_query_device_error",
           "attn_status_string", "attn_last_cuda_error", "attn_ring_fwd_static",
           "attn_debug_expire_wait", "attn_debug_exp2", "attn_partial_blocks", "attn_fwd_varlen", "attn_fwd_fp8", "attn_bwd",
           "attn_ring_fwd_host_workspace_bytes", "attn_ring_fwd_host"]

# Every function include/seqattn_paged.h declares.
PAGED_EXPORTS = ["attn_paged", "attn_paged_workspace_bytes", "rope_axes", "paged_append", "paged_reserve",
                 "paged_free", "paged_fork", "paged_copy", "paged_compact", "paged_compact_workspace_bytes",
                 "paged_append_guarded", "paged_reserve_guarded", "paged_append_e4m3", "paged_read", "draft_tree",
                 "attn_paged_tree", "attn_paged_e4m3", "draft_accept", "draft_accept_words", "paged_keep"]

STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED",
          3: "ATTN_ERR_CUDA", 4: "ATTN_ERR_TIMEOUT"}


class AttnBlock(ctypes.Structure):
    """attn_block of include/seqattn.h."""
    _fields_ = [("q_row", ctypes.c_longlong), ("kv_row", ctypes.c_longlong), ("o_row", ctypes.c_longlong),
                ("q_pos", ctypes.c_longlong), ("kv_pos", ctypes.c_longlong), ("Sq", ctypes.c_int),
                ("Skv", ctypes.c_int), ("part", ctypes.c_int)]


class PagedCacheView(ctypes.Structure):
    """paged_cache of include/seqattn_paged.h."""
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("page_stride", ctypes.c_longlong),
                ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_longlong), ("kv_lens", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p), ("B", ctypes.c_int), ("n_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int)]


class PagedScales(ctypes.Structure):
    """paged_scales of include/seqattn_paged.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_longlong)]


class RopeRows(ctypes.Structure):
    """rope_rows of include/seqattn_paged.h."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("in_b", ctypes.c_longlong),
                ("in_h", ctypes.c_longlong), ("in_s", ctypes.c_longlong), ("out_b", ctypes.c_longlong),
                ("out_h", ctypes.c_longlong), ("out_s", ctypes.c_longlong), ("heads", ctypes.c_int)]


class PagedPool(ctypes.Structure):
    """paged_pool of include/seqattn_paged.h."""
    _fields_ = [("base", ctypes.c_void_p), ("layer_stride", ctypes.c_longlong), ("page_stride", ctypes.c_longlong),
                ("page_bytes", ctypes.c_longlong), ("n_layers", ctypes.c_int)]


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        name = STATUS.get(status, str(status))
        detail = lib.attn_status_string(status).decode() if lib is not None else ""
        extra = f" (cudaError {lib.attn_last_cuda_error()})" if status == 3 and lib is not None else ""
        super().__init__(f"{what}: {name}: {detail}{extra}")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing; build it with `python sequence_attn_fwd_gb300/build.py`")
    L = ctypes.CDLL(path)
    P, I, LL, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    L.attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, P]
    L.attn_partial.argtypes = [P, P, P, LL, LL, LL, P, P, I, I, I, I, I, I, I, F, I, P]
    L.lse_merge.argtypes = [P, P, I, P, I, P, I, I, I, I, P]
    L.attn_query_device_error.argtypes = [P]
    L.attn_status_string.argtypes = [I]
    L.attn_status_string.restype = ctypes.c_char_p
    L.attn_last_cuda_error.argtypes = []
    L.attn_ring_fwd_static.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, F, P]
    L.attn_ring_fwd_static.restype = ctypes.c_int
    L.attn_ring_fwd_host_workspace_bytes.argtypes = [I, I, I, I, I, I]
    L.attn_ring_fwd_host_workspace_bytes.restype = ctypes.c_size_t
    L.attn_ring_fwd_host.argtypes = [P, P, P, P, P, P, ctypes.c_size_t, I, I, I, I, I, I, I, F, P]
    L.attn_ring_fwd_host.restype = ctypes.c_int
    L.attn_debug_expire_wait.argtypes = [ctypes.c_uint, P]
    L.attn_debug_expire_wait.restype = ctypes.c_int
    L.attn_debug_exp2.argtypes = [P, P, ctypes.c_longlong, ctypes.c_int, P]
    L.attn_debug_exp2.restype = ctypes.c_int
    L.attn_partial_blocks.argtypes = [P, P, P, P, P, P, I, I, I, I, LL, LL, LL, I, I, I, F, I, P]
    L.attn_partial_blocks.restype = ctypes.c_int
    L.attn_fwd_varlen.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, P]
    L.attn_fwd_varlen.restype = ctypes.c_int
    L.attn_fwd_fp8.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, F, F, F, P]
    L.attn_fwd_fp8.restype = ctypes.c_int
    L.attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P]
    L.attn_bwd.restype = ctypes.c_int
    Z = ctypes.c_size_t
    L.attn_paged.argtypes = [P, LL, LL, P, P, LL, LL, P, P, Z, I, I, I, F, P]
    L.attn_paged_workspace_bytes.argtypes = [I, I, I, I]
    L.rope_axes.argtypes = [P, P, P, LL, LL, I, P, P, I, I, I, I, I, I, P]
    L.paged_append.argtypes = [P, P, P, P, P, LL, I, P, P, I, I, P]
    L.paged_reserve.argtypes = [P, LL, P, P, P, P, I, I, I, I, P]
    L.paged_append_guarded.argtypes = [P, P, P, P, P, LL, I, P, P, I, I, P, P]
    L.paged_reserve_guarded.argtypes = [P, LL, P, P, P, P, P, I, I, I, I, P]
    L.paged_free.argtypes = [P, LL, P, P, P, I, I, I, I, P]
    L.paged_fork.argtypes = [P, I, P, LL, P, P, P, P, P, I, I, I, I, I, P]
    L.paged_copy.argtypes = [P, I, P, P, I, I, P]
    L.paged_compact.argtypes = [P, I, P, P, LL, P, P, P, P, Z, I, I, I, P]
    L.paged_compact_workspace_bytes.argtypes = [I]
    L.attn_paged_tree.argtypes = [P, LL, LL, P, P, LL, LL, P, P, Z, I, I, P, I, F, P]
    L.attn_paged_e4m3.argtypes = [P, LL, LL, P, P, P, LL, LL, P, P, Z, I, I, I, P, I, F, P]
    L.paged_append_e4m3.argtypes = [P, P, P, P, P, P, LL, I, P, P, I, I, P, P]
    L.paged_read.argtypes = [P, P, P, P, LL, LL, P, LL, LL, I, P]
    L.draft_tree.argtypes = [P, P, P, P, I, I, I, P]
    L.draft_accept.argtypes = [P, P, P, P, P, P, P, P, I, I, P]
    L.draft_accept_words.argtypes = [P, P, P, P, P, P, P, P, I, I, I, P]
    L.paged_keep.argtypes = [P, P, I, P, LL, P, P, P, P, P, P, P, I, I, I, I, I, P]
    for name in PAGED_EXPORTS:
        getattr(L, name).restype = Z if name.endswith("_bytes") else I
    for name in ("attn_fwd", "attn_partial", "lse_merge", "attn_query_device_error",
                 "attn_last_cuda_error"):
        getattr(L, name).restype = ctypes.c_int
    return L


lib = None
lib = load()
