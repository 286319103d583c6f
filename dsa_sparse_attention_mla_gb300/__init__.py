"""GB300-native DSA sparse MLA attention (sm_103a).

Thin Python binding over the C ABI of ``libdsa_gb300.so`` (declared in ``include/dsa.h``).
The functions below carry the C entry points' names and only marshal arguments: they take
torch CUDA tensors for device memory and the current torch stream, pass raw pointers and
sizes, and raise :class:`DsaError` on a non-zero status. Every step of the computation runs
in the library's CUDA kernels; there is no CPU or eager-PyTorch fallback, and a missing
library is an error.

What is computed (sglang PR #38547 "Enable zero-RoPE TileLang DSA on gfx950"): the packed
scaled-FP8 latent cache row (Contract table), quant_k_cache / dequant_k_cache (Scope list)
and the sparse attention over top-k gathered latent rows (Summary; Direct GLM geometry
coverage list).
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "DsaError", "CACHE_BF16", "CACHE_FP8_SCALED", "DEVERR_INDEX_OUT_OF_RANGE", "DEVERR_TIMEOUT",
    "DEVERR_SLOT_OUT_OF_RANGE", "library_path", "load_library", "dsa_status_string",
    "dsa_packed_row_bytes", "dsa_cache_row_bytes", "dsa_quant_k_cache", "dsa_gather_dequant", "dsa_gather_requant",
    "dsa_sparse_attn_workspace_size", "dsa_sparse_attn", "dsa_sparse_attn_static_ws", "dsa_topk_select", "DsaAttnArgs",
    "DEVERR_REQUEST_ORDER", "DsaPagedArgs", "DsaEvictArgs", "dsa_paged_attn_workspace_size", "dsa_paged_attn",
    "dsa_paged_attn_mass", "dsa_cache_evict_workspace_size", "dsa_cache_evict",
    "DEVERR_OUT_OF_PAGES", "DEVERR_TOKEN_CAPACITY", "DsaPlanArgs", "DsaQkArgs", "dsa_batch_plan", "dsa_qk_norm_rope",
    "dsa_block_pool", "dsa_block_scores", "dsa_block_select",
]

CACHE_BF16 = 0
CACHE_FP8_SCALED = 1
DEVERR_INDEX_OUT_OF_RANGE = 0x1
DEVERR_TIMEOUT = 0x2
DEVERR_SLOT_OUT_OF_RANGE = 0x4
DEVERR_REQUEST_ORDER = 0x8
DEVERR_OUT_OF_PAGES = 0x10
DEVERR_TOKEN_CAPACITY = 0x20

_HERE = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_LIB = None


def library_path() -> str:
    return os.path.join(_HERE, "libdsa_gb300.so")


class DsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dsa_status_string(status)} (status {status})")


class DsaAttnArgs(ctypes.Structure):
    """ctypes mirror of ``dsa_attn_args_t``."""

    _fields_ = [
        ("q", ctypes.c_void_p), ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
        ("T", ctypes.c_int64), ("H", ctypes.c_int),
        ("cache", ctypes.c_void_p), ("kind", ctypes.c_int), ("num_slots", ctypes.c_int64),
        ("d_nope", ctypes.c_int), ("d_rope", ctypes.c_int), ("d_v", ctypes.c_int),
        ("indices", ctypes.c_void_p), ("idx_stride_t", ctypes.c_int64), ("topk", ctypes.c_int),
        ("block_table", ctypes.c_void_p), ("bt_stride", ctypes.c_int64),
        ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
        ("req_of_token", ctypes.c_void_p), ("sm_scale", ctypes.c_float),
        ("out", ctypes.c_void_p), ("out_stride_t", ctypes.c_int64), ("out_stride_h", ctypes.c_int64),
        ("lse", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("error_word", ctypes.c_void_p),
    ]


class DsaPagedArgs(ctypes.Structure):
    """ctypes mirror of ``dsa_paged_args_t``."""

    _fields_ = [
        ("q", ctypes.c_void_p), ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
        ("T", ctypes.c_int64), ("H", ctypes.c_int),
        ("cache", ctypes.c_void_p), ("kind", ctypes.c_int), ("num_slots", ctypes.c_int64),
        ("d_nope", ctypes.c_int), ("d_rope", ctypes.c_int), ("d_v", ctypes.c_int),
        ("block_table", ctypes.c_void_p), ("bt_stride", ctypes.c_int64),
        ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_requests", ctypes.c_int64),
        ("req_of_token", ctypes.c_void_p), ("starts", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
        ("q_positions", ctypes.c_void_p), ("key_positions", ctypes.c_void_p),
        ("kp_stride", ctypes.c_int64), ("kp_width", ctypes.c_int64),
        ("sm_scale", ctypes.c_float), ("logit_cap", ctypes.c_float), ("slopes", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("out_stride_t", ctypes.c_int64), ("out_stride_h", ctypes.c_int64),
        ("lse", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("error_word", ctypes.c_void_p),
    ]


class DsaEvictArgs(ctypes.Structure):
    """ctypes mirror of ``dsa_evict_args_t``."""

    _fields_ = [
        ("cache", ctypes.c_void_p), ("kind", ctypes.c_int), ("num_slots", ctypes.c_int64),
        ("d_nope", ctypes.c_int), ("d_rope", ctypes.c_int),
        ("block_table", ctypes.c_void_p), ("bt_stride", ctypes.c_int64),
        ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_requests", ctypes.c_int64),
        ("lengths", ctypes.c_void_p), ("budgets", ctypes.c_void_p), ("budget", ctypes.c_int),
        ("sink", ctypes.c_int), ("recent", ctypes.c_int), ("width", ctypes.c_int64),
        ("mass", ctypes.c_void_p), ("mass_stride", ctypes.c_int64),
        ("positions", ctypes.c_void_p), ("positions_stride", ctypes.c_int64),
        ("mass_out", ctypes.c_void_p), ("mass_out_stride", ctypes.c_int64),
        ("positions_out", ctypes.c_void_p), ("positions_out_stride", ctypes.c_int64),
        ("lengths_out", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("error_word", ctypes.c_void_p),
    ]


class DsaPlanArgs(ctypes.Structure):
    """ctypes mirror of ``dsa_plan_args_t``."""

    _fields_ = [
        ("num_requests", ctypes.c_int64), ("lengths", ctypes.c_void_p), ("new_tokens", ctypes.c_void_p),
        ("held", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("bt_stride", ctypes.c_int64),
        ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
        ("free_pages", ctypes.c_void_p), ("free_capacity", ctypes.c_int64), ("num_free", ctypes.c_void_p),
        ("lengths_out", ctypes.c_void_p), ("held_out", ctypes.c_void_p), ("num_free_out", ctypes.c_void_p),
        ("T", ctypes.c_int64), ("cu_tokens", ctypes.c_void_p), ("req_of_token", ctypes.c_void_p),
        ("positions", ctypes.c_void_p), ("token_lengths", ctypes.c_void_p), ("out_loc", ctypes.c_void_p),
        ("error_word", ctypes.c_void_p),
        ("seen", ctypes.c_void_p), ("seen_out", ctypes.c_void_p), ("token_positions", ctypes.c_void_p),
        ("key_positions", ctypes.c_void_p), ("kp_stride", ctypes.c_int64), ("kp_width", ctypes.c_int64),
    ]


class DsaQkArgs(ctypes.Structure):
    """ctypes mirror of ``dsa_qk_args_t``."""

    _fields_ = [
        ("T", ctypes.c_int64), ("d_nope", ctypes.c_int), ("d_rope", ctypes.c_int),
        ("q", ctypes.c_void_p), ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64), ("H", ctypes.c_int),
        ("q_out", ctypes.c_void_p), ("q_out_stride_t", ctypes.c_int64), ("q_out_stride_h", ctypes.c_int64),
        ("q_norm", ctypes.c_int), ("q_weight", ctypes.c_void_p),
        ("k", ctypes.c_void_p), ("k_stride_t", ctypes.c_int64), ("k_norm", ctypes.c_int), ("k_weight", ctypes.c_void_p),
        ("cache", ctypes.c_void_p), ("kind", ctypes.c_int), ("num_slots", ctypes.c_int64), ("out_loc", ctypes.c_void_p),
        ("eps", ctypes.c_float), ("positions", ctypes.c_void_p), ("cos_sin", ctypes.c_void_p),
        ("cs_stride", ctypes.c_int64), ("num_positions", ctypes.c_int64), ("interleaved", ctypes.c_int),
        ("error_word", ctypes.c_void_p),
    ]


def load_library():
    """Load libdsa_gb300.so (built in-tree by ``__graft_entry__.build()``)."""
    global _LIB
    with _lock:
        if _LIB is not None:
            return _LIB
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build the CUDA library first (__graft_entry__.build())")
        lib = ctypes.CDLL(path)
        P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.dsa_status_string.argtypes = [i32]
        lib.dsa_status_string.restype = ctypes.c_char_p
        lib.dsa_last_cuda_error.argtypes = []
        lib.dsa_last_cuda_error.restype = i32
        lib.dsa_packed_row_bytes.argtypes = [i32, i32]
        lib.dsa_packed_row_bytes.restype = i64
        lib.dsa_cache_row_bytes.argtypes = [i32, i32, i32]
        lib.dsa_cache_row_bytes.restype = i64
        lib.dsa_quant_k_cache.argtypes = [P, i64, P, i64, i64, i32, i32, P, P, i64, P, P]
        lib.dsa_quant_k_cache.restype = i32
        lib.dsa_gather_dequant.argtypes = [P, i32, i64, i32, i32, P, i64, P, i64, i32, i32, P, P, P, P]
        lib.dsa_gather_dequant.restype = i32
        lib.dsa_gather_requant.argtypes = [P, i64, i32, i32, P, i64, P, i64, i32, i32, P, P, P, i64, P, P]
        lib.dsa_gather_requant.restype = i32
        lib.dsa_sparse_attn_workspace_size.argtypes = [ctypes.POINTER(DsaAttnArgs), ctypes.POINTER(ctypes.c_size_t)]
        lib.dsa_sparse_attn_workspace_size.restype = i32
        lib.dsa_sparse_attn.argtypes = [ctypes.POINTER(DsaAttnArgs), P]
        lib.dsa_sparse_attn.restype = i32
        lib.dsa_sparse_attn_static_ws.argtypes = [ctypes.POINTER(DsaAttnArgs), P]
        lib.dsa_sparse_attn_static_ws.restype = i32
        lib.dsa_topk_select.argtypes = [P, i64, i64, i64, P, i32, P, i64, P]
        lib.dsa_topk_select.restype = i32
        lib.dsa_blockscale_bytes.argtypes = [i64, i64]
        lib.dsa_blockscale_bytes.restype = i64
        lib.dsa_quant_fp8_blockscale.argtypes = [P, i64, i64, i64, i32, P, P, P]
        lib.dsa_quant_fp8_blockscale.restype = i32
        lib.dsa_proj_gemm.argtypes = [P, P, P, P, i64, i64, i64, P, i64, P, ctypes.c_size_t, P]
        lib.dsa_proj_gemm.restype = i32
        lib.dsa_paged_attn_workspace_size.argtypes = [ctypes.POINTER(DsaPagedArgs), ctypes.POINTER(ctypes.c_size_t)]
        lib.dsa_paged_attn_workspace_size.restype = i32
        lib.dsa_paged_attn.argtypes = [ctypes.POINTER(DsaPagedArgs), P]
        lib.dsa_paged_attn.restype = i32
        lib.dsa_paged_attn_mass.argtypes = [ctypes.POINTER(DsaPagedArgs), P, i64, P, i64, i64, P]
        lib.dsa_paged_attn_mass.restype = i32
        lib.dsa_cache_evict_workspace_size.argtypes = [i64, i64, ctypes.POINTER(ctypes.c_size_t)]
        lib.dsa_cache_evict_workspace_size.restype = i32
        lib.dsa_cache_evict.argtypes = [ctypes.POINTER(DsaEvictArgs), P]
        lib.dsa_cache_evict.restype = i32
        lib.dsa_batch_plan.argtypes = [ctypes.POINTER(DsaPlanArgs), P]
        lib.dsa_batch_plan.restype = i32
        lib.dsa_qk_norm_rope.argtypes = [ctypes.POINTER(DsaQkArgs), P]
        lib.dsa_qk_norm_rope.restype = i32
        lib.dsa_block_pool.argtypes = [P, i32, i64, P, i64, i32, i32, i64, P, P, i64, P, P, i64, P, P]
        lib.dsa_block_pool.restype = i32
        lib.dsa_block_scores.argtypes = [P, i64, i64, i64, i32, P, i64, P, i64, i32, i32, i64, P, P, ctypes.c_float, P, P,
                                         i64, i64, P, P]
        lib.dsa_block_scores.restype = i32
        lib.dsa_block_select.argtypes = [P, i64, i64, i64, P, i64, i32, i32, i64, P, P, i32, i32, i32, P, i64, P, i64, P,
                                         P, P]
        lib.dsa_block_select.restype = i32
        _LIB = lib
        return lib


def _check(status: int, where: str):
    if status != 0:
        raise DsaError(status, where)


def dsa_status_string(status: int) -> str:
    return load_library().dsa_status_string(int(status)).decode()


def dsa_packed_row_bytes(d_nope: int, d_rope: int) -> int:
    return int(load_library().dsa_packed_row_bytes(d_nope, d_rope))


def dsa_cache_row_bytes(kind: int, d_nope: int, d_rope: int) -> int:
    return int(load_library().dsa_cache_row_bytes(kind, d_nope, d_rope))


# ----------------------------------------------------------------------------- helpers --
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    import torch

    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_cuda(name, t, dtype=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")


# --------------------------------------------------------------------------- entry points --
def dsa_quant_k_cache(k_nope, k_rope=None, *, out_loc=None, cache=None, num_slots=None, error_word=None):
    """Pack bf16 latent rows into scaled-FP8 rows; returns the uint8 cache [num_slots, row_bytes]."""
    import torch

    _need_cuda("k_nope", k_nope, torch.bfloat16)
    _need_cuda("k_rope", k_rope, torch.bfloat16)
    _need_cuda("out_loc", out_loc, torch.int64)
    n, d_nope = k_nope.shape
    d_rope = 0 if k_rope is None or k_rope.numel() == 0 else k_rope.shape[1]
    if d_rope == 0:
        k_rope = None
    rb = dsa_packed_row_bytes(d_nope, d_rope)
    if cache is None:
        num_slots = n if num_slots is None else num_slots
        cache = torch.zeros((num_slots, rb), dtype=torch.uint8, device=k_nope.device)
    _need_cuda("cache", cache, torch.uint8)
    if num_slots is None:
        num_slots = cache.shape[0]
    if k_nope.stride(1) != 1 or (k_rope is not None and k_rope.stride(1) != 1):
        raise ValueError("rows must be contiguous along d")
    if out_loc is not None:
        out_loc = out_loc.contiguous()
    st = load_library().dsa_quant_k_cache(
        _ptr(k_nope), k_nope.stride(0), _ptr(k_rope), 0 if k_rope is None else k_rope.stride(0), n, d_nope, d_rope,
        _ptr(out_loc), _ptr(cache), num_slots, _ptr(error_word), _stream(k_nope.device))
    _check(st, "dsa_quant_k_cache")
    return cache


def dsa_gather_dequant(cache, kind: int, d_nope: int, d_rope: int, indices, *, block_table=None, page_size=0,
                       req_of_index=None, out=None, error_word=None):
    """bf16 rows [n, d_nope + d_rope] gathered (and dequantised) by index."""
    import torch

    _need_cuda("cache", cache)
    _need_cuda("indices", indices, torch.int32)
    _need_cuda("block_table", block_table, torch.int32)
    _need_cuda("req_of_index", req_of_index, torch.int32)
    indices = indices.contiguous().view(-1)
    n = indices.numel()
    if out is None:
        out = torch.empty((n, d_nope + d_rope), dtype=torch.bfloat16, device=indices.device)
    _need_cuda("out", out, torch.bfloat16)
    bt_stride = 0 if block_table is None else block_table.stride(0)
    max_pages = 0 if block_table is None else block_table.shape[1]
    st = load_library().dsa_gather_dequant(
        _ptr(cache), kind, cache.shape[0], d_nope, d_rope, _ptr(indices), n, _ptr(block_table), bt_stride, page_size,
        max_pages, _ptr(None if req_of_index is None else req_of_index.contiguous()), _ptr(out), _ptr(error_word),
        _stream(indices.device))
    _check(st, "dsa_gather_dequant")
    return out


def dsa_gather_requant(cache, d_nope: int, d_rope: int, indices, *, block_table=None, page_size=0,
                       req_of_index=None, out_loc=None, out=None, out_slots=None, error_word=None):
    """Packed rows gathered by index and packed again (uint8 [n, row_bytes], or written into
    rows out_loc of ``out``)."""
    import torch

    _need_cuda("cache", cache, torch.uint8)
    _need_cuda("indices", indices, torch.int32)
    _need_cuda("block_table", block_table, torch.int32)
    _need_cuda("req_of_index", req_of_index, torch.int32)
    _need_cuda("out_loc", out_loc, torch.int64)
    indices = indices.contiguous().view(-1)
    n = indices.numel()
    rb = dsa_packed_row_bytes(d_nope, d_rope)
    if out is None:
        out = torch.empty((n if out_loc is None else int(out_slots), rb), dtype=torch.uint8, device=indices.device)
    _need_cuda("out", out, torch.uint8)
    bt_stride = 0 if block_table is None else block_table.stride(0)
    max_pages = 0 if block_table is None else block_table.shape[1]
    st = load_library().dsa_gather_requant(
        _ptr(cache), cache.shape[0], d_nope, d_rope, _ptr(indices), n, _ptr(block_table), bt_stride, page_size,
        max_pages, _ptr(None if req_of_index is None else req_of_index.contiguous()),
        _ptr(None if out_loc is None else out_loc.contiguous()), _ptr(out), out.shape[0], _ptr(error_word),
        _stream(indices.device))
    _check(st, "dsa_gather_requant")
    return out


_WS = {}


def _workspace(device, nbytes: int):
    """The default workspace of the current stream on ``device``: one zero-filled buffer per
    (device, stream), so that calls on different streams, which may run at the same time on the
    GPU, never share one (calls on one stream run in order, so they can). The library leaves a
    workspace with no flag set after every call that completes without a timeout."""
    import torch

    index = device.index if device.index is not None else torch.cuda.current_device()
    key = (index, torch.cuda.current_stream(index).cuda_stream)
    with _lock:
        ws = _WS.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = torch.zeros(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
            _WS[key] = ws
    return ws


def _attn_args(q, cache, kind, indices, sm_scale, d_nope, d_rope, d_v, block_table, page_size, req_of_token, out,
               lse, workspace, error_word) -> DsaAttnArgs:
    a = DsaAttnArgs()
    T, H, D = q.shape
    a.q = q.data_ptr()
    a.q_stride_t, a.q_stride_h = q.stride(0), q.stride(1)
    a.T, a.H = T, H
    a.cache = cache.data_ptr()
    a.kind = kind
    a.num_slots = cache.shape[0]
    a.d_nope, a.d_rope, a.d_v = d_nope, d_rope, d_v
    a.indices = indices.data_ptr()
    a.idx_stride_t = indices.stride(0)
    a.topk = indices.shape[1]
    if block_table is not None:
        a.block_table = block_table.data_ptr()
        a.bt_stride = block_table.stride(0)
        a.page_size = page_size
        a.max_pages = block_table.shape[1]
    if req_of_token is not None:
        a.req_of_token = req_of_token.data_ptr()
    a.sm_scale = float(sm_scale)
    a.out = out.data_ptr()
    a.out_stride_t, a.out_stride_h = out.stride(0), out.stride(1)
    if lse is not None:
        a.lse = lse.data_ptr()
    if workspace is not None:
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    if error_word is not None:
        a.error_word = error_word.data_ptr()
    return a


def dsa_sparse_attn_workspace_size(d_v: int = 256) -> int:
    """Workspace bytes dsa_sparse_attn needs on the current device."""
    a = DsaAttnArgs()
    a.H, a.d_v = 64, d_v
    n = ctypes.c_size_t(0)
    _check(load_library().dsa_sparse_attn_workspace_size(ctypes.byref(a), ctypes.byref(n)),
           "dsa_sparse_attn_workspace_size")
    return int(n.value)


def _check_attn_inputs(q, cache, kind, indices, block_table, req_of_token, out, lse, error_word):
    import torch

    _need_cuda("q", q, torch.bfloat16)
    _need_cuda("cache", cache, torch.uint8 if kind == CACHE_FP8_SCALED else torch.bfloat16)
    _need_cuda("indices", indices, torch.int32)
    _need_cuda("block_table", block_table, torch.int32)
    _need_cuda("req_of_token", req_of_token, torch.int32)
    _need_cuda("out", out, torch.bfloat16)
    _need_cuda("lse", lse, torch.float32)
    _need_cuda("error_word", error_word, torch.int32)
    for name, t in (("cache", cache), ("indices", indices), ("block_table", block_table),
                    ("req_of_token", req_of_token), ("out", out), ("lse", lse), ("error_word", error_word)):
        if t is not None and t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}: every tensor must be on one device")
    if q.dim() != 3 or indices.dim() != 2:
        raise ValueError("q must be [T, H, D] and indices [T, topk]")
    if q.stride(2) != 1 or indices.stride(1) != 1:
        raise ValueError("q and indices must be contiguous along their last dimension")
    if req_of_token is not None and not req_of_token.is_contiguous():
        raise ValueError("req_of_token must be contiguous")
    if lse is not None and not lse.is_contiguous():
        raise ValueError("lse must be a contiguous [T, H] tensor")


def _prepare_attn(q, cache, kind, indices, d_v, block_table, req_of_token, out, lse, error_word):
    import torch

    if kind == CACHE_BF16 and cache.dim() == 3:
        cache = cache.view(cache.shape[0], -1)
    if out is None:
        out = torch.empty((q.shape[0], q.shape[1], d_v), dtype=torch.bfloat16, device=q.device)
    _check_attn_inputs(q, cache, kind, indices, block_table, req_of_token, out, lse, error_word)
    return cache, out


def dsa_sparse_attn(q, cache, kind: int, indices, sm_scale: float, *, d_nope: int = 256, d_rope: int = 0,
                    d_v: int = None, block_table=None, page_size: int = 0, req_of_token=None, out=None, lse=None,
                    workspace=None, error_word=None):
    """Sparse MLA attention: out[t, h] = softmax_j(sm_scale * q[t,h].k_j) @ k_j[:d_v] over valid indices.

    Without ``workspace`` the call takes the default workspace of the current stream (one per
    device and stream)."""
    import torch

    d_v = d_nope if d_v is None else d_v
    cache, out = _prepare_attn(q, cache, kind, indices, d_v, block_table, req_of_token, out, lse, error_word)
    if workspace is None:
        workspace = _workspace(q.device, dsa_sparse_attn_workspace_size(d_v))
    _need_cuda("workspace", workspace, torch.uint8)
    a = _attn_args(q, cache, kind, indices, sm_scale, d_nope, d_rope, d_v, block_table, page_size, req_of_token,
                   out, lse, workspace, error_word)
    _check(load_library().dsa_sparse_attn(ctypes.byref(a), _stream(q.device)), "dsa_sparse_attn")
    return out


def dsa_sparse_attn_static_ws(q, cache, kind: int, indices, sm_scale: float, *, d_nope: int = 256, d_rope: int = 0,
                              d_v: int = None, block_table=None, page_size: int = 0, req_of_token=None, out=None,
                              lse=None, error_word=None):
    """dsa_sparse_attn without a workspace: the library's fixed device scratch is used, so the
    call allocates no device memory (``out`` aside, when the caller passes none). For callers
    that cannot allocate device memory when they call; the first call on a device does one-time
    set-up. Calls whose kernels may overlap on the GPU share the one scratch array and race on it."""
    d_v = d_nope if d_v is None else d_v
    cache, out = _prepare_attn(q, cache, kind, indices, d_v, block_table, req_of_token, out, lse, error_word)
    a = _attn_args(q, cache, kind, indices, sm_scale, d_nope, d_rope, d_v, block_table, page_size, req_of_token,
                   out, lse, None, error_word)
    _check(load_library().dsa_sparse_attn_static_ws(ctypes.byref(a), _stream(q.device)), "dsa_sparse_attn_static_ws")
    return out


def dsa_topk_select(scores, K: int, *, lengths=None, out=None):
    """int32 [T, K]: per row, the positions of its K largest scores (ties: lower position first),
    in that order, then -1 (positions at or past lengths[t] are not considered)."""
    import torch

    _need_cuda("scores", scores, torch.float32)
    _need_cuda("lengths", lengths, torch.int32)
    if scores.dim() != 2 or scores.stride(1) != 1:
        raise ValueError("scores must be [T, S], contiguous along S")
    T, S = scores.shape
    if out is None:
        out = torch.empty((T, K), dtype=torch.int32, device=scores.device)
    _need_cuda("out", out, torch.int32)
    if out.dim() != 2 or out.shape[0] != T or out.shape[1] < K or out.stride(1) != 1:
        raise ValueError("out must be [T, >=K] int32, contiguous along its last dimension")
    if lengths is not None:
        lengths = lengths.contiguous()
        if lengths.numel() != T:
            raise ValueError("lengths must have one entry per row")
    st = load_library().dsa_topk_select(_ptr(scores), T, S, scores.stride(0), _ptr(lengths), int(K), _ptr(out),
                                        out.stride(0), _stream(scores.device))
    _check(st, "dsa_topk_select")
    return out


def dsa_blockscale_bytes(rows: int, cols: int) -> int:
    return int(load_library().dsa_blockscale_bytes(rows, cols))


def dsa_quant_fp8_blockscale(x, block_rows: int, *, codes=None, scales=None):
    """(codes uint8 [R, C], scales uint8 [dsa_blockscale_bytes(R, C)]) of bf16 x [R, C]: e4m3 codes
    with one power-of-two scale per block_rows x 128 block (128: weights, 1: activations), the
    scales in the projection GEMM's block-scale layout."""
    import torch

    _need_cuda("x", x, torch.bfloat16)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be [rows, cols], contiguous along cols")
    R, C = x.shape
    nb = dsa_blockscale_bytes(R, C)
    if nb < 0:
        raise ValueError("cols must be a positive multiple of 128")
    if codes is None:
        codes = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(nb, dtype=torch.uint8, device=x.device)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    if tuple(codes.shape) != (R, C) or not codes.is_contiguous() or scales.numel() < nb or not scales.is_contiguous():
        raise ValueError("codes must be contiguous [rows, cols] and scales hold dsa_blockscale_bytes(rows, cols)")
    st = load_library().dsa_quant_fp8_blockscale(_ptr(x), R, C, x.stride(0), int(block_rows), _ptr(codes), _ptr(scales),
                                                 _stream(x.device))
    _check(st, "dsa_quant_fp8_blockscale")
    return codes, scales


_GEMM_WS = {}


def _gemm_workspace(device, nbytes: int = 32 << 20):
    """The GEMM's scratch for the current stream on ``device`` (its own buffer: the attention's
    default workspace must keep its flags)."""
    import torch

    index = device.index if device.index is not None else torch.cuda.current_device()
    key = (index, torch.cuda.current_stream(index).cuda_stream)
    with _lock:
        ws = _GEMM_WS.get(key)
        if ws is None:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
            _GEMM_WS[key] = ws
    return ws


def dsa_proj_gemm(x_codes, x_scales, w_codes, w_scales, *, out=None, workspace=None):
    """bf16 [M, N] = X W^T over block-scaled FP8 operands (x from block_rows=1 [M, K], w from
    block_rows=128 [N, K])."""
    import torch

    for name, t in (("x_codes", x_codes), ("x_scales", x_scales), ("w_codes", w_codes), ("w_scales", w_scales)):
        _need_cuda(name, t, torch.uint8)
    M, K = x_codes.shape
    N, K2 = w_codes.shape
    if K2 != K:
        raise ValueError("x and w must share K")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x_codes.device)
    _need_cuda("out", out, torch.bfloat16)
    if out.dim() != 2 or tuple(out.shape) != (M, N) or out.stride(1) != 1:
        raise ValueError("out must be [M, N] bf16, contiguous along N")
    if workspace is None:
        workspace = _gemm_workspace(x_codes.device)
    _need_cuda("workspace", workspace, torch.uint8)
    st = load_library().dsa_proj_gemm(_ptr(x_codes), _ptr(x_scales), _ptr(w_codes), _ptr(w_scales), M, N, K, _ptr(out),
                                      out.stride(0), _ptr(workspace), workspace.numel(), _stream(x_codes.device))
    _check(st, "dsa_proj_gemm")
    return out


# ------------------------------------------------------- dense attention over the paged cache --
# A decode step calls these once per layer, so the checks touch each tensor a few times only.
def _cuda_index(t, name: str, dtype) -> int:
    """The tensor's CUDA device index; raises unless it is a CUDA tensor of the dtype."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    return t.get_device()


def _ptr_on(t, name: str, dtype, index: int):
    """data_ptr() of a tensor that must be on the device, or None."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == index:
        return t.data_ptr()
    i = _cuda_index(t, name, dtype)
    if i != index:
        raise ValueError(f"{name} is on cuda:{i}, not on cuda:{index}: every tensor must be on one device")
    return t.data_ptr()


def _vector(t, name: str, n: int, dtype, index: int):
    """data_ptr() of a contiguous tensor of n entries, or None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == (n,) and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    p = _ptr_on(t, name, dtype, index)
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} entries")
    return p


def _rows(t, name: str, dtype, index: int, rows=None, cols: int = 0):
    """(data_ptr(), row stride, rows, columns) of a matrix contiguous along its columns."""
    p = _ptr_on(t, name, dtype, index)
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or shape[1] < cols:
        raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, {'columns' if cols == 0 else f'>={cols}'}]")
    st = t.stride()
    if st[1] != 1 and shape[1] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    # a single row has no second one to step to: torch may report any stride
    return p, (st[0] if shape[0] > 1 else shape[1]), shape[0], shape[1]


def _cache_rows(cache, kind: int, row: int):
    """(device index, data_ptr(), slots) of a cache of contiguous rows."""
    import torch

    if kind == CACHE_FP8_SCALED:
        index = _cuda_index(cache, "cache", torch.uint8)
    elif kind == CACHE_BF16:
        index = _cuda_index(cache, "cache", torch.bfloat16)
    else:
        raise ValueError("kind must be CACHE_BF16 or CACHE_FP8_SCALED")
    shape = cache.shape
    if len(shape) == 3 and shape[1] == 1:
        shape = (shape[0], shape[2])
    if len(shape) != 2 or shape[1] != row or not cache.is_contiguous():
        raise ValueError(f"cache must be contiguous [num_slots, {row}]")
    return index, cache.data_ptr(), shape[0]


def _c_int(name: str, v) -> int:
    """An argument of a C int: a wider one would wrap silently on its way (2**32 to 0)."""
    if not -(1 << 31) <= v < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits, got {v}")
    return v


class _on_device:
    """Makes the device current, unless it is already."""

    def __init__(self, index: int):
        import torch

        self.guard = None if torch.cuda.current_device() == index else torch.cuda.device(index)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


_PAGED_WS = {}


def _workspace_for(workspace, nbytes: int, index: int):
    """(tensor, data_ptr(), bytes): the caller's workspace, or memory of the current stream for this
    call. The caching allocator orders its reuse with the stream, and inside a graph capture it
    belongs to the graph, so no two calls that may overlap share one."""
    import torch

    if workspace is None:
        workspace = torch.empty(nbytes if nbytes > 0 else 1, dtype=torch.uint8, device=index)
        return workspace, workspace.data_ptr(), nbytes
    p = _ptr_on(workspace, "workspace", torch.uint8, index)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, p, workspace.numel()


def _paged_args(q, cache, kind, block_table, lengths, sm_scale, page_size, starts, req_of_token, logit_cap, slopes,
                q_positions, key_positions, lse, error_word):
    """(device index, the filled DsaPagedArgs); ``out`` and the workspace are left to the caller."""
    import torch

    i32 = torch.int32
    _c_int("page_size", page_size)
    index, cache_ptr, slots = _cache_rows(cache, kind, 264 if kind == CACHE_FP8_SCALED else 256)
    q_ptr = _ptr_on(q, "q", torch.bfloat16, index)
    shape = q.shape
    if len(shape) != 3 or shape[2] != 256:
        raise ValueError("q must be [T, H, 256]")
    T, H = shape[0], shape[1]
    st = q.stride()
    if st[2] != 1:
        raise ValueError("q must be contiguous along its last dimension")
    # without a table or key positions every request reads the same slots: no row to run out of
    bt_ptr, bt_stride, pages, requests = None, 0, 0, 1 << 31
    if block_table is not None:
        # (an empty tensor has no address, and the library would read direct slots)
        bt_ptr, bt_stride, requests, pages = _rows(block_table, "block_table", i32, index, cols=1 if T else 0)
    kp_ptr, kp_stride, kp_width = None, 0, 0
    if key_positions is not None:
        kp_ptr, kp_stride, requests, kp_width = _rows(key_positions, "key_positions", i32, index,
                                                      None if block_table is None else requests, 1 if T else 0)
    if lse is not None and (tuple(lse.shape) != (T, H) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous [T, H] tensor")
    a = DsaPagedArgs(
        q_ptr, st[0] if T > 1 else 0, st[1] if H > 1 else 0, T, H, cache_ptr, kind, slots, 256, 0, 256,
        bt_ptr, bt_stride, page_size, pages, requests, _vector(req_of_token, "req_of_token", T, i32, index),
        _vector(starts, "starts", T, i32, index), _vector(lengths, "lengths", T, i32, index),
        _vector(q_positions, "q_positions", T, i32, index), kp_ptr, kp_stride, kp_width, sm_scale, logit_cap,
        _vector(slopes, "slopes", H, torch.float32, index), None, 0, 0, _ptr_on(lse, "lse", torch.float32, index), None, 0,
        _ptr_on(error_word, "error_word", i32, index))
    return index, a


def dsa_paged_attn_workspace_size(T: int, H: int = 64) -> int:
    """Workspace bytes dsa_paged_attn needs on the current device."""
    a = DsaPagedArgs()
    a.T, a.H = T, H
    n = ctypes.c_size_t(0)
    _check(load_library().dsa_paged_attn_workspace_size(ctypes.byref(a), ctypes.byref(n)),
           "dsa_paged_attn_workspace_size")
    return int(n.value)


def dsa_paged_attn(q, cache, kind: int, block_table, lengths, sm_scale: float, *, page_size: int = 0, starts=None,
                   req_of_token=None, logit_cap: float = 0.0, slopes=None, q_positions=None, key_positions=None,
                   out=None, lse=None, workspace=None, error_word=None):
    """Dense attention of q [T, H, 256] over positions starts[t] .. lengths[t] - 1 of each token's
    request (token t's own request t without ``req_of_token``): bf16 [T, H, 256].

    ``block_table`` int32 [R, pages], or None: position j is slot j. ``logit_cap`` > 0 caps scores
    by a tanh; ``slopes`` fp32 [H] subtracts slopes[h] * |q_position - key_position|. ``lse`` fp32
    [T, H] receives the natural log sum of exp(score)."""
    import torch

    index, a = _paged_args(q, cache, kind, block_table, lengths, sm_scale, page_size, starts, req_of_token, logit_cap,
                           slopes, q_positions, key_positions, lse, error_word)
    T, H = a.T, a.H
    if out is None:
        out = torch.empty((T, H, 256), dtype=torch.bfloat16, device=index)
        a.out, a.out_stride_t, a.out_stride_h = out.data_ptr(), 256 * H, 256
    else:
        a.out = _ptr_on(out, "out", torch.bfloat16, index)
        st = out.stride()
        if tuple(out.shape) != (T, H, 256) or st[2] != 1:
            raise ValueError("out must be [T, H, 256], contiguous along its last dimension")
        a.out_stride_t = st[0] if T > 1 else 256 * H
        a.out_stride_h = st[1] if H > 1 else 256
    with _on_device(index):
        need = _PAGED_WS.get(index)
        if need is None:  # the same for every call on a device
            need = _PAGED_WS[index] = dsa_paged_attn_workspace_size(1)
        workspace, a.workspace, a.workspace_bytes = _workspace_for(workspace, need, index)
        _check((_LIB or load_library()).dsa_paged_attn(ctypes.byref(a), torch.cuda.current_stream(index).cuda_stream),
               "dsa_paged_attn")
    return out


def dsa_paged_attn_mass(q, cache, kind: int, block_table, lengths, sm_scale: float, lse, mass, *, page_size: int = 0,
                        starts=None, req_of_token=None, logit_cap: float = 0.0, slopes=None, q_positions=None,
                        key_positions=None, mass_out=None, error_word=None):
    """Adds each position's attention weight, summed over heads, to ``mass`` fp32 [R, S]: in place,
    or into ``mass_out`` (entries outside the tokens' ranges are left as they are). ``lse`` is
    dsa_paged_attn's on the same arguments. Requests must be strictly ascending. Returns mass_out."""
    import torch

    if lse is None:
        raise ValueError("lse is required")
    index, a = _paged_args(q, cache, kind, block_table, lengths, sm_scale, page_size, starts, req_of_token, logit_cap,
                           slopes, q_positions, key_positions, lse, error_word)
    m_ptr, m_stride, rows, width = _rows(mass, "mass", torch.float32, index,
                                         None if block_table is None and key_positions is None else a.num_requests)
    if mass_out is None:
        mass_out, o_ptr, o_stride = mass, m_ptr, m_stride
    else:
        o_ptr, o_stride, _, o_width = _rows(mass_out, "mass_out", torch.float32, index, rows)
        if o_width != width:
            raise ValueError("mass_out must have mass's shape")
    a.num_requests = rows
    with _on_device(index):
        _check((_LIB or load_library()).dsa_paged_attn_mass(ctypes.byref(a), m_ptr, m_stride, o_ptr, o_stride, width,
                                                            torch.cuda.current_stream(index).cuda_stream),
               "dsa_paged_attn_mass")
    return mass_out


def dsa_cache_evict_workspace_size(num_requests: int, width: int) -> int:
    """Workspace bytes dsa_cache_evict needs for mass rows of ``width`` entries."""
    n = ctypes.c_size_t(0)
    _check(load_library().dsa_cache_evict_workspace_size(num_requests, width, ctypes.byref(n)),
           "dsa_cache_evict_workspace_size")
    return int(n.value)


def dsa_cache_evict(cache, kind: int, block_table, lengths, mass, budget=None, *, page_size: int = 0, sink: int = 0,
                    recent: int = 0, budgets=None, positions=None, mass_out=None, positions_out=None, lengths_out=None,
                    d_nope: int = 256, d_rope: int = 0, workspace=None, error_word=None):
    """Shrinks request r from lengths[r] to at most ``budget`` positions, or budgets[r] (one of the two is
    given), in place in the paged cache: the positions of largest ``mass`` fp32 [R, S] stay, the first
    ``sink`` and ``recent`` newest token positions always. Kept rows past the budget move into the
    evicted places below it; ``mass``, ``positions`` int32 [R, S] (each entry's token position; its
    index without them) and ``lengths`` follow, in place or into the ``_out`` tensors. Returns
    (lengths_out, mass_out, positions_out)."""
    import torch

    i32, f32 = torch.int32, torch.float32
    for name, v in (("budget", 0 if budget is None else budget), ("page_size", page_size), ("sink", sink),
                    ("recent", recent)):
        _c_int(name, v)
    # left out, a budget of 0 would evict everything; beside budgets it would go unused
    if (budget is None) == (budgets is None):
        raise ValueError("one of budget and budgets is required")
    if budget is None:
        budget = 0
    row = d_nope + d_rope if kind == CACHE_BF16 else dsa_packed_row_bytes(d_nope, d_rope)
    index, cache_ptr, slots = _cache_rows(cache, kind, row)
    m_ptr, m_stride, R, S = _rows(mass, "mass", f32, index)
    len_ptr = _vector(lengths, "lengths", R, i32, index)
    if lengths_out is None:
        lengths_out, len_out_ptr = lengths, len_ptr
    else:
        len_out_ptr = _vector(lengths_out, "lengths_out", R, i32, index)
    if mass_out is None:
        mass_out, mo_ptr, mo_stride = mass, m_ptr, m_stride
    else:
        mo_ptr, mo_stride, _, _ = _rows(mass_out, "mass_out", f32, index, R, S)
    p_ptr, p_stride, po_ptr, po_stride = None, 0, None, 0
    if positions is not None:
        p_ptr, p_stride, _, _ = _rows(positions, "positions", i32, index, R, S)
    if positions_out is None:
        positions_out, po_ptr, po_stride = positions, p_ptr, p_stride
    else:
        po_ptr, po_stride, _, _ = _rows(positions_out, "positions_out", i32, index, R, S)
    if R <= 1:  # a single row's stride says nothing; the width passes the library's checks
        m_stride = mo_stride = p_stride = po_stride = S
    bt_ptr, bt_stride, pages = None, 0, 0
    if block_table is not None:
        bt_ptr, bt_stride, _, pages = _rows(block_table, "block_table", i32, index, R, 1 if R else 0)
    a = DsaEvictArgs(cache_ptr, kind, slots, d_nope, d_rope, bt_ptr, bt_stride, page_size, pages, R, len_ptr,
                     _vector(budgets, "budgets", R, i32, index), budget, sink, recent, S, m_ptr, m_stride, p_ptr, p_stride,
                     mo_ptr, mo_stride, po_ptr, po_stride, len_out_ptr, None, 0,
                     _ptr_on(error_word, "error_word", i32, index))
    with _on_device(index):
        need = 0 if workspace is not None else dsa_cache_evict_workspace_size(R, S)
        workspace, a.workspace, a.workspace_bytes = _workspace_for(workspace, need, index)
        _check((_LIB or load_library()).dsa_cache_evict(ctypes.byref(a), torch.cuda.current_stream(index).cuda_stream),
               "dsa_cache_evict")
    return lengths_out, mass_out, positions_out


# --------------------------------------------------------- a serving step around the paged cache --
def _raw_stream(index: int) -> int:
    """The current stream's handle. (torch.cuda.current_stream makes a Python object of it for a microsecond.)"""
    import torch

    return torch._C._cuda_getCurrentRawStream(index)


def dsa_batch_plan(lengths, new_tokens, held, block_table, free_pages, num_free, tokens: int, *, page_size: int,
                   lengths_out=None, held_out=None, num_free_out=None, cu_tokens=None, req_of_token=None, positions=None,
                   token_lengths=None, out_loc=None, error_word=None, seen=None, seen_out=None, token_positions=None,
                   key_positions=None):
    """Brings block tables int32 [R, pages] to the requests' lengths and builds the step's slot maps.

    Request r of ``lengths`` int32 [R] adds ``new_tokens[r]`` positions, or ends when that is negative;
    it holds the first ``held[r]`` pages of its table row. Pages come from, and go back to, the stack
    ``free_pages`` int32 [N] with ``num_free`` int32 [1] entries. ``tokens`` is the room for new tokens
    (a captured step keeps it fixed; entries behind the last token read as padding). ``lengths``,
    ``held`` and ``num_free`` change in place, unless their ``_out`` tensors are given. Returns
    (cu_tokens int32 [R + 1], req_of_token, positions, token_lengths int32 [tokens], out_loc int64
    [tokens]).

    Where the cache evicts, ``seen`` int32 [R] counts each request's tokens (in place, or into ``seen_out``), and
    token_positions int32 [tokens], returned last, are the tokens' places in their sequences, which the rotation
    goes by; ``positions`` then are those among the cached ones. ``key_positions`` int32 [R, S] receives the place
    at each new token's position: what dsa_paged_attn and dsa_cache_evict (as ``positions``) take."""
    import torch

    i32 = torch.int32
    _c_int("page_size", page_size)
    index = _cuda_index(lengths, "lengths", i32)
    R, T = lengths.shape[0], tokens
    if not 0 <= T <= 1 << 30:  # before anything is allocated for them
        raise ValueError("tokens must be 0 .. 2^30")
    bt_ptr, bt_stride, _, pages = _rows(block_table, "block_table", i32, index, R)
    free_ptr = _ptr_on(free_pages, "free_pages", i32, index)
    if free_pages.dim() != 1 or not free_pages.is_contiguous():
        raise ValueError("free_pages must be a contiguous vector")
    if new_tokens is None or held is None or num_free is None:
        raise ValueError("new_tokens, held and num_free are required")
    len_ptr, held_ptr = _vector(lengths, "lengths", R, i32, index), _vector(held, "held", R, i32, index)
    free_n = _vector(num_free, "num_free", 1, i32, index)
    # (between launches a tensor costs 2 us of host time, a view as much again: one tensor each)
    if req_of_token is None:
        req_of_token = torch.empty(T, dtype=i32, device=index)
    if positions is None:
        positions = torch.empty(T, dtype=i32, device=index)
    if token_lengths is None:
        token_lengths = torch.empty(T, dtype=i32, device=index)
    if cu_tokens is None:
        cu_tokens = torch.empty(R + 1, dtype=i32, device=index)
    if out_loc is None:
        out_loc = torch.empty(T, dtype=torch.int64, device=index)
    seen_ptr = _vector(seen, "seen", R, i32, index)
    if seen is None and seen_out is not None:
        raise ValueError("seen_out without seen")
    if seen is not None and token_positions is None:
        token_positions = torch.empty(T, dtype=i32, device=index)
    kp_ptr, kp_stride, kp_width = None, 0, 0
    if key_positions is not None:
        kp_ptr, kp_stride, _, kp_width = _rows(key_positions, "key_positions", i32, index, R)
    a = DsaPlanArgs(
        R, len_ptr, _vector(new_tokens, "new_tokens", R, i32, index), held_ptr, bt_ptr, bt_stride, page_size, pages,
        free_ptr, free_pages.shape[0], free_n,
        len_ptr if lengths_out is None else _vector(lengths_out, "lengths_out", R, i32, index),
        held_ptr if held_out is None else _vector(held_out, "held_out", R, i32, index),
        free_n if num_free_out is None else _vector(num_free_out, "num_free_out", 1, i32, index),
        T, _vector(cu_tokens, "cu_tokens", R + 1, i32, index), _vector(req_of_token, "req_of_token", T, i32, index),
        _vector(positions, "positions", T, i32, index), _vector(token_lengths, "token_lengths", T, i32, index),
        _vector(out_loc, "out_loc", T, torch.int64, index), _ptr_on(error_word, "error_word", i32, index),
        seen_ptr, seen_ptr if seen_out is None else _vector(seen_out, "seen_out", R, i32, index),
        _vector(token_positions, "token_positions", T, i32, index), kp_ptr, kp_stride, kp_width)
    with _on_device(index):
        _check((_LIB or load_library()).dsa_batch_plan(ctypes.byref(a), _raw_stream(index)),
               "dsa_batch_plan")
    got = cu_tokens, req_of_token, positions, token_lengths, out_loc
    return got if token_positions is None else (*got, token_positions)


def dsa_qk_norm_rope(q=None, k=None, positions=None, cos_sin=None, eps: float = 1e-6, cache=None, kind: int = None,
                     out_loc=None, *, d_nope: int = 256, d_rope: int = 0, q_norm: int = 0, k_norm: int = 0,
                     q_weight=None, k_weight=None, interleaved: bool = False, q_out=None, error_word=None):
    """Norm of every query head and of the latent key, rotation of their RoPE columns, and the key's
    cache row, in one pass. Returns q_out (a new tensor by default; q itself for in place), None without q.

    q bf16 [T, H, d_nope + d_rope] and k bf16 [T, d_nope + d_rope], either may be None. The norm covers
    the first ``q_norm`` (``k_norm``) columns: 0 (none), d_nope or d_nope + d_rope, with weights bf16 of
    that size. ``cos_sin`` fp32 [positions, d_rope]: cosines, then sines, of each position's angles; None
    for no rotation. k's row goes to slot ``out_loc[t]`` (t when None) of ``cache``. A token with a
    negative position is padding and left alone."""
    import torch

    bf16, i32 = torch.bfloat16, torch.int32
    lead = q if q is not None else k
    if lead is None:
        raise ValueError("q or k is required")
    index = _cuda_index(lead, "q" if q is not None else "k", bf16)
    T, D = lead.shape[0], d_nope + d_rope
    _c_int("q_norm", q_norm)
    _c_int("k_norm", k_norm)
    H, q_ptr, q_st, q_sh, o_ptr, o_st, o_sh = 0, None, 0, 0, None, 0, 0
    if q is not None:
        st = q.stride()
        shape = q.shape
        if len(shape) != 3 or shape[2] != D or st[2] != 1:
            raise ValueError("q must be [T, H, d_nope + d_rope], contiguous along its last dimension")
        H = shape[1]
        q_ptr, q_st, q_sh = q.data_ptr(), st[0] if T > 1 else 0, st[1] if H > 1 else 0
        if q_out is None:
            q_out = torch.empty((T, H, D), dtype=bf16, device=index)
        o_ptr = _ptr_on(q_out, "q_out", bf16, index)
        st = q_out.stride()
        if q_out.shape != shape or st[2] != 1:
            raise ValueError("q_out must have q's shape, contiguous along its last dimension")
        o_st, o_sh = st[0] if T > 1 else 0, st[1] if H > 1 else 0
    elif q_out is not None:
        raise ValueError("q_out without q")
    k_ptr, k_st, c_ptr, slots = None, 0, None, 0
    if k is not None:
        if cache is None or kind is None:
            raise ValueError("k needs cache and kind")
        k_ptr, k_st, _, width = _rows(k, "k", bf16, index, T)
        if width != D:
            raise ValueError("k must be [T, d_nope + d_rope]")
        # (the packed row of geometries that the library does not know is refused there)
        row = D if kind == CACHE_BF16 else D + d_nope // 32 + d_rope
        c_index, c_ptr, slots = _cache_rows(cache, kind, row)
        if c_index != index:
            raise ValueError(f"cache is on cuda:{c_index}, not on cuda:{index}: every tensor must be on one device")
    cs_ptr, cs_st, cs_n = None, 0, 0
    if cos_sin is not None:
        cs_ptr, cs_st, cs_n, _ = _rows(cos_sin, "cos_sin", torch.float32, index, None, d_rope)
    a = DsaQkArgs(
        T, d_nope, d_rope, q_ptr, q_st, q_sh, H, o_ptr, o_st, o_sh, q_norm,
        None if q is None else _vector(q_weight, "q_weight", q_norm, bf16, index), k_ptr, k_st if T > 1 else 0, k_norm,
        None if k is None else _vector(k_weight, "k_weight", k_norm, bf16, index), c_ptr, 0 if kind is None else kind, slots,
        None if k is None else _vector(out_loc, "out_loc", T, torch.int64, index), eps,
        _vector(positions, "positions", T, i32, index), cs_ptr, cs_st, cs_n, bool(interleaved),
        _ptr_on(error_word, "error_word", i32, index))
    with _on_device(index):
        _check((_LIB or load_library()).dsa_qk_norm_rope(ctypes.byref(a), _raw_stream(index)),
               "dsa_qk_norm_rope")
    return q_out


def dsa_block_pool(cache, kind: int, block_table, positions, lengths, summary, *, page_size: int, req_of_token=None,
                   error_word=None):
    """Writes the mean row of every block (page) that a token of this step lies in to ``summary`` bf16
    [pages, 256]: token t is position positions[t] of request req_of_token[t] (t without it), whose cache
    holds lengths[r] positions. Returns summary."""
    import torch

    i32 = torch.int32
    _c_int("page_size", page_size)
    index, cache_ptr, slots = _cache_rows(cache, kind, 264 if kind == CACHE_FP8_SCALED else 256)
    T = positions.shape[0]
    bt_ptr, bt_stride, R, pages = _rows(block_table, "block_table", i32, index, None, 1 if T else 0)
    s_ptr = _ptr_on(summary, "summary", torch.bfloat16, index)
    if summary.dim() != 2 or summary.shape[1] != 256 or not summary.is_contiguous():
        raise ValueError("summary must be contiguous [pages, 256]")
    with _on_device(index):
        _check((_LIB or load_library()).dsa_block_pool(
            cache_ptr, kind, slots, bt_ptr, bt_stride, page_size, pages, R, _vector(positions, "positions", T, i32, index),
            _vector(req_of_token, "req_of_token", T, i32, index), T, _vector(lengths, "lengths", R, i32, index), s_ptr,
            summary.shape[0], _ptr_on(error_word, "error_word", i32, index),
            _raw_stream(index)), "dsa_block_pool")
    return summary


def dsa_block_scores(q, summary, block_table, lengths, sm_scale: float, *, page_size: int, req_of_token=None, weights=None,
                     out=None, error_word=None):
    """fp32 [T, pages]: for token t and each block b of its first lengths[t] positions, the sum over
    heads of weights[t, h] * max(0, sm_scale * q[t, h] . summary[page of b]) (weight 1 without
    ``weights`` fp32 [T, H]). Entries past the token's blocks are left as they are (-inf in a new result)."""
    import torch

    i32, f32 = torch.int32, torch.float32
    _c_int("page_size", page_size)
    index = _cuda_index(q, "q", torch.bfloat16)
    st = q.stride()
    if q.dim() != 3 or q.shape[2] != 256 or st[2] != 1:
        raise ValueError("q must be [T, H, 256], contiguous along its last dimension")
    T, H = q.shape[0], q.shape[1]
    bt_ptr, bt_stride, R, pages = _rows(block_table, "block_table", i32, index, None, 1 if T else 0)
    s_ptr = _ptr_on(summary, "summary", torch.bfloat16, index)
    if summary.dim() != 2 or summary.shape[1] != 256 or not summary.is_contiguous():
        raise ValueError("summary must be contiguous [pages, 256]")
    if out is None:
        out = torch.full((T, pages), -float("inf"), dtype=f32, device=index)
    o_ptr, o_stride, _, width = _rows(out, "out", f32, index, T, 1)
    if weights is not None and (tuple(weights.shape) != (T, H) or not weights.is_contiguous()):
        raise ValueError("weights must be a contiguous [T, H] tensor")
    with _on_device(index):
        _check((_LIB or load_library()).dsa_block_scores(
            q.data_ptr(), st[0] if T > 1 else 0, st[1] if H > 1 else 0, T, H, s_ptr, summary.shape[0], bt_ptr, bt_stride,
            page_size, pages, R, _vector(req_of_token, "req_of_token", T, i32, index),
            _vector(lengths, "lengths", T, i32, index), sm_scale, _ptr_on(weights, "weights", f32, index), o_ptr, o_stride,
            width, _ptr_on(error_word, "error_word", i32, index), _raw_stream(index)),
            "dsa_block_scores")
    return out


def dsa_block_select(scores, block_table, lengths, K: int, *, page_size: int, req_of_token=None, sink: int = 0,
                     recent: int = 1, blocks=None, table=None, lengths_out=None, error_word=None):
    """The K best blocks of each token by ``scores`` fp32 [T, S], its first ``sink`` and last ``recent``
    always: (blocks int32 [T, K] in ascending order, then -1; table int32 [T, K], their pages;
    lengths_out int32 [T], their positions). dsa_paged_attn(q, cache, kind, table, lengths_out, ...)
    attends to exactly these blocks."""
    import torch

    i32 = torch.int32
    for name, v in (("page_size", page_size), ("K", K), ("sink", sink), ("recent", recent)):
        _c_int(name, v)
    index = _cuda_index(scores, "scores", torch.float32)
    s_ptr, s_stride, T, width = _rows(scores, "scores", torch.float32, index, None, 1)
    bt_ptr, bt_stride, R, pages = _rows(block_table, "block_table", i32, index, None, 1 if T else 0)
    if K < 1:
        raise ValueError("K must be positive")
    if K > 16384:  # before anything is allocated for it
        raise DsaError(2, "dsa_block_select")
    if blocks is None:
        blocks = torch.empty((T, K), dtype=i32, device=index)
    if table is None:
        table = torch.empty((T, K), dtype=i32, device=index)
    if lengths_out is None:
        lengths_out = torch.empty(T, dtype=i32, device=index)
    b_ptr, b_stride, _, b_width = _rows(blocks, "blocks", i32, index, T, K)
    t_ptr, t_stride, _, t_width = _rows(table, "table", i32, index, T, K)
    with _on_device(index):
        _check((_LIB or load_library()).dsa_block_select(
            s_ptr, s_stride, width, T, bt_ptr, bt_stride, page_size, pages, R,
            _vector(req_of_token, "req_of_token", T, i32, index), _vector(lengths, "lengths", T, i32, index), K, sink, recent,
            b_ptr, b_stride, t_ptr, t_stride, _vector(lengths_out, "lengths_out", T, i32, index),
            _ptr_on(error_word, "error_word", i32, index), _raw_stream(index)),
            "dsa_block_select")
    return blocks, table, lengths_out
