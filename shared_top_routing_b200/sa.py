"""Python binding of libsa.so: argument marshalling only.

Every function here passes raw device pointers, sizes and the current CUDA
stream to the C ABI declared in ``include/sa.h``; every step of the path runs
in the library's CUDA kernels.  torch is used for device memory (outputs and
workspaces) and streams.  If ``libsa.so`` is missing the import of a compute
function fails loudly; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsa.so")
LIB_DEBUG_PATH = os.path.join(_HERE, "libsa_debug.so")

SA_OK = 0
SA_ERR_INVALID_ARG = 1
SA_ERR_UNSUPPORTED = 2
SA_ERR_WORKSPACE = 3
SA_ERR_CUDA = 4
SA_ERR_TIMEOUT = 5
SA_ERR_STALE_INDEX = 6
SA_MAX_K = 4096
SA_WS_ALIGN = 256
SA_KV_BF16 = 0
SA_KV_E4M3 = 1
SA_PAGED_MAX_HKV = 8

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_Z = ctypes.c_size_t
_L = ctypes.c_int64

# name -> (restype, argtypes); mirrors include/sa.h
SIGNATURES = {
    "sa_status_string": (ctypes.c_char_p, [_I]),
    "sa_last_error": (ctypes.c_char_p, []),
    "sa_version": (_I, []),
    "sa_index_score_topk_workspace": (_Z, [_I, _I, _I, _I, _I]),
    "sa_index_score_topk": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P]),
    "sa_index_score_topk_mh_workspace": (_Z, [_I, _I, _I, _I, _I, _I]),
    "sa_index_score_topk_mh": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P]),
    "sa_index_score_topk_fp8_workspace": (_Z, [_I, _I, _I, _I, _I]),
    "sa_workspace_status": (_I, [_P, _P]),
    "sa_index_score_topk_fp8": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P]),
    "sa_sparse_attn_prefill": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "sa_sparse_attn_decode_workspace": (_Z, [_I, _I, _I, _I, _I]),
    "sa_sparse_attn_decode": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _Z, _P]),
    "sa_sparse_attn_decode_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "sa_gather_rows": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "sa_sparse_attn_decode_rows": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P, _Z, _P]),
    "sa_paged_row_bytes": (_Z, [_I, _I]),
    "sa_paged_kv_write": (_I, [_P, _P, _L, _L, _P, _P, _P] + [_I] * 8 + [_P, _P, _P]),
    "sa_paged_kv_gather": (_I, [_P] * 5 + [_I] * 8 + [_P, _P, _P]),
    "sa_paged_attn_workspace": (_Z, [_I] * 9),
    "sa_paged_attn": (_I, [_P, _L] + [_P] * 5 + [_I] * 10 + [_F, _P, _P, _P, _Z, _P]),
    "sa_paged_sparse_attn_decode_workspace": (_Z, [_I] * 6),
    "sa_paged_sparse_attn_decode": (_I, [_P] * 6 + [_I] * 9 + [_F, _P, _P, _P, _Z, _P]),
    "sa_self_test_bounded_wait": (_I, [_P, ctypes.c_uint32, _P]),
    "sa_gist_route_unfold_workspace": (_Z, [_I, _I, _I, _I]),
    "sa_gist_route_unfold": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P]),
    "sa_hier_gist_route_unfold": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "sa_index_overlap": (_I, [_P, _P, _P, _P, _I, _I, _P, _P]),
    "sa_index_pattern_greedy": (_I, [_P, _I, _I, ctypes.c_char_p]),
    "sa_debug_enabled": (_I, []),
    "sa_debug_read": (_I, [_P, _I]),
    "sa_debug_check_canary": (_I, [_P, _Z, _I, _P]),
    "sa_index_cache_create": (_I, [_I, ctypes.c_char_p, _I, _I, _I, _I, _P, _P, ctypes.POINTER(_P)]),
    "sa_index_cache_destroy": (None, [_P]),
    "sa_index_cache_is_full": (_I, [_P, _I]),
    "sa_index_cache_owner": (_I, [_P, _I]),
    "sa_index_cache_begin_step": (_I, [_P]),
    "sa_index_cache_update": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "sa_index_cache_mark_written": (_I, [_P, _I]),
    "sa_index_cache_get": (_I, [_P, _I, ctypes.POINTER(_P), ctypes.POINTER(_P),
                                ctypes.POINTER(ctypes.c_uint64)]),
}

_lib = None
_lock = threading.Lock()


class SAError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str):
        super().__init__(f"{func} -> {status_string(status)}: {detail}")
        self.status = status


def lib():
    """The loaded libsa.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"libsa.so not found at {LIB_PATH}; build it with "
                        "`python -m shared_top_routing_b200.build` (no fallback exists)")
                L = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in SIGNATURES.items():
                    f = getattr(L, name)
                    f.restype = res
                    f.argtypes = args
                _lib = L
    return _lib


_lib_debug = None


def lib_debug():
    """The debug build libsa_debug.so (same ABI; see sa.h), loaded on its own."""
    global _lib_debug
    if _lib_debug is None:
        with _lock:
            if _lib_debug is None:
                if not os.path.exists(LIB_DEBUG_PATH):
                    raise RuntimeError(f"libsa_debug.so not found at {LIB_DEBUG_PATH}; build it with "
                                       "`python -m shared_top_routing_b200.build --debug`")
                L = ctypes.CDLL(LIB_DEBUG_PATH)
                for name, (res, args) in SIGNATURES.items():
                    f = getattr(L, name)
                    f.restype = res
                    f.argtypes = args
                _lib_debug = L
    return _lib_debug


def debug_read(L=None, reset: bool = True):
    """The debug record {code, detail, detail, count} of a library (see sa.h)."""
    rec = (ctypes.c_int32 * 4)()
    st = (L or lib_debug()).sa_debug_read(ctypes.cast(rec, ctypes.c_void_p), 1 if reset else 0)
    if st != SA_OK:
        raise SAError(st, "sa_debug_read", last_error())
    return list(rec)


def status_string(s: int) -> str:
    return lib().sa_status_string(s).decode()


def last_error() -> str:
    return lib().sa_last_error().decode()


def _check(status: int, func: str):
    if status != SA_OK:
        raise SAError(status, func, last_error())


# ------------------------------------------------------------ torch plumbing

def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype_size, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.element_size() != dtype_size:
        raise ValueError(f"{name} must have {dtype_size}-byte elements")


_ws_cache: dict = {}


def workspace(nbytes: int, device, key: str = "", stream=None):
    """A cached, zero-filled device workspace of at least ``nbytes`` (256-byte
    aligned).  The decode-attention workspace must start zero-filled; the
    library returns its ticket region to zero after each call, so the cache
    can hand the same buffer to later calls of any shape.  Host threads that
    call on one stream at the same time must pass workspaces of their own."""
    torch = _torch()
    if nbytes <= 0:
        return None
    s = stream if stream is not None else torch.cuda.current_stream(device)
    k = (str(device), s.cuda_stream, key)
    buf = _ws_cache.get(k)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        _ws_cache[k] = buf
    return buf


# --------------------------------------------------------------- the calls

def sa_index_score_topk(q_idx, k_idx, k: int, Tk: int | None = None, q_pos0: int | None = None,
                        kv_len=None, idx_out=None, count_out=None, with_scores: bool = False,
                        ws=None, stream=None):
    """Indexer scores + per-query top-k (see sa.h).

    q_idx [B, Tq, d] or [B, d] (decode) bf16; k_idx [B, Tk_max, d] bf16.
    Tk defaults to Tk_max; q_pos0 defaults to Tk - Tq (prefill whose queries
    are the last Tq cached tokens; for decode Tk - 1).
    Returns (idx [B, Tq, k] int32, count [B, Tq] int32[, score [B, Tq, k] fp32]).
    """
    torch = _torch()
    decode_shape = q_idx.dim() == 2
    q3 = q_idx.unsqueeze(1) if decode_shape else q_idx
    B, Tq, d = q3.shape
    Tk_max = k_idx.shape[1]
    Tk = Tk_max if Tk is None else Tk
    q_pos0 = Tk - Tq if q_pos0 is None else q_pos0
    _need(q3, "q_idx", 2)
    _need(k_idx, "k_idx", 2)
    dev = q3.device
    if idx_out is None:
        idx_out = torch.empty((B, Tq, k), dtype=torch.int32, device=dev)
    if count_out is None:
        count_out = torch.empty((B, Tq), dtype=torch.int32, device=dev)
    score = torch.empty((B, Tq, k), dtype=torch.float32, device=dev) if with_scores else None
    need = lib().sa_index_score_topk_workspace(B, Tq, Tk_max, d, k)
    if ws is None:
        ws = workspace(need, dev, "index", stream)
    st = lib().sa_index_score_topk(_ptr(q3), _ptr(k_idx), B, Tq, Tk, Tk_max, d, k, q_pos0,
                                   _ptr(kv_len), _ptr(idx_out), _ptr(count_out), _ptr(score),
                                   _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))
    _check(st, "sa_index_score_topk")
    if decode_shape:
        idx_v, cnt_v = idx_out.view(B, k), count_out.view(B)
        return (idx_v, cnt_v, score.view(B, k)) if with_scores else (idx_v, cnt_v)
    return (idx_out, count_out, score) if with_scores else (idx_out, count_out)


def sa_index_score_topk_mh(q_idx, w, k_idx, k: int, Tk: int | None = None, q_pos0: int | None = None,
                           kv_len=None, idx_out=None, count_out=None, with_scores: bool = False,
                           ws=None, stream=None):
    """Multi-head weighted indexer scores + per-query top-k (see sa.h).

    q_idx [B, Tq, H, d] or [B, H, d] (decode) bf16; w [B, Tq, H] or [B, H]
    fp32; k_idx [B, Tk_max, d] bf16.  Defaults and results as for
    sa_index_score_topk.
    """
    torch = _torch()
    decode_shape = q_idx.dim() == 3
    q4 = q_idx.unsqueeze(1) if decode_shape else q_idx
    w3 = w.unsqueeze(1) if decode_shape else w
    B, Tq, H, d = q4.shape
    Tk_max = k_idx.shape[1]
    Tk = Tk_max if Tk is None else Tk
    q_pos0 = Tk - Tq if q_pos0 is None else q_pos0
    _need(q4, "q_idx", 2)
    _need(w3, "w", 4)
    _need(k_idx, "k_idx", 2)
    dev = q4.device
    if idx_out is None:
        idx_out = torch.empty((B, Tq, k), dtype=torch.int32, device=dev)
    if count_out is None:
        count_out = torch.empty((B, Tq), dtype=torch.int32, device=dev)
    score = torch.empty((B, Tq, k), dtype=torch.float32, device=dev) if with_scores else None
    need = lib().sa_index_score_topk_mh_workspace(B, Tq, Tk_max, H, d, k)
    if ws is None:
        ws = workspace(need, dev, "index_mh", stream)
    st = lib().sa_index_score_topk_mh(_ptr(q4), _ptr(w3), _ptr(k_idx), B, Tq, H, Tk, Tk_max, d, k, q_pos0,
                                      _ptr(kv_len), _ptr(idx_out), _ptr(count_out), _ptr(score),
                                      _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))
    _check(st, "sa_index_score_topk_mh")
    if decode_shape:
        idx_v, cnt_v = idx_out.view(B, k), count_out.view(B)
        return (idx_v, cnt_v, score.view(B, k)) if with_scores else (idx_v, cnt_v)
    return (idx_out, count_out, score) if with_scores else (idx_out, count_out)


def sa_index_score_topk_fp8(q_idx, k_idx, k: int, w=None, Tk: int | None = None, q_pos0: int | None = None,
                            kv_len=None, idx_out=None, count_out=None, with_scores: bool = False,
                            ws=None, stream=None):
    """fp8 (E4M3) indexer scores + top-k of one decode query per sequence
    (see sa.h).

    q_idx [B, d] (one head) or [B, H, d]; k_idx [B, Tk_max, d]: E4M3 codes as
    uint8 (or torch.float8_e4m3fn) tensors.  w [B, H] fp32 selects the
    multi-head score; without it H must be 1.  Tk defaults to Tk_max, q_pos0
    to Tk - 1.  Returns (idx [B, k] int32, count [B] int32[, score [B, k]]).
    """
    torch = _torch()
    as_bytes = lambda t: t.view(torch.uint8) if t.dtype != torch.uint8 else t
    q3 = as_bytes(q_idx)
    q3 = q3.unsqueeze(1) if q3.dim() == 2 else q3
    kb = as_bytes(k_idx)
    B, H, d = q3.shape
    Tk_max = kb.shape[1]
    Tk = Tk_max if Tk is None else Tk
    q_pos0 = Tk - 1 if q_pos0 is None else q_pos0
    _need(q3, "q_idx", 1)
    _need(kb, "k_idx", 1)
    if w is not None:
        _need(w, "w", 4)
    dev = q3.device
    if idx_out is None:
        idx_out = torch.empty((B, k), dtype=torch.int32, device=dev)
    if count_out is None:
        count_out = torch.empty((B,), dtype=torch.int32, device=dev)
    score = torch.empty((B, k), dtype=torch.float32, device=dev) if with_scores else None
    need = lib().sa_index_score_topk_fp8_workspace(B, Tk_max, H, d, k)
    if ws is None:
        ws = workspace(need, dev, "index", stream)
    st = lib().sa_index_score_topk_fp8(_ptr(q3), _ptr(w), _ptr(kb), B, H, Tk, Tk_max, d, k, q_pos0, _ptr(kv_len),
                                       _ptr(idx_out), _ptr(count_out), _ptr(score), _ptr(ws),
                                       0 if ws is None else ws.numel(), _stream(stream))
    _check(st, "sa_index_score_topk_fp8")
    return (idx_out, count_out, score) if with_scores else (idx_out, count_out)


def sa_workspace_status(ws, stream=None) -> int:
    """The status the error word at the start of a workspace reports (see
    sa.h): SA_OK, or SA_ERR_TIMEOUT when a kernel wait of a call that used it
    gave up.  Synchronizes `stream`."""
    return lib().sa_workspace_status(_ptr(ws), _stream(stream))


def sa_sparse_attn_prefill(q, k_cache, v_cache, idx, count, scale: float = 0.0, out=None,
                           with_lse: bool = False, stream=None):
    """q [B, T, Hq, D]; k_cache/v_cache [B, Tk_max, Hkv, D]; idx [B, T, k]; count [B, T]."""
    torch = _torch()
    B, T, Hq, D = q.shape
    _, Tk_max, Hkv, _ = k_cache.shape
    k = idx.shape[-1]
    for t, n, sz in ((q, "q", 2), (k_cache, "k_cache", 2), (v_cache, "v_cache", 2),
                     (idx, "idx", 4), (count, "count", 4)):
        _need(t, n, sz)
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device) if with_lse else None
    st = lib().sa_sparse_attn_prefill(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx), _ptr(count),
                                      B, T, Tk_max, Hq, Hkv, D, k, scale, _ptr(out), _ptr(lse),
                                      _stream(stream))
    _check(st, "sa_sparse_attn_prefill")
    return (out, lse) if with_lse else out


def sa_sparse_attn_decode(q, k_cache, v_cache, idx, count, scale: float = 0.0, out=None,
                          with_lse: bool = False, ws=None, stream=None):
    """q [B, Hq, D]; k_cache/v_cache [B, Tk_max, Hkv, D]; idx [B, k]; count [B]."""
    torch = _torch()
    B, Hq, D = q.shape
    _, Tk_max, Hkv, _ = k_cache.shape
    k = idx.shape[-1]
    for t, n, sz in ((q, "q", 2), (k_cache, "k_cache", 2), (v_cache, "v_cache", 2),
                     (idx, "idx", 4), (count, "count", 4)):
        _need(t, n, sz)
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if with_lse else None
    need = lib().sa_sparse_attn_decode_workspace(B, Hq, Hkv, D, k)
    if ws is None:
        ws = workspace(need, q.device, "attn_decode", stream)
    st = lib().sa_sparse_attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx), _ptr(count),
                                     B, Tk_max, Hq, Hkv, D, k, scale, _ptr(out), _ptr(lse),
                                     _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream))
    _check(st, "sa_sparse_attn_decode")
    return (out, lse) if with_lse else out


def sa_gather_rows(k_cache, v_cache, idx, count, k_rows=None, v_rows=None, stream=None):
    """Compact copies [B, k, Hkv * D + 8] of the selected rows (zeros past
    count; the last 8 values of each row are a zero pad, see sa.h)."""
    torch = _torch()
    B, Tk_max, Hkv, D = k_cache.shape
    k = idx.shape[-1]
    for t, n, sz in ((k_cache, "k_cache", 2), (v_cache, "v_cache", 2), (idx, "idx", 4), (count, "count", 4)):
        _need(t, n, sz)
    if k_rows is None:
        k_rows = torch.empty((B, k, Hkv * D + 8), dtype=k_cache.dtype, device=k_cache.device)
    if v_rows is None:
        v_rows = torch.empty((B, k, Hkv * D + 8), dtype=v_cache.dtype, device=v_cache.device)
    st = lib().sa_gather_rows(_ptr(k_cache), _ptr(v_cache), _ptr(idx), _ptr(count), B, Tk_max, Hkv, D, k,
                              _ptr(k_rows), _ptr(v_rows), _stream(stream))
    _check(st, "sa_gather_rows")
    return k_rows, v_rows


def sa_sparse_attn_decode_rows(q, k_rows, v_rows, count, scale: float = 0.0, out=None, with_lse: bool = False,
                               ws=None, stream=None):
    """q [B, Hq, D]; k_rows / v_rows [B, k, Hkv * D + 8] compact rows (from
    sa_gather_rows); count [B]."""
    torch = _torch()
    B, Hq, D = q.shape
    _, k, row = k_rows.shape
    Hkv = (row - 8) // D
    for t, n, sz in ((q, "q", 2), (k_rows, "k_rows", 2), (v_rows, "v_rows", 2), (count, "count", 4)):
        _need(t, n, sz)
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if with_lse else None
    need = lib().sa_sparse_attn_decode_workspace(B, Hq, Hkv, D, k)
    if ws is None:
        ws = workspace(need, q.device, "attn_decode", stream)
    st = lib().sa_sparse_attn_decode_rows(_ptr(q), _ptr(k_rows), _ptr(v_rows), _ptr(count), B, Hq, Hkv, D, k,
                                          scale, _ptr(out), _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(),
                                          _stream(stream))
    _check(st, "sa_sparse_attn_decode_rows")
    return (out, lse) if with_lse else out


# ------------------------------------------------------------- paged cache

_D = 128


def sa_paged_kv_alloc(num_pages: int, page_size: int, Hkv: int, kv_type: int = SA_KV_BF16, device=None):
    """Zero-filled K and V pools [num_pages, page_size, row] of a paged cache
    (see sa.h): bf16 rows of Hkv * 128 + 8 values, or uint8 rows of
    Hkv * 128 E4M3 codes and 16 bytes of scales."""
    torch = _torch()
    nbytes = lib().sa_paged_row_bytes(kv_type, Hkv)
    if nbytes == 0:
        raise ValueError(f"no paged cache of kv_type {kv_type} and {Hkv} kv heads (1 to {SA_PAGED_MAX_HKV})")
    dtype, row = (torch.bfloat16, nbytes // 2) if kv_type == SA_KV_BF16 else (torch.uint8, nbytes)
    return tuple(torch.zeros((num_pages, page_size, row), dtype=dtype, device=device) for _ in range(2))


# The checks below run on every call of a decode step, so they are written for
# few interpreter steps: devices as ordinals, one tuple comparison per shape,
# torch's names looked up once.  Of the ways to allocate, empty_like and
# empty_strided take the least time.

_bf16 = _u8 = _i32 = _f32 = _cuda = _empty_like = _empty_strided = None


def _names():
    global _bf16, _u8, _i32, _f32, _cuda, _empty_like, _empty_strided
    torch = _torch()
    _u8, _i32, _f32, _cuda = torch.uint8, torch.int32, torch.float32, torch._C
    _empty_like, _empty_strided, _bf16 = torch.empty_like, torch.empty_strided, torch.bfloat16


def _pools(k_pages, v_pages, dev):
    """(kv_type, Hkv) of a pair of pools on CUDA device `dev` (an ordinal): by
    their element type and row size."""
    if _bf16 is None:
        _names()
    dtype, shape = k_pages.dtype, k_pages.shape
    if dtype is _bf16:
        kv_type, pad = SA_KV_BF16, 8
    elif dtype is _u8:
        kv_type, pad = SA_KV_E4M3, 16
    else:
        raise ValueError("k_pages must be bfloat16, or uint8 for E4M3 rows")
    if len(shape) != 3 or v_pages.shape != shape or v_pages.dtype is not dtype:
        raise ValueError("k_pages and v_pages must be pools [num_pages, page_size, row] of one shape and type")
    Hkv, rest = divmod(shape[2] - pad, _D)
    if rest or Hkv < 1:
        raise ValueError(f"rows of {shape[2]} elements are not a paged cache's (see sa.h)")
    if k_pages.get_device() != dev or v_pages.get_device() != dev:
        raise ValueError(f"k_pages and v_pages must be on {_name(dev)}")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages and v_pages must be contiguous")
    return kv_type, Hkv


def _name(dev):
    return "the CPU" if dev < 0 else f"cuda:{dev}"


def _ints32(t, name, dev, shape):
    if t.dtype is not (_i32 or _torch().int32) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on {_name(dev)}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, has {list(t.shape)}")


def _tokens(t, name):
    """(device ordinal, shape, token stride) of [N, H, 128] bf16 rows whose
    heads lie side by side."""
    if _bf16 is None:
        _names()
    dev = t.get_device()
    if dev < 0 or t.dtype is not _bf16:
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must have shape [N, heads, {_D}]")
    N, H, D = shape
    st = t.stride()
    if D > 1 and st[2] != 1 or H > 1 and st[1] != D:
        raise ValueError(f"{name}'s heads must lie side by side in a token")
    return dev, shape, st[0] if N > 1 else max(8, H * D)


def _result(t, name, dev, shape, dtype):
    """An output buffer the caller gave, checked."""
    if t.dtype != dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {_name(dev)}")
    return t


def _call_stream(dev, stream):
    """(raw stream, context or None) a call on tensors of device `dev` runs on:
    the given stream, or the current one of that device.  The context makes
    the device (and a given stream, so that outputs belong to it) current;
    None when they are already."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"the stream is of {stream.device}, the tensors are on {_name(dev)}")
        return stream.cuda_stream, _torch().cuda.stream(stream)
    raw = _cuda._cuda_getCurrentRawStream(dev)
    return raw, None if _cuda._cuda_getDevice() == dev else _torch().cuda.device(dev)


_paged_ws: dict = {}
_paged_ws_need: dict = {}

# A call's kernels hand results to one another through the stream's workspace,
# and ctypes lets other host threads run meanwhile: a call on the same stream
# must come before or after them all, and must not replace the buffer between
# them.  So a lock per stream (default streams of all devices share one) is
# held from the look-up until all kernels are enqueued; a call that was given a
# workspace holds none.
_paged_locks: dict = {}
_no_lock = contextlib.nullcontext()


def _new_lock(raw):
    return _paged_locks.setdefault(raw, threading.Lock())


def _paged_workspace(nbytes: int, dev: int, raw_stream: int):
    """A workspace for one call on a stream (whose device is current).  Outside
    a capture, one buffer per stream is kept and grows.  A capture gets a
    buffer of its own from the graph's memory, zeroed by the graph, so that
    graphs share none with each other or with calls outside."""
    if _cuda._cuda_isCurrentStreamCapturing():
        buf = _torch().empty(nbytes, dtype=_u8, device=f"cuda:{dev}")
        buf[:SA_WS_ALIGN].zero_()
        return buf
    key = (dev, raw_stream)
    buf = _paged_ws.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = _torch().zeros(nbytes, dtype=_u8, device=f"cuda:{dev}")
        _paged_ws[key] = buf
    return buf


def _paged_ws_args(L, size_of, sizes, ws, dev, raw):
    """(pointer, bytes, tensor) of the call's workspace, the tensor to be held
    until the launch; its size is a function of the call's sizes alone and is
    looked up once."""
    key = (L._handle, dev, size_of, sizes)
    need = _paged_ws_need.get(key)
    if need is None:
        if len(_paged_ws_need) > 4096:   # (a server meets new sizes for ever)
            _paged_ws_need.clear()
        need = _paged_ws_need[key] = getattr(L, size_of)(*sizes)
    if ws is None:
        if need == 0:
            return None, 0, None
        ws = _paged_workspace(need, dev, raw)
        return ws.data_ptr(), need, ws
    if ws.get_device() != dev:
        raise ValueError(f"ws must be on {_name(dev)}")
    if not ws.is_contiguous():   # (an expanded tensor has less memory than elements)
        raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def sa_paged_kv_write(k_new, v_new, k_pages, v_pages, block_table, q_start, kv_len, stream=None):
    """Writes the new tokens' K and V into the pools, in place (see sa.h).

    k_new, v_new [N, Hkv, 128] bf16 (slices of a fused projection are fine);
    pools from sa_paged_kv_alloc; block_table [B, max_pages], q_start [B + 1],
    kv_len [B] int32, kv_len counting the new tokens.  Returns the pools."""
    dev, kshape, ks = _tokens(k_new, "k_new")
    vdev, vshape, vs = _tokens(v_new, "v_new")
    kv_type, Hkv = _pools(k_pages, v_pages, dev)
    pages, page_size, _ = k_pages.shape
    N = kshape[0]
    if kshape != (N, Hkv, _D) or vshape != kshape or vdev != dev:
        raise ValueError(f"k_new and v_new must have shape [N, {Hkv}, {_D}], on one device")
    B, cols = _table(block_table, dev)
    _ints32(q_start, "q_start", dev, (B + 1,))
    _ints32(kv_len, "kv_len", dev, (B,))
    raw, ctx = _call_stream(dev, stream)
    args = (k_new.data_ptr(), v_new.data_ptr(), ks, vs, q_start.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(), B,
            N, cols, pages, page_size, Hkv, _D, kv_type, k_pages.data_ptr(), v_pages.data_ptr(), raw)
    if ctx is None:
        st = lib().sa_paged_kv_write(*args)
    else:
        with ctx:
            st = lib().sa_paged_kv_write(*args)
    _check(st, "sa_paged_kv_write")
    return k_pages, v_pages


def _table(block_table, dev):
    """(sequences, columns) of a block table."""
    shape = block_table.shape
    if len(shape) != 2:
        raise ValueError("block_table must have shape [B, max_pages]")
    if block_table.dtype is not _i32 or block_table.get_device() != dev or not block_table.is_contiguous():
        _ints32(block_table, "block_table", dev, shape)   # (says what is wrong)
    return shape


def _selection(idx, count, B, dev):
    """k of a selection idx [B, k], count [B]."""
    if idx.dim() != 2:
        raise ValueError("idx must have shape [B, k]")
    k = idx.shape[1]
    _ints32(idx, "idx", dev, (B, k))
    _ints32(count, "count", dev, (B,))
    return k


def sa_paged_kv_gather(k_pages, v_pages, block_table, idx, count, k_rows=None, v_rows=None, stream=None):
    """Selected rows of a paged cache as compact bf16 rows [B, k, Hkv * 128 + 8]
    (zeros past count), for sa_sparse_attn_decode_rows.  idx [B, k], count [B]."""
    dev = k_pages.get_device()
    kv_type, Hkv = _pools(k_pages, v_pages, dev)
    pages, page_size, _ = k_pages.shape
    B, cols = _table(block_table, dev)
    k = _selection(idx, count, B, dev)
    if dev < 0:
        raise ValueError("k_pages must be a CUDA tensor")
    raw, ctx = _call_stream(dev, stream)
    if ctx is not None:
        with ctx:
            return _gather(k_pages, v_pages, block_table, idx, count, k_rows, v_rows, kv_type, Hkv, pages, page_size, B,
                           cols, k, dev, raw)
    return _gather(k_pages, v_pages, block_table, idx, count, k_rows, v_rows, kv_type, Hkv, pages, page_size, B, cols, k,
                   dev, raw)


def _gather(k_pages, v_pages, block_table, idx, count, k_rows, v_rows, kv_type, Hkv, pages, page_size, B, cols, k, dev,
            raw):
    row = Hkv * _D + 8
    shape = (B, k, row)

    def rows(t, name):
        if t is None:
            return _empty_strided(shape, (k * row, row, 1), dtype=_bf16, device=k_pages.device)
        return _result(t, name, dev, shape, _bf16)

    k_rows, v_rows = rows(k_rows, "k_rows"), rows(v_rows, "v_rows")
    st = lib().sa_paged_kv_gather(k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), idx.data_ptr(),
                                  count.data_ptr(), B, cols, pages, page_size, Hkv, _D, k, kv_type, k_rows.data_ptr(),
                                  v_rows.data_ptr(), raw)
    _check(st, "sa_paged_kv_gather")
    return k_rows, v_rows


def _outputs(q, shape, out, with_lse, dev):
    """(out, lse or None) of queries q [N, Hq, 128]."""
    N, Hq, D = shape
    if out is not None:
        _result(out, "out", dev, shape, _bf16)
    elif q.is_contiguous():
        out = _empty_like(q)
    else:
        out = _empty_strided(shape, (Hq * D, D, 1), dtype=_bf16, device=q.device)
    return out, _empty_strided((N, Hq), (Hq, 1), dtype=_f32, device=q.device) if with_lse else None


def sa_paged_attn(q, k_pages, v_pages, block_table, q_start, kv_len, max_q: int | None = None, scale: float = 0.0,
                  out=None, with_lse: bool = False, ws=None, stream=None):
    """Attention of a chunk of new tokens per sequence over a paged cache, each
    token over every position up to its own (see sa.h).

    q [N, Hq, 128] bf16, the sequences' tokens packed by q_start [B + 1];
    kv_len [B] counts them; max_q bounds the tokens of one sequence (1 for
    decode).  By default it is N, which is always right but plans a batch of
    single tokens as long chunks: give the bound where it is known (see sa.h).
    Returns out [N, Hq, 128][, lse [N, Hq] fp32]; rows of tokens that belong to
    no sequence are left as they were, in an out of the call's own undefined.

    ws: uint8 device memory, zero-filled before first use, for one call at a
    time.  Without it a buffer per stream is kept for the life of the process
    (a call captured into a graph gets its own); for long chunks of E4M3 caches
    it may reach 1 GiB, so a program that wants that memory back passes ws."""
    dev, shape, qs = _tokens(q, "q")
    kv_type, Hkv = _pools(k_pages, v_pages, dev)
    pages, page_size, _ = k_pages.shape
    B, cols = _table(block_table, dev)
    _ints32(q_start, "q_start", dev, (B + 1,))
    _ints32(kv_len, "kv_len", dev, (B,))
    raw, ctx = _call_stream(dev, stream)
    if ctx is not None:
        with ctx:
            return _attn(q, k_pages, v_pages, block_table, q_start, kv_len, max_q, scale, out, with_lse, ws, dev, shape,
                         qs, kv_type, Hkv, pages, page_size, B, cols, raw)
    return _attn(q, k_pages, v_pages, block_table, q_start, kv_len, max_q, scale, out, with_lse, ws, dev, shape, qs,
                 kv_type, Hkv, pages, page_size, B, cols, raw)


def _attn(q, k_pages, v_pages, block_table, q_start, kv_len, max_q, scale, out, with_lse, ws, dev, shape, qs, kv_type,
          Hkv, pages, page_size, B, cols, raw):
    L = lib()
    N, Hq, D = shape
    max_q = N if max_q is None else max_q
    out, lse = _outputs(q, shape, out, with_lse, dev)
    with _no_lock if ws is not None else _paged_locks.get(raw) or _new_lock(raw):
        wp, wn, ws = _paged_ws_args(L, "sa_paged_attn_workspace", (B, N, max_q, cols, page_size, Hq, Hkv, D, kv_type),
                                    ws, dev, raw)
        st = L.sa_paged_attn(q.data_ptr(), qs, k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                             q_start.data_ptr(), kv_len.data_ptr(), B, N, max_q, cols, pages, page_size, Hq, Hkv, D,
                             kv_type, scale, out.data_ptr(), None if lse is None else lse.data_ptr(), wp, wn, raw)
    _check(st, "sa_paged_attn")
    return (out, lse) if with_lse else out


def sa_paged_sparse_attn_decode(q, k_pages, v_pages, block_table, idx, count, scale: float = 0.0, out=None,
                                with_lse: bool = False, ws=None, stream=None):
    """sa_sparse_attn_decode over a paged cache: q [B, Hq, 128]; idx [B, k]
    positions; count [B]; ws as for sa_paged_attn.  Returns out [B, Hq, 128][,
    lse [B, Hq] fp32]."""
    dev, shape, _ = _tokens(q, "q")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    kv_type, Hkv = _pools(k_pages, v_pages, dev)
    pages, page_size, _ = k_pages.shape
    B, cols = _table(block_table, dev)
    if shape[0] != B:
        raise ValueError(f"q must have shape [{B}, heads, {_D}]: one token per sequence")
    k = _selection(idx, count, B, dev)
    raw, ctx = _call_stream(dev, stream)
    if ctx is not None:
        with ctx:
            return _sparse(q, k_pages, v_pages, block_table, idx, count, scale, out, with_lse, ws, dev, shape, kv_type,
                           Hkv, pages, page_size, cols, k, raw)
    return _sparse(q, k_pages, v_pages, block_table, idx, count, scale, out, with_lse, ws, dev, shape, kv_type, Hkv,
                   pages, page_size, cols, k, raw)


def _sparse(q, k_pages, v_pages, block_table, idx, count, scale, out, with_lse, ws, dev, shape, kv_type, Hkv, pages,
            page_size, cols, k,
            raw):
    L = lib()
    B, Hq, D = shape
    out, lse = _outputs(q, shape, out, with_lse, dev)
    with _no_lock if ws is not None else _paged_locks.get(raw) or _new_lock(raw):
        wp, wn, ws = _paged_ws_args(L, "sa_paged_sparse_attn_decode_workspace", (B, Hq, Hkv, D, k, kv_type), ws, dev, raw)
        st = L.sa_paged_sparse_attn_decode(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                                           idx.data_ptr(), count.data_ptr(), B, cols, pages, page_size, Hq, Hkv, D, k,
                                           kv_type, scale, out.data_ptr(), None if lse is None else lse.data_ptr(), wp,
                                           wn, raw)
    _check(st, "sa_paged_sparse_attn_decode")
    return (out, lse) if with_lse else out


def sa_sparse_attn_decode_noalloc(q, k_cache, v_cache, idx, count, scale: float = 0.0, out=None,
                                  with_lse: bool = False, stream=None):
    """sa_sparse_attn_decode for callers that cannot allocate: no workspace
    argument; the library's fixed scratch array is used (see sa.h)."""
    torch = _torch()
    B, Hq, D = q.shape
    _, Tk_max, Hkv, _ = k_cache.shape
    k = idx.shape[-1]
    for t, n, sz in ((q, "q", 2), (k_cache, "k_cache", 2), (v_cache, "v_cache", 2),
                     (idx, "idx", 4), (count, "count", 4)):
        _need(t, n, sz)
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device) if with_lse else None
    st = lib().sa_sparse_attn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(idx),
                                             _ptr(count), B, Tk_max, Hq, Hkv, D, k, scale, _ptr(out),
                                             _ptr(lse), _stream(stream))
    _check(st, "sa_sparse_attn_decode_noalloc")
    return (out, lse) if with_lse else out


def sa_self_test_bounded_wait(poll_limit: int = 4096, stream=None):
    """Runs the library's bounded-wait probe on the GPU and returns its five
    result words (see sa.h): a wait nothing completes must give up with code
    77 and set its abort flag; a wait that completes must succeed."""
    import torch
    err = torch.zeros(5, dtype=torch.int32, device="cuda")
    st = lib().sa_self_test_bounded_wait(_ptr(err), poll_limit, _stream(stream))
    _check(st, "sa_self_test_bounded_wait")
    return err


def sa_gist_route_unfold(q_route, gist_key, chunk_len: int, k_chunks: int, partial_len,
                         rows_out=None, count_out=None, with_chunks: bool = False, ws=None,
                         stream=None):
    """q_route [B, d]; gist_key [B, n_chunks, d]; partial_len [B] int32 (device).
    Returns (rows [B, k_chunks*(chunk_len+1)+chunk_len], count [B][, chunks [B, k_chunks]])."""
    torch = _torch()
    B, d = q_route.shape
    n_chunks = gist_key.shape[1]
    _need(q_route, "q_route", 2)
    _need(gist_key, "gist_key", 2)
    _need(partial_len, "partial_len", 4)
    dev = q_route.device
    stride = k_chunks * (chunk_len + 1) + chunk_len
    if rows_out is None:
        rows_out = torch.empty((B, stride), dtype=torch.int32, device=dev)
    if count_out is None:
        count_out = torch.empty((B,), dtype=torch.int32, device=dev)
    chunks = torch.empty((B, k_chunks), dtype=torch.int32, device=dev) if with_chunks else None
    need = lib().sa_gist_route_unfold_workspace(B, n_chunks, d, k_chunks)
    if ws is None:
        ws = workspace(need, dev, "gist", stream)
    st = lib().sa_gist_route_unfold(_ptr(q_route), _ptr(gist_key), B, n_chunks, chunk_len, d,
                                    k_chunks, _ptr(partial_len), _ptr(rows_out), _ptr(count_out),
                                    _ptr(chunks), _ptr(ws), 0 if ws is None else ws.numel(),
                                    _stream(stream))
    _check(st, "sa_gist_route_unfold")
    return (rows_out, count_out, chunks) if with_chunks else (rows_out, count_out)


def sa_hier_gist_route_unfold(q_route, meta_key, gist_key, chunk_len: int, group_size: int, k_groups: int,
                              k_chunks: int, partial_len=None, rows_out=None, count_out=None,
                              with_chunks: bool = False, with_groups: bool = False, stream=None):
    """Two-level gist routing (see sa.h).  q_route [B, d]; meta_key
    [B, n_chunks // group_size, d]; gist_key [B, n_chunks, d].
    Returns (rows, count[, chunks][, groups])."""
    torch = _torch()
    B, d = q_route.shape
    n_chunks = gist_key.shape[1]
    _need(q_route, "q_route", 2)
    _need(meta_key, "meta_key", 2)
    _need(gist_key, "gist_key", 2)
    if partial_len is not None:
        _need(partial_len, "partial_len", 4)
    dev = q_route.device
    stride = k_chunks * (chunk_len + 1) + chunk_len
    if rows_out is None:
        rows_out = torch.empty((B, stride), dtype=torch.int32, device=dev)
    if count_out is None:
        count_out = torch.empty((B,), dtype=torch.int32, device=dev)
    chunks = torch.empty((B, k_chunks), dtype=torch.int32, device=dev) if with_chunks else None
    groups = torch.empty((B, k_groups), dtype=torch.int32, device=dev) if with_groups else None
    st = lib().sa_hier_gist_route_unfold(_ptr(q_route), _ptr(meta_key), _ptr(gist_key), B, n_chunks, chunk_len,
                                         group_size, d, k_groups, k_chunks, _ptr(partial_len), _ptr(rows_out),
                                         _ptr(count_out), _ptr(chunks), _ptr(groups), _stream(stream))
    _check(st, "sa_hier_gist_route_unfold")
    res = [rows_out, count_out]
    if with_chunks:
        res.append(chunks)
    if with_groups:
        res.append(groups)
    return tuple(res)


def sa_index_overlap(idx_a, count_a, idx_b, count_b, out=None, stream=None):
    """Per-row count of the positions two selections share.  idx_* [..., k]
    int32 (ascending rows); count_* [...] int32.  Returns int32 [rows]."""
    torch = _torch()
    k = idx_a.shape[-1]
    rows = idx_a.numel() // k
    for t, n in ((idx_a, "idx_a"), (idx_b, "idx_b"), (count_a, "count_a"), (count_b, "count_b")):
        _need(t, n, 4)
    if out is None:
        out = torch.empty((rows,), dtype=torch.int32, device=idx_a.device)
    st = lib().sa_index_overlap(_ptr(idx_a), _ptr(count_a), _ptr(idx_b), _ptr(count_b), rows, k, _ptr(out),
                                _stream(stream))
    _check(st, "sa_index_overlap")
    return out


def sa_index_pattern_greedy(overlap, n_full: int) -> str:
    """Greedy layer-role search on an [L, L] overlap matrix (host; see sa.h)."""
    import numpy as np
    ov = np.ascontiguousarray(np.asarray(overlap, dtype=np.float64))
    L = ov.shape[0]
    buf = ctypes.create_string_buffer(L + 1)
    st = lib().sa_index_pattern_greedy(ov.ctypes.data_as(ctypes.c_void_p), L, n_full, buf)
    _check(st, "sa_index_pattern_greedy")
    return buf.value.decode()


class IndexCache:
    """Shared index cache: full layers run the indexer into one buffer, shared
    layers read it (see sa_index_cache_* in sa.h).  The buffers are device
    tensors owned by this object (or passed in)."""

    def __init__(self, n_layers: int, B: int, Tq: int, k: int, pattern: str | None = None,
                 share_every: int = 4, device=None, idx_buf=None, count_buf=None):
        self._h = None
        self.idx_buf = idx_buf
        self.count_buf = count_buf
        if B > 0 and (idx_buf is None or count_buf is None):
            torch = _torch()
            self.idx_buf = torch.empty((B, Tq, k), dtype=torch.int32, device=device)
            self.count_buf = torch.empty((B, Tq), dtype=torch.int32, device=device)
        h = ctypes.c_void_p()
        pat = pattern.encode() if pattern is not None else None
        st = lib().sa_index_cache_create(n_layers, pat, share_every, B, Tq, k,
                                         _ptr(self.idx_buf), _ptr(self.count_buf), ctypes.byref(h))
        _check(st, "sa_index_cache_create")
        self._h = h
        self.n_layers, self.B, self.Tq, self.k = n_layers, B, Tq, k

    def close(self):
        if self._h is not None and self._h.value:
            lib().sa_index_cache_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def is_full(self, layer: int) -> int:
        return lib().sa_index_cache_is_full(self._h, layer)

    def owner(self, layer: int) -> int:
        return lib().sa_index_cache_owner(self._h, layer)

    def begin_step(self):
        _check(lib().sa_index_cache_begin_step(self._h), "sa_index_cache_begin_step")

    def mark_written(self, layer: int):
        _check(lib().sa_index_cache_mark_written(self._h, layer), "sa_index_cache_mark_written")

    def update(self, layer: int, q_idx, k_idx, Tk: int | None = None, q_pos0: int | None = None,
               kv_len=None, ws=None, stream=None):
        q3 = q_idx.unsqueeze(1) if q_idx.dim() == 2 else q_idx
        B, Tq, d = q3.shape
        Tk_max = k_idx.shape[1]
        Tk = Tk_max if Tk is None else Tk
        q_pos0 = Tk - Tq if q_pos0 is None else q_pos0
        need = lib().sa_index_score_topk_workspace(B, Tq, Tk_max, d, self.k)
        if ws is None:
            ws = workspace(need, q3.device, "index", stream)
        st = lib().sa_index_cache_update(self._h, layer, _ptr(q3), _ptr(k_idx), Tk, Tk_max, d, q_pos0,
                                         _ptr(kv_len), _ptr(ws), 0 if ws is None else ws.numel(),
                                         _stream(stream))
        _check(st, "sa_index_cache_update")

    def get(self, layer: int):
        """(idx_ptr, count_ptr, version) for `layer`; raises SAError on a stale read."""
        ip, cp, ver = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_uint64()
        st = lib().sa_index_cache_get(self._h, layer, ctypes.byref(ip), ctypes.byref(cp),
                                      ctypes.byref(ver))
        _check(st, "sa_index_cache_get")
        return ip.value, cp.value, ver.value

    def get_tensors(self, layer: int):
        """The index buffers for `layer` (checked against the C object)."""
        ip, cp, ver = self.get(layer)
        assert ip == self.idx_buf.data_ptr() and cp == self.count_buf.data_ptr()
        return self.idx_buf, self.count_buf, ver
