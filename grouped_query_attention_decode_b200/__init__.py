"""Python binding of libgqa: one grouped-query-attention decode step on B200.

This module only marshals arguments: it takes torch tensors (device memory the caller
allocated), passes their pointers, sizes and the current CUDA stream to the C ABI declared in
``include/gqa.h``, and turns error codes into exceptions.  Every step of the computation runs in
the library's CUDA kernels; there is no fallback.  If ``libgqa.so`` has not been built, importing
the binding's functions raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgqa.so")

DTYPE_F32 = 0
DTYPE_BF16 = 1
_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}

# status bits written by the kernels (include/gqa.h)
STATUS_APPEND_OVERFLOW = 1
STATUS_SEQLEN_RANGE = 2
STATUS_WAIT_TIMEOUT = 4
STATUS_INTERNAL = 8
STATUS_PAGE_RANGE = 16
STATUS_GROUP_RANGE = 32
STATUS_PAGE_REFS = 64
STATUS_POOL_FULL = 128
STATUS_INDEX_RANGE = 256

# C-ABI symbols declared in include/gqa.h
EXPORTED = ("gqa_kv_append", "gqa_decode_workspace_size", "gqa_decode", "gqa_status_string",
            "gqa_set_wait_timeout_ns", "gqa_profile_events", "gqa_decode_noalloc",
            "gqa_decode_window", "gqa_kv_append_paged", "gqa_decode_paged",
            "gqa_kv_append_multi", "gqa_decode_multi_workspace_size", "gqa_decode_multi",
            "gqa_kv_append_fp8", "gqa_kv_append_paged_fp8", "gqa_decode_fp8",
            "gqa_decode_paged_fp8", "gqa_kv_append_decode",
            "gqa_decode_shared_workspace_size", "gqa_decode_shared", "gqa_decode_shared_paged",
            "gqa_cross_attend_workspace_size", "gqa_cross_attend", "gqa_pages_workspace_size",
            "gqa_pages_fork", "gqa_pages_free", "gqa_pages_reserve", "gqa_pages_compact",
            "gqa_pages_copy")


class GQAError(RuntimeError):
    """A libgqa call returned a negative GQA_ERR_* code."""

    def __init__(self, code: int, msg: str):
        super().__init__(f"libgqa error {code}: {msg}")
        self.code = code


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgqa.so (once).  Raises OSError when it is missing: build it first with
    ``python -m grouped_query_attention_decode_b200.build``."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"{path} not found; build it with `python -m grouped_query_attention_decode_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i32p = ctypes.c_void_p, ctypes.c_void_p
    c_int, c_size = ctypes.c_int, ctypes.c_size_t
    lib.gqa_kv_append.argtypes = [vp, vp, vp, vp, i32p, c_int, c_int, c_int, c_int, c_int, i32p, vp]
    lib.gqa_kv_append.restype = c_int
    lib.gqa_decode_workspace_size.argtypes = [c_int, c_int, c_int, c_int, c_int]
    lib.gqa_decode_workspace_size.restype = c_size
    lib.gqa_decode.argtypes = [vp, vp, vp, i32p, c_int, c_int, c_int, c_int, c_int,
                               ctypes.c_float, c_int, vp, vp, c_size, i32p, vp]
    lib.gqa_decode.restype = c_int
    lib.gqa_kv_append_decode.argtypes = [vp, vp, vp, vp, vp, i32p, i32p, c_int, c_int, c_int,
                                         c_int, c_int, ctypes.c_float, c_int, vp, vp, c_size,
                                         i32p, vp]
    lib.gqa_kv_append_decode.restype = c_int
    lib.gqa_decode_window.argtypes = [vp, vp, vp, i32p, c_int, c_int, c_int, c_int, c_int, c_int,
                                      ctypes.c_float, c_int, vp, vp, c_size, i32p, vp]
    lib.gqa_decode_window.restype = c_int
    lib.gqa_kv_append_paged.argtypes = [vp, vp, vp, vp, i32p, c_int, i32p, c_int, c_int, c_int,
                                        c_int, c_int, c_int, i32p, vp]
    lib.gqa_kv_append_paged.restype = c_int
    lib.gqa_decode_paged.argtypes = [vp, vp, vp, i32p, c_int, i32p, c_int, c_int, c_int, c_int,
                                     c_int, c_int, ctypes.c_float, c_int, vp, vp, c_size, i32p, vp]
    lib.gqa_decode_paged.restype = c_int
    lib.gqa_kv_append_multi.argtypes = [vp, vp, vp, vp, i32p, c_int, c_int, c_int, c_int, c_int,
                                        c_int, i32p, vp]
    lib.gqa_kv_append_multi.restype = c_int
    lib.gqa_decode_multi_workspace_size.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int]
    lib.gqa_decode_multi_workspace_size.restype = c_size
    lib.gqa_decode_multi.argtypes = [vp, vp, vp, i32p, c_int, c_int, c_int, c_int, c_int, c_int,
                                     ctypes.c_float, c_int, vp, vp, c_size, i32p, vp]
    lib.gqa_decode_multi.restype = c_int
    lib.gqa_decode_noalloc.argtypes = [vp, vp, vp, i32p, c_int, c_int, c_int, c_int, c_int,
                                       ctypes.c_float, c_int, vp, i32p, vp]
    lib.gqa_decode_noalloc.restype = c_int
    fp = ctypes.POINTER(ctypes.c_float)
    lib.gqa_kv_append_fp8.argtypes = [vp, vp, c_int, vp, vp, vp, vp, i32p, c_int, c_int, c_int,
                                      c_int, i32p, vp]
    lib.gqa_kv_append_fp8.restype = c_int
    lib.gqa_kv_append_paged_fp8.argtypes = [vp, vp, c_int, vp, vp, vp, vp, i32p, c_int, i32p,
                                            c_int, c_int, c_int, c_int, c_int, i32p, vp]
    lib.gqa_kv_append_paged_fp8.restype = c_int
    lib.gqa_decode_fp8.argtypes = [vp, vp, vp, vp, vp, i32p, c_int, c_int, c_int, c_int, c_int,
                                   c_int, ctypes.c_float, vp, vp, ctypes.c_size_t, i32p, vp]
    lib.gqa_decode_fp8.restype = c_int
    lib.gqa_decode_paged_fp8.argtypes = [vp, vp, vp, vp, vp, i32p, c_int, i32p, c_int, c_int,
                                         c_int, c_int, c_int, c_int, ctypes.c_float, vp, vp,
                                         ctypes.c_size_t, i32p, vp]
    lib.gqa_decode_paged_fp8.restype = c_int
    c_float = ctypes.c_float
    lib.gqa_decode_shared_workspace_size.argtypes = [c_int] * 7
    lib.gqa_decode_shared_workspace_size.restype = c_size
    lib.gqa_decode_shared.argtypes = [vp, vp, vp, i32p, i32p, c_int, c_int, vp, vp, i32p, c_int, c_int,
                                      c_int, c_int, c_int, c_int, c_float, c_int, vp, vp, c_size,
                                      i32p, vp]
    lib.gqa_decode_shared.restype = c_int
    lib.gqa_decode_shared_paged.argtypes = [vp, vp, vp, i32p, c_int, i32p, i32p, i32p, c_int, c_int,
                                            c_int, c_int, c_int, c_int, c_int, c_int, c_float,
                                            c_int, vp, vp, c_size, i32p, vp]
    lib.gqa_decode_shared_paged.restype = c_int
    lib.gqa_cross_attend_workspace_size.argtypes = [c_int] * 6
    lib.gqa_cross_attend_workspace_size.restype = c_size
    lib.gqa_cross_attend.argtypes = [vp, vp, vp, i32p, i32p, c_int, c_int, c_int, c_int, c_int, c_int,
                                     c_float, c_int, vp, vp, c_size, i32p, vp]
    lib.gqa_cross_attend.restype = c_int
    lib.gqa_pages_workspace_size.argtypes = [c_int]
    lib.gqa_pages_workspace_size.restype = c_size
    lib.gqa_pages_fork.argtypes = [i32p, i32p, i32p, c_int, i32p, i32p, c_int, c_int, i32p, c_int,
                                   i32p, vp]
    lib.gqa_pages_fork.restype = c_int
    lib.gqa_pages_free.argtypes = [i32p, c_int, i32p, i32p, c_int, c_int, i32p, c_int, i32p, vp]
    lib.gqa_pages_free.restype = c_int
    lib.gqa_pages_reserve.argtypes = [i32p, i32p, c_int, c_int, c_int, c_int, i32p, c_int, i32p, vp,
                                      c_size, i32p, vp]
    lib.gqa_pages_reserve.restype = c_int
    lib.gqa_pages_compact.argtypes = [i32p, c_int, c_int, i32p, c_int, i32p, i32p, vp, c_size, i32p,
                                      vp]
    lib.gqa_pages_compact.restype = c_int
    lib.gqa_pages_copy.argtypes = [vp, vp, i32p, c_int, c_int, c_int, c_int, c_int, c_int, i32p, vp]
    lib.gqa_pages_copy.restype = c_int
    lib.gqa_status_string.argtypes = [c_int]
    lib.gqa_status_string.restype = ctypes.c_char_p
    lib.gqa_set_wait_timeout_ns.argtypes = [ctypes.c_ulonglong]
    lib.gqa_set_wait_timeout_ns.restype = c_int
    lib.gqa_profile_events.argtypes = [vp, vp]
    lib.gqa_profile_events.restype = c_int
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().gqa_status_string(int(code)).decode()


def _check(rc: int):
    if rc != 0:
        raise GQAError(rc, status_string(rc))


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("libgqa needs contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def kv_append(k_new, v_new, k_cache, v_cache, seq_lens, status=None, stream=None) -> None:
    """gqa_kv_append: k_cache[b, seq_lens[b]] = k_new[b] (and V), then seq_lens[b] += 1."""
    B, L_max, H_kv, d = k_cache.shape
    _check(load_library().gqa_kv_append(
        _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
        B, H_kv, d, L_max, _dtype(k_cache), _ptr(status), _stream(stream)))


def workspace_size(B: int, H_q: int, H_kv: int, d: int, dtype: torch.dtype) -> int:
    """Bytes of workspace gqa_decode needs on the current device."""
    return int(load_library().gqa_decode_workspace_size(B, H_q, H_kv, d, _DTYPES[dtype]))


def alloc_workspace(B: int, H_q: int, H_kv: int, d: int, dtype: torch.dtype, device=None):
    n = workspace_size(B, H_q, H_kv, d, dtype)
    if n == 0:
        raise GQAError(-9, "no usable sm_100 device is current, or invalid sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def decode(q, k_cache, v_cache, seq_lens, scale: float, out=None, workspace=None, status=None,
           stream=None) -> torch.Tensor:
    """gqa_decode: attention of one decode step.  Returns ``out`` [B, H_q, d] float32."""
    B, H_q, d = q.shape
    _, L_max, H_kv, _ = k_cache.shape
    if out is None:
        out = torch.empty((B, H_q, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(B, H_q, H_kv, d, k_cache.dtype, device=q.device)
    _check(load_library().gqa_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), B, H_q, H_kv, d, L_max,
        float(scale), _dtype(k_cache), _ptr(out), _ptr(workspace), workspace.numel(),
        _ptr(status), _stream(stream)))
    return out


def kv_append_decode(q, k_new, v_new, k_cache, v_cache, seq_lens, seq_lens_out, scale: float,
                     out=None, workspace=None, status=None, stream=None) -> torch.Tensor:
    """gqa_kv_append_decode: append k_new/v_new at row seq_lens[b] and attend the rows up to and
    including it, in one launch; the new lengths go to ``seq_lens_out`` (``seq_lens`` is only
    read).  Returns ``out`` [B, H_q, d] float32."""
    B, H_q, d = q.shape
    _, L_max, H_kv, _ = k_cache.shape
    if out is None:
        out = torch.empty((B, H_q, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(B, H_q, H_kv, d, k_cache.dtype, device=q.device)
    _check(load_library().gqa_kv_append_decode(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
        _ptr(seq_lens_out), B, H_q, H_kv, d, L_max, float(scale), _dtype(k_cache), _ptr(out),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)))
    return out


def decode_window(q, k_cache, v_cache, seq_lens, window: int, scale: float, out=None,
                  workspace=None, status=None, stream=None) -> torch.Tensor:
    """gqa_decode_window: each sequence attends only its last ``window`` cached rows."""
    B, H_q, d = q.shape
    _, L_max, H_kv, _ = k_cache.shape
    if out is None:
        out = torch.empty((B, H_q, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(B, H_q, H_kv, d, k_cache.dtype, device=q.device)
    _check(load_library().gqa_decode_window(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), B, H_q, H_kv, d, L_max,
        int(window), float(scale), _dtype(k_cache), _ptr(out), _ptr(workspace),
        workspace.numel(), _ptr(status), _stream(stream)))
    return out


def kv_append_paged(k_new, v_new, k_pool, v_pool, block_table, seq_lens, status=None,
                    stream=None) -> None:
    """gqa_kv_append_paged: pools [n_pages, page_size, H_kv, d], block_table [B, max_pages]."""
    n_pages, page_size, H_kv, d = k_pool.shape
    B, max_pages = block_table.shape
    _check(load_library().gqa_kv_append_paged(
        _ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), max_pages,
        _ptr(seq_lens), B, H_kv, d, page_size, n_pages, _dtype(k_pool), _ptr(status),
        _stream(stream)))


def decode_paged(q, k_pool, v_pool, block_table, seq_lens, scale: float, out=None,
                 workspace=None, status=None, stream=None) -> torch.Tensor:
    """gqa_decode_paged: the decode over a paged cache."""
    B, H_q, d = q.shape
    n_pages, page_size, H_kv, _ = k_pool.shape
    _, max_pages = block_table.shape
    if out is None:
        out = torch.empty((B, H_q, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(B, H_q, H_kv, d, k_pool.dtype, device=q.device)
    _check(load_library().gqa_decode_paged(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), max_pages, _ptr(seq_lens), B,
        H_q, H_kv, d, page_size, n_pages, float(scale), _dtype(k_pool), _ptr(out),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)))
    return out


def kv_append_multi(k_new, v_new, k_cache, v_cache, seq_lens, status=None, stream=None) -> None:
    """gqa_kv_append_multi: k_new, v_new [B, Q, H_kv, d] to rows seq_lens[b] .. + Q - 1."""
    B, L_max, H_kv, d = k_cache.shape
    Q = k_new.shape[1]
    _check(load_library().gqa_kv_append_multi(
        _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), B, Q, H_kv, d,
        L_max, _dtype(k_cache), _ptr(status), _stream(stream)))


def decode_multi(q, k_cache, v_cache, seq_lens, scale: float, out=None, workspace=None,
                 status=None, stream=None) -> torch.Tensor:
    """gqa_decode_multi: q [B, Q, H_q, d]; token j attends rows [0, n - Q + 1 + j)."""
    B, Q, H_q, d = q.shape
    _, L_max, H_kv, _ = k_cache.shape
    lib = load_library()
    if out is None:
        out = torch.empty((B, Q, H_q, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = int(lib.gqa_decode_multi_workspace_size(B, Q, H_q, H_kv, d, _DTYPES[k_cache.dtype]))
        if n == 0:
            raise GQAError(-9, "no usable sm_100 device is current, or invalid sizes")
        workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
    _check(lib.gqa_decode_multi(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), B, Q, H_q, H_kv, d, L_max,
        float(scale), _dtype(k_cache), _ptr(out), _ptr(workspace), workspace.numel(),
        _ptr(status), _stream(stream)))
    return out


def decode_noalloc(q, k_cache, v_cache, seq_lens, scale: float, out=None, status=None,
                   stream=None) -> torch.Tensor:
    """gqa_decode_noalloc: like ``decode`` but with the library's own fixed scratch array
    instead of a caller workspace (for callers that cannot allocate one).  Calls that may run
    at the same time on the GPU must not overlap: they share that array."""
    B, H_q, d = q.shape
    _, L_max, H_kv, _ = k_cache.shape
    if out is None:
        out = torch.empty((B, H_q, d), dtype=torch.float32, device=q.device)
    _check(load_library().gqa_decode_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), B, H_q, H_kv, d, L_max,
        float(scale), _dtype(k_cache), _ptr(out), _ptr(status), _stream(stream)))
    return out


def set_wait_timeout_ns(ns: int) -> None:
    """Time limit of the decode kernels' internal waits (0 restores the 2 s default)."""
    _check(load_library().gqa_set_wait_timeout_ns(int(ns)))


def profile_events(before_split=None, after_split=None) -> None:
    """Record these torch.cuda.Events around every later split-KV kernel (None, None stops)."""
    a = ctypes.c_void_p(before_split.cuda_event) if before_split is not None else None
    b = ctypes.c_void_p(after_split.cuda_event) if after_split is not None else None
    _check(load_library().gqa_profile_events(a, b))


# ------------------------------------------------------------------ FP8 (e4m3) cache
DTYPE_E4M3 = 2


def _codes(t: torch.Tensor) -> torch.Tensor:
    """An e4m3 cache as bytes: torch.uint8, or torch.float8_e4m3fn viewed as uint8."""
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise ValueError(f"an e4m3 cache must be uint8 or float8_e4m3fn, not {t.dtype}")
    return t


def _scales(t: torch.Tensor, H_kv: int) -> torch.Tensor:
    if t.dtype != torch.float32 or t.shape != (H_kv,):
        raise ValueError(f"scales must be float32 [{H_kv}]")
    return t


def alloc_workspace_fp8(B: int, H_q: int, H_kv: int, d: int, device=None):
    n = int(load_library().gqa_decode_workspace_size(B, H_q, H_kv, d, DTYPE_E4M3))
    if n == 0:
        raise GQAError(-9, "no usable sm_100 device is current, or invalid sizes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def kv_append_fp8(k_new, v_new, k_cache, v_cache, k_scale, v_scale, seq_lens, status=None,
                  stream=None) -> None:
    """gqa_kv_append_fp8: quantise k_new/v_new [B, H_kv, d] (bf16 or float32) to e4m3 codes of
    their head's scale and write them at row seq_lens[b]; then seq_lens[b] += 1."""
    kc, vc = _codes(k_cache), _codes(v_cache)
    B, L_max, H_kv, d = kc.shape
    _check(load_library().gqa_kv_append_fp8(
        _ptr(k_new), _ptr(v_new), _dtype(k_new), _ptr(kc), _ptr(vc),
        _ptr(_scales(k_scale, H_kv)), _ptr(_scales(v_scale, H_kv)), _ptr(seq_lens), B, H_kv, d,
        L_max, _ptr(status), _stream(stream)))


def kv_append_paged_fp8(k_new, v_new, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens,
                        status=None, stream=None) -> None:
    """gqa_kv_append_paged_fp8: the quantising append into e4m3 page pools."""
    kp, vp_ = _codes(k_pool), _codes(v_pool)
    n_pages, page_size, H_kv, d = kp.shape
    B, max_pages = block_table.shape
    _check(load_library().gqa_kv_append_paged_fp8(
        _ptr(k_new), _ptr(v_new), _dtype(k_new), _ptr(kp), _ptr(vp_),
        _ptr(_scales(k_scale, H_kv)), _ptr(_scales(v_scale, H_kv)), _ptr(block_table), max_pages,
        _ptr(seq_lens), B, H_kv, d, page_size, n_pages, _ptr(status), _stream(stream)))


def decode_fp8(q, k_cache, v_cache, k_scale, v_scale, seq_lens, scale: float, window: int = 0,
               out=None, workspace=None, status=None, stream=None) -> torch.Tensor:
    """gqa_decode_fp8: the decode over an e4m3 cache (window > 0: sliding window).  q is bf16
    [B, H_q, d]; returns out [B, H_q, d] float32."""
    kc, vc = _codes(k_cache), _codes(v_cache)
    B, H_q, d = q.shape
    _, L_max, H_kv, _ = kc.shape
    if q.dtype != torch.bfloat16:
        raise ValueError("q must be bfloat16 for an e4m3 cache")
    if out is None:
        out = torch.empty((B, H_q, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace_fp8(B, H_q, H_kv, d, device=q.device)
    _check(load_library().gqa_decode_fp8(
        _ptr(q), _ptr(kc), _ptr(vc), _ptr(_scales(k_scale, H_kv)), _ptr(_scales(v_scale, H_kv)),
        _ptr(seq_lens), B, H_q, H_kv, d, L_max, int(window), float(scale), _ptr(out),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)))
    return out


def decode_paged_fp8(q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, scale: float,
                     out=None, workspace=None, status=None, stream=None) -> torch.Tensor:
    """gqa_decode_paged_fp8: the decode over e4m3 page pools."""
    kp, vp_ = _codes(k_pool), _codes(v_pool)
    B, H_q, d = q.shape
    n_pages, page_size, H_kv, _ = kp.shape
    _, max_pages = block_table.shape
    if q.dtype != torch.bfloat16:
        raise ValueError("q must be bfloat16 for an e4m3 cache")
    if out is None:
        out = torch.empty((B, H_q, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace_fp8(B, H_q, H_kv, d, device=q.device)
    _check(load_library().gqa_decode_paged_fp8(
        _ptr(q), _ptr(kp), _ptr(vp_), _ptr(_scales(k_scale, H_kv)), _ptr(_scales(v_scale, H_kv)),
        _ptr(block_table), max_pages, _ptr(seq_lens), B, H_q, H_kv, d, page_size, n_pages,
        float(scale), _ptr(out), _ptr(workspace), workspace.numel(), _ptr(status),
        _stream(stream)))
    return out


# ------------------------------------------------------------------ rows that sequences share
# Small calls are bound by the host, so what follows makes few Python calls per argument.
def _tensors(status, first: torch.Tensor, *tensors) -> int:
    """The device number of ``first``; every tensor (None: absent) has to be dense and on it, and
    ``status`` hold the word that a kernel may write."""
    dev = first.get_device()
    if status is not None:
        if status.dtype is not torch.int32 or status.numel() < 1:
            raise ValueError(f"status must be torch.int32 of one element or more, not {status.dtype} {list(status.shape)}")
        tensors += (status,)
    if dev < 0:
        raise ValueError("libgqa needs CUDA tensors")
    if not first.is_contiguous():
        raise ValueError("libgqa needs contiguous tensors")
    for t in tensors:
        if t is not None:
            if t.get_device() != dev:
                raise ValueError(f"tensors on {first.device} and {t.device}")
            if not t.is_contiguous():
                raise ValueError("libgqa needs contiguous tensors")
    return dev


def _want(t: torch.Tensor, shape, dtype, name: str) -> None:
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _made(t: torch.Tensor, stream) -> torch.Tensor:
    """A tensor that the binding allocated (on its device's current stream) for a call on
    ``stream``: its memory's earlier users come first, and it is not given away before the call is
    done."""
    if stream is not None:
        current = torch.cuda.current_stream(t.device)
        if stream != current:
            stream.wait_stream(current)
            t.record_stream(stream)
    return t


def _run(dev: int, fn, *args) -> None:
    """fn(*args) with the tensors' device as the current one, which is the library's."""
    if torch.cuda.current_device() == dev:
        _check(fn(*args))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args))


@functools.lru_cache(maxsize=1024)
def _bytes_on(dev: int, fn: str, *sizes) -> int:
    with torch.cuda.device(dev):
        n = int(getattr(load_library(), fn)(*sizes))
    if n == 0:
        raise GQAError(-9, "no usable sm_100 device is current, or invalid sizes")
    return n


def _workspace(q: torch.Tensor, dev: int, workspace, stream, fn: str, *sizes) -> torch.Tensor:
    if workspace is None:
        workspace = _made(torch.empty(_bytes_on(dev, fn, *sizes), dtype=torch.uint8, device=q.device), stream)
    return workspace


def _addr(t):
    return None if t is None else t.data_ptr()


def shared_workspace_size(B: int, Q: int, P: int, H_q: int, H_kv: int, d: int, dtype: torch.dtype) -> int:
    """Bytes of workspace decode_shared and decode_shared_paged need on the current device."""
    return int(load_library().gqa_decode_shared_workspace_size(B, Q, P, H_q, H_kv, d, _DTYPES[dtype]))


def decode_shared(q, k_prefix, v_prefix, prefix_lens, group_start, k_cache, v_cache, seq_lens,
                  scale: float, out=None, workspace=None, status=None, stream=None) -> torch.Tensor:
    """gqa_decode_shared: the sequences [group_start[g], group_start[g+1]) attend the prefix_lens[g]
    rows of k_prefix[g], read once for all of them, and then their own seq_lens[b] rows.  q is
    [B, H_q, d], or [B, Q, H_q, d] for Q query tokens per sequence; returns out of q's shape,
    float32."""
    lib = _lib or load_library()
    shape, dtype = q.shape, q.dtype
    B, Q, H_q, d = shape if len(shape) == 4 else (shape[0], 1, *shape[1:])
    P, L_prefix, H_kv, _ = k_prefix.shape
    L_max = k_cache.shape[1]
    code = _dtype(q)
    _want(k_prefix, (P, L_prefix, H_kv, d), dtype, "k_prefix")
    _want(v_prefix, (P, L_prefix, H_kv, d), dtype, "v_prefix")
    _want(k_cache, (B, L_max, H_kv, d), dtype, "k_cache")
    _want(v_cache, (B, L_max, H_kv, d), dtype, "v_cache")
    _want(prefix_lens, (P,), torch.int32, "prefix_lens")
    _want(group_start, (P + 1,), torch.int32, "group_start")
    _want(seq_lens, (B,), torch.int32, "seq_lens")
    dev = _tensors(status, q, k_prefix, v_prefix, prefix_lens, group_start, k_cache, v_cache, seq_lens, out, workspace)
    if out is None:
        out = _made(torch.empty_like(q, dtype=torch.float32), stream)
    else:
        _want(out, shape, torch.float32, "out")
    workspace = _workspace(q, dev, workspace, stream, "gqa_decode_shared_workspace_size", B, Q, P, H_q, H_kv, d, code)
    _run(dev, lib.gqa_decode_shared, q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), prefix_lens.data_ptr(),
         group_start.data_ptr(), P, L_prefix, k_cache.data_ptr(), v_cache.data_ptr(), seq_lens.data_ptr(), B, Q, H_q, H_kv, d,
         L_max, scale, code, out.data_ptr(), workspace.data_ptr(), workspace.numel(), _addr(status), _raw_stream(stream, dev))
    return out


def decode_shared_paged(q, k_pool, v_pool, block_table, seq_lens, group_start, shared_rows,
                        scale: float, out=None, workspace=None, status=None, stream=None) -> torch.Tensor:
    """gqa_decode_shared_paged: decode_paged for sequences [group_start[g], group_start[g+1]) whose
    first shared_rows[g] rows lie in the same pages, which are read once for all of them.  q is
    [B, H_q, d] or [B, Q, H_q, d]; returns out of q's shape, float32."""
    lib = _lib or load_library()
    shape, dtype = q.shape, q.dtype
    B, Q, H_q, d = shape if len(shape) == 4 else (shape[0], 1, *shape[1:])
    n_pages, page_size, H_kv, _ = k_pool.shape
    max_pages = block_table.shape[1]
    P = shared_rows.shape[0]
    code = _dtype(q)
    _want(k_pool, (n_pages, page_size, H_kv, d), dtype, "k_pool")
    _want(v_pool, (n_pages, page_size, H_kv, d), dtype, "v_pool")
    _want(block_table, (B, max_pages), torch.int32, "block_table")
    _want(seq_lens, (B,), torch.int32, "seq_lens")
    _want(group_start, (P + 1,), torch.int32, "group_start")
    _want(shared_rows, (P,), torch.int32, "shared_rows")
    dev = _tensors(status, q, k_pool, v_pool, block_table, seq_lens, group_start, shared_rows, out, workspace)
    if out is None:
        out = _made(torch.empty_like(q, dtype=torch.float32), stream)
    else:
        _want(out, shape, torch.float32, "out")
    workspace = _workspace(q, dev, workspace, stream, "gqa_decode_shared_workspace_size", B, Q, P, H_q, H_kv, d, code)
    _run(dev, lib.gqa_decode_shared_paged, q.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), block_table.data_ptr(), max_pages,
         seq_lens.data_ptr(), group_start.data_ptr(), shared_rows.data_ptr(), P, B, Q, H_q, H_kv, d, page_size, n_pages, scale,
         code, out.data_ptr(), workspace.data_ptr(), workspace.numel(), _addr(status), _raw_stream(stream, dev))
    return out


# ------------------------------------------------------------------ cross attention
def cross_workspace_size(E: int, N: int, H_q: int, H_kv: int, d: int, dtype: torch.dtype) -> int:
    """Bytes of workspace cross_attend needs on the current device."""
    return int(load_library().gqa_cross_attend_workspace_size(E, N, H_q, H_kv, d, _DTYPES[dtype]))


def cross_attend(q, k_enc, v_enc, enc_lens, q_start, scale: float, out=None, workspace=None,
                 status=None, stream=None) -> torch.Tensor:
    """gqa_cross_attend: tokens [q_start[e], q_start[e+1]) of q [N, H_q, d] attend the states
    [0, enc_lens[e]) of k_enc, v_enc [E, S_max, H_kv, d].  Returns out [N, H_q, d] float32; tokens
    before q_start[0] or from q_start[E] on are left as they were in ``out``."""
    lib = _lib or load_library()
    shape, dtype = q.shape, q.dtype
    N, H_q, d = shape
    E, S_max, H_kv, _ = k_enc.shape
    code = _dtype(q)
    _want(k_enc, (E, S_max, H_kv, d), dtype, "k_enc")
    _want(v_enc, (E, S_max, H_kv, d), dtype, "v_enc")
    _want(enc_lens, (E,), torch.int32, "enc_lens")
    _want(q_start, (E + 1,), torch.int32, "q_start")
    dev = _tensors(status, q, k_enc, v_enc, enc_lens, q_start, out, workspace)
    if out is None:
        out = _made(torch.empty_like(q, dtype=torch.float32), stream)
    else:
        _want(out, shape, torch.float32, "out")
    workspace = _workspace(q, dev, workspace, stream, "gqa_cross_attend_workspace_size", E, N, H_q, H_kv, d, code)
    _run(dev, lib.gqa_cross_attend, q.data_ptr(), k_enc.data_ptr(), v_enc.data_ptr(), enc_lens.data_ptr(), q_start.data_ptr(), E, N,
         H_q, H_kv, d, S_max, scale, code, out.data_ptr(), workspace.data_ptr(), workspace.numel(), _addr(status),
         _raw_stream(stream, dev))
    return out


# ------------------------------------------------------------------ pages that sequences share
def pages_fork(parents, table_in, lens_in, table_out, lens_out, ref_counts, status=None, stream=None) -> None:
    """gqa_pages_fork: sequence i of (table_out, lens_out) becomes a copy of sequence parents[i] of
    (table_in, lens_in), -1: empty; ref_counts [n_pages] follows."""
    lib = _lib or load_library()
    (B_in, max_pages), B_out = table_in.shape, table_out.shape[0]
    n_pages = ref_counts.shape[0]
    _want(table_in, (B_in, max_pages), torch.int32, "table_in")
    _want(table_out, (B_out, max_pages), torch.int32, "table_out")
    _want(lens_in, (B_in,), torch.int32, "lens_in")
    _want(lens_out, (B_out,), torch.int32, "lens_out")
    _want(parents, (B_out,), torch.int32, "parents")
    _want(ref_counts, (n_pages,), torch.int32, "ref_counts")
    dev = _tensors(status, table_in, parents, lens_in, table_out, lens_out, ref_counts)
    _run(dev, lib.gqa_pages_fork, parents.data_ptr(), table_in.data_ptr(), lens_in.data_ptr(), B_in, table_out.data_ptr(),
         lens_out.data_ptr(), B_out, max_pages, ref_counts.data_ptr(), n_pages, _addr(status), _raw_stream(stream, dev))


def pages_free(seqs, block_table, seq_lens, ref_counts, status=None, stream=None) -> None:
    """gqa_pages_free: empty the sequences listed in ``seqs`` (int32 [n]; none: nothing is done)."""
    lib = _lib or load_library()
    B, max_pages = block_table.shape
    n, n_pages = seqs.shape[0], ref_counts.shape[0]
    _want(seqs, (n,), torch.int32, "seqs")
    _want(block_table, (B, max_pages), torch.int32, "block_table")
    _want(seq_lens, (B,), torch.int32, "seq_lens")
    _want(ref_counts, (n_pages,), torch.int32, "ref_counts")
    dev = _tensors(status, block_table, seqs, seq_lens, ref_counts)
    if n == 0:
        return
    _run(dev, lib.gqa_pages_free, seqs.data_ptr(), n, block_table.data_ptr(), seq_lens.data_ptr(), B, max_pages,
         ref_counts.data_ptr(), n_pages, _addr(status), _raw_stream(stream, dev))


def pages_reserve(block_table, seq_lens, ref_counts, rows: int, page_size: int, copies=None,
                  workspace=None, status=None, stream=None) -> torch.Tensor:
    """gqa_pages_reserve: every sequence gets pages of its own for its next ``rows`` rows.  Returns
    copies [B, 2] (old page, new page; -1: none): run pages_copy on them in every layer before the
    next change, when the pool ran out (STATUS_POOL_FULL) too."""
    lib = _lib or load_library()
    B, max_pages = block_table.shape
    n_pages = ref_counts.shape[0]
    _want(block_table, (B, max_pages), torch.int32, "block_table")
    _want(seq_lens, (B,), torch.int32, "seq_lens")
    _want(ref_counts, (n_pages,), torch.int32, "ref_counts")
    dev = _tensors(status, block_table, seq_lens, ref_counts, copies, workspace)
    if copies is None:
        copies = _made(torch.empty((B, 2), dtype=torch.int32, device=block_table.device), stream)
    else:
        _want(copies, (B, 2), torch.int32, "copies")
    workspace = _workspace(block_table, dev, workspace, stream, "gqa_pages_workspace_size", n_pages)
    _run(dev, lib.gqa_pages_reserve, block_table.data_ptr(), seq_lens.data_ptr(), B, max_pages, page_size, rows,
         ref_counts.data_ptr(), n_pages, copies.data_ptr(), workspace.data_ptr(), workspace.numel(), _addr(status),
         _raw_stream(stream, dev))
    return copies


def pages_compact(block_table, ref_counts, copies=None, n_live=None, workspace=None, status=None,
                  stream=None):
    """gqa_pages_compact: the pages in use take the lowest numbers.  Returns (copies
    [max(1, n_pages // 2), 2], n_live [1]); run pages_copy on the copies."""
    lib = _lib or load_library()
    B, max_pages = block_table.shape
    n_pages = ref_counts.shape[0]
    _want(block_table, (B, max_pages), torch.int32, "block_table")
    _want(ref_counts, (n_pages,), torch.int32, "ref_counts")
    dev = _tensors(status, block_table, ref_counts, copies, n_live, workspace)
    most = max(1, n_pages // 2)
    if copies is None:
        copies = _made(torch.empty((most, 2), dtype=torch.int32, device=block_table.device), stream)
    else:
        _want(copies, (most, 2), torch.int32, "copies")
    if n_live is None:
        n_live = _made(torch.empty(1, dtype=torch.int32, device=block_table.device), stream)
    else:
        _want(n_live, (1,), torch.int32, "n_live")
    workspace = _workspace(block_table, dev, workspace, stream, "gqa_pages_workspace_size", n_pages)
    _run(dev, lib.gqa_pages_compact, block_table.data_ptr(), B, max_pages, ref_counts.data_ptr(), n_pages, copies.data_ptr(),
         n_live.data_ptr(), workspace.data_ptr(), workspace.numel(), _addr(status), _raw_stream(stream, dev))
    return copies, n_live


def pages_copy(k_pool, v_pool, copies, status=None, stream=None) -> None:
    """gqa_pages_copy: carry out ``copies`` [n, 2] (from, to) in the pools of one layer,
    [n_pages, page_size, H_kv, d] of bfloat16, float32 or e4m3 codes; no copies: nothing is done."""
    lib = _lib or load_library()
    if k_pool.dtype in _DTYPES:
        code = _DTYPES[k_pool.dtype]
    else:
        k_pool, v_pool, code = _codes(k_pool), _codes(v_pool), DTYPE_E4M3
    n_pages, page_size, H_kv, d = k_pool.shape
    n = copies.shape[0]
    _want(v_pool, k_pool.shape, k_pool.dtype, "v_pool")
    _want(copies, (n, 2), torch.int32, "copies")
    dev = _tensors(status, k_pool, v_pool, copies)
    if n == 0:
        return
    _run(dev, lib.gqa_pages_copy, k_pool.data_ptr(), v_pool.data_ptr(), copies.data_ptr(), n, page_size, n_pages, H_kv, d, code,
         _addr(status), _raw_stream(stream, dev))
