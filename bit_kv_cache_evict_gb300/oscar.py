"""Thin ctypes binding of liboscar (include/oscar.h), same call names.

Argument marshalling only: every step of the hot path runs in the CUDA
kernels of liboscar.so.  There is no CPU fallback: if the library is missing
or cannot be loaded, every call raises.
"""
from __future__ import annotations

import array
import ctypes
import os
import re

import numpy as np

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "liboscar.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "oscar.h")

OSCAR_OK, OSCAR_ERR_INVALID_ARG, OSCAR_ERR_UNSUPPORTED, OSCAR_ERR_OUT_OF_PAGES, OSCAR_ERR_WORKSPACE, \
    OSCAR_ERR_CUDA = range(6)
OSCAR_STATUS_BAD_PAGE, OSCAR_STATUS_BAD_POS, OSCAR_STATUS_TIMEOUT = 1, 2, 4
BLOCK_BYTES = 6144


class OscarError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


class oscar_shape(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("quant_group", ctypes.c_int32), ("sink", ctypes.c_int32),
                ("recent", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32)]


def make_shape(num_q_heads: int, num_kv_heads: int, head_dim: int = 128, quant_group: int = 32, sink: int = 64,
               recent: int = 256, page_size: int = 64) -> oscar_shape:
    return oscar_shape(head_dim, quant_group, sink, recent, page_size, num_q_heads, num_kv_heads)


_LIB = None
_P = ctypes.c_void_p


def lib() -> ctypes.CDLL:
    """Load liboscar.so (built in-tree by ``build.build()``); raise if absent."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"liboscar.so not built ({LIB_PATH}); run bit_kv_cache_evict_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        S = ctypes.POINTER(oscar_shape)
        L.oscar_block_bytes.restype = ctypes.c_size_t
        L.oscar_block_bytes.argtypes = [S]
        L.oscar_status_string.restype = ctypes.c_char_p
        L.oscar_status_string.argtypes = [ctypes.c_int]
        L.oscar_last_cuda_error.restype = ctypes.c_int
        L.oscar_pool_layout.restype = ctypes.c_int
        L.oscar_pool_layout.argtypes = [S, ctypes.c_int32, _P, _P, ctypes.c_int32, ctypes.c_uint64, ctypes.c_int32,
                                        _P, _P, _P]
        I32, PP = ctypes.c_int32, ctypes.POINTER(ctypes.c_void_p)
        L.oscar_pages_create.restype = ctypes.c_int
        L.oscar_pages_create.argtypes = [I32, PP]
        L.oscar_pages_destroy.restype = None
        L.oscar_pages_destroy.argtypes = [_P]
        for fn in ("oscar_pages_alloc", "oscar_pages_retain", "oscar_pages_release"):
            getattr(L, fn).restype = ctypes.c_int
            getattr(L, fn).argtypes = [_P, I32, _P]
        L.oscar_pages_refcount.restype = I32
        L.oscar_pages_refcount.argtypes = [_P, I32]
        L.oscar_pages_free_count.restype = I32
        L.oscar_pages_free_count.argtypes = [_P]
        L.oscar_pages_prepare_write.restype = ctypes.c_int
        L.oscar_pages_prepare_write.argtypes = [_P, I32, _P, _P, _P, I32, I32, _P, _P, _P]
        L.oscar_pages_copy.restype = ctypes.c_int
        L.oscar_pages_copy.argtypes = [S, I32, _P, _P, _P, _P, I32, _P]
        L.oscar_radix_create.restype = ctypes.c_int
        L.oscar_radix_create.argtypes = [_P, PP]
        L.oscar_radix_destroy.restype = None
        L.oscar_radix_destroy.argtypes = [_P]
        L.oscar_radix_insert.restype = ctypes.c_int
        L.oscar_radix_insert.argtypes = [_P, _P, I32, _P, I32]
        L.oscar_radix_match.restype = ctypes.c_int
        L.oscar_radix_match.argtypes = [_P, _P, I32, I32, _P, _P]
        L.oscar_radix_evict.restype = ctypes.c_int
        L.oscar_radix_evict.argtypes = [_P, I32, _P]
        L.oscar_radix_cached_pages.restype = I32
        L.oscar_radix_cached_pages.argtypes = [_P]
        L.oscar_evict_quantize.restype = ctypes.c_int
        L.oscar_evict_quantize.argtypes = [S, ctypes.c_int32, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P, _P, _P,
                                           ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P]
        L.oscar_decode_attn.restype = ctypes.c_int
        L.oscar_decode_attn.argtypes = [S, ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, _P,
                                        _P, ctypes.c_float, _P, _P, ctypes.POINTER(ctypes.c_size_t), _P, _P]
        L.oscar_decode_attn_noalloc.restype = ctypes.c_int
        L.oscar_decode_attn_noalloc.argtypes = [S, ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.c_int32,
                                                ctypes.c_int32, _P, _P, ctypes.c_float, _P, _P, _P]
        L.oscar_time_next_int2.restype = None
        L.oscar_time_next_int2.argtypes = [_P, _P]
        L.oscar_evict_quantize_codebook.restype = ctypes.c_int
        L.oscar_evict_quantize_codebook.argtypes = [S, ctypes.c_int32, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P,
                                                    _P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P,
                                                    _P]
        L.oscar_decode_attn_codebook.restype = ctypes.c_int
        L.oscar_decode_attn_codebook.argtypes = [S, ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.c_int32,
                                                 ctypes.c_int32, _P, _P, _P, ctypes.c_float, _P, _P,
                                                 ctypes.POINTER(ctypes.c_size_t), _P, _P]
        L.oscar_evict_quantize_boost.restype = ctypes.c_int
        L.oscar_evict_quantize_boost.argtypes = [S, ctypes.c_int32, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P,
                                                 _P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P]
        L.oscar_decode_attn_boost.restype = ctypes.c_int
        L.oscar_decode_attn_boost.argtypes = [S, ctypes.c_int32, _P, _P, _P, _P, _P, _P, ctypes.c_int32,
                                              ctypes.c_int32, _P, _P, ctypes.c_float, _P, _P,
                                              ctypes.POINTER(ctypes.c_size_t), _P, _P]
        L.oscar_block_bytes_int4.restype = ctypes.c_size_t
        L.oscar_block_bytes_int4.argtypes = [S]
        L.oscar_evict_quantize_int4.restype = ctypes.c_int
        L.oscar_evict_quantize_int4.argtypes = L.oscar_evict_quantize.argtypes
        L.oscar_decode_attn_int4.restype = ctypes.c_int
        L.oscar_decode_attn_int4.argtypes = [S, I32, _P, _P, _P, _P, _P, I32, I32, _P, _P, ctypes.c_float, _P, I32, _P,
                                             ctypes.POINTER(ctypes.c_size_t), _P, _P]
        L.oscar_history_read.restype = ctypes.c_int
        L.oscar_history_read.argtypes = [S, I32, I32, _P, _P, _P, _P, I32, I32, I32, _P, I32, _P, _P]
        L.oscar_history_gather.restype = ctypes.c_int
        L.oscar_history_gather.argtypes = [S, I32, I32, _P, _P, _P, I32, _P, I32, _P, I32, _P, I32, _P, _P]
        L.oscar_pages_copy_device.restype = ctypes.c_int
        L.oscar_pages_copy_device.argtypes = [ctypes.c_size_t, I32, _P, _P, _P, I32, I32, _P, _P]
        F32 = ctypes.c_float
        L.oscar_decode_attn_weights.restype = ctypes.c_int
        L.oscar_decode_attn_weights.argtypes = [S, I32, I32, _P, _P, _P, _P, _P, I32, I32, _P, _P, F32, _P, I32, _P, I32, _P,
                                                F32, _P, ctypes.POINTER(ctypes.c_size_t), _P, _P]
        L.oscar_decode_attn_shared.restype = ctypes.c_int
        L.oscar_decode_attn_shared.argtypes = [S, I32, I32, _P, _P, _P, _P, _P, I32, I32, _P, _P, I32, _P, I32, _P, F32, _P, I32, _P,
                                               ctypes.POINTER(ctypes.c_size_t), _P, _P]
        L.oscar_history_select.restype = ctypes.c_int
        L.oscar_history_select.argtypes = [I32, _P, I32, _P, _P, I32, _P, I32, _P, _P, I32, _P, _P]
        L.oscar_calibrate_codebook.restype = ctypes.c_int
        L.oscar_calibrate_codebook.argtypes = [S, ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.POINTER(ctypes.c_size_t),
                                               _P]
        L.oscar_calibrate_clip.restype = ctypes.c_int
        L.oscar_calibrate_clip.argtypes = [S, ctypes.c_int32, _P, _P, _P, ctypes.c_int32, _P, _P, _P,
                                           ctypes.POINTER(ctypes.c_size_t), _P]
        L.oscar_calibrate_rotation.restype = ctypes.c_int
        L.oscar_calibrate_rotation.argtypes = [S, ctypes.c_int32, _P, ctypes.c_int32, _P, ctypes.c_float, _P, _P,
                                               _P, ctypes.POINTER(ctypes.c_size_t), _P, _P]
        _LIB = L
    return _LIB


def declared_functions() -> list[str]:
    """Entry points declared in include/oscar.h."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:[\w\s\*]+?)\b(oscar_\w+)\s*\(", text, re.M)))


def _check(fn: str, st: int) -> None:
    if st != OSCAR_OK:
        msg = lib().oscar_status_string(st).decode()
        if st == OSCAR_ERR_CUDA:
            msg += f" (cudaError {lib().oscar_last_cuda_error()})"
        raise OscarError(fn, st, msg)


def _dptr(t, what: str, dtype=None, align: int = 1):
    """Device pointer of a CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what}: expected a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def block_bytes(shape: oscar_shape) -> int:
    return int(lib().oscar_block_bytes(ctypes.byref(shape)))


def oscar_pool_layout(shape: oscar_shape, hist_capacity, prefix_group=None, shared_hist_tokens: int = 0,
                      perm_seed: int = 0, max_pages: int | None = None):
    """Host page-table layout.  Returns (page_table int32 [B][max_pages],
    num_pages, pool_bytes)."""
    cap = np.ascontiguousarray(hist_capacity, np.int32)
    B = cap.shape[0]
    if max_pages is None:
        max_pages = max(1, int((int(cap.max(initial=0)) + shape.page_size - 1) // shape.page_size))
    pg = None if prefix_group is None else np.ascontiguousarray(prefix_group, np.int32)
    table = np.zeros((B, max_pages), np.int32)
    n = ctypes.c_int32(0)
    nbytes = ctypes.c_uint64(0)
    st = lib().oscar_pool_layout(ctypes.byref(shape), B, cap.ctypes.data_as(_P),
                                 None if pg is None else pg.ctypes.data_as(_P), shared_hist_tokens,
                                 ctypes.c_uint64(perm_seed), max_pages, table.ctypes.data_as(_P), ctypes.byref(n),
                                 ctypes.byref(nbytes))
    _check("oscar_pool_layout", st)
    return table, int(n.value), int(nbytes.value)


def oscar_evict_quantize(shape: oscar_shape, src_kv, dst_seq, dst_pos, U, clip, pool, page_table, batch: int,
                         max_pages: int, num_pages: int, src_row=None, new_kv=None, dev_status=None,
                         stream=None) -> None:
    """Fused rotate/clip/quantise/pack of dst_seq.numel() token rows into the
    pool (see include/oscar.h).  src_kv: bf16 [rows][Hk][2][d]."""
    import torch
    n_tok = int(dst_seq.numel())
    st = lib().oscar_evict_quantize(
        ctypes.byref(shape), n_tok, _dptr(src_kv, "src_kv", torch.bfloat16), int(src_kv.shape[0]),
        _dptr(src_row, "src_row", torch.int32), _dptr(dst_seq, "dst_seq", torch.int32),
        _dptr(dst_pos, "dst_pos", torch.int32), _dptr(new_kv, "new_kv", torch.bfloat16),
        _dptr(U, "U", torch.float32), _dptr(clip, "clip", torch.float32), _dptr(pool, "pool", torch.uint8),
        _dptr(page_table, "page_table", torch.int32), batch, max_pages, num_pages,
        _dptr(dev_status, "dev_status", torch.int32), _stream_ptr(stream))
    _check("oscar_evict_quantize", st)


def oscar_time_next_int2(ev_start, ev_stop) -> None:
    """Measurement hook: the next oscar_decode_attn on this thread records the
    two (already recorded once, timing-enabled) torch.cuda.Event objects
    around its INT2 split-K kernel."""
    lib().oscar_time_next_int2(ctypes.c_void_p(ev_start.cuda_event), ctypes.c_void_p(ev_stop.cuda_event))


def oscar_decode_workspace_bytes(shape: oscar_shape, batch: int, max_pages: int) -> int:
    ws = ctypes.c_size_t(0)
    st = lib().oscar_decode_attn(ctypes.byref(shape), batch, None, None, None, None, None, max_pages, 0, None,
                                 None, ctypes.c_float(1.0), None, None, ctypes.byref(ws), None, None)
    _check("oscar_decode_attn", st)
    return int(ws.value)


def oscar_decode_attn(shape: oscar_shape, q, bf16_kv, bf16_len, pool, page_table, max_pages: int, num_pages: int,
                      hist_len, U, sm_scale: float, out, workspace, dev_status=None, stream=None) -> None:
    """Decode attention over sink + INT2 history + recent (see
    include/oscar.h).  ``workspace``: CUDA uint8 tensor of at least
    oscar_decode_workspace_bytes(shape, batch, max_pages) bytes."""
    import torch
    B = int(q.shape[0])
    ws = ctypes.c_size_t(int(workspace.numel()))
    st = lib().oscar_decode_attn(
        ctypes.byref(shape), B, _dptr(q, "q", torch.bfloat16), _dptr(bf16_kv, "bf16_kv", torch.bfloat16),
        _dptr(bf16_len, "bf16_len", torch.int32), _dptr(pool, "pool", torch.uint8),
        _dptr(page_table, "page_table", torch.int32), max_pages, num_pages, _dptr(hist_len, "hist_len", torch.int32),
        _dptr(U, "U", torch.float32), ctypes.c_float(sm_scale), _dptr(out, "out", torch.float32),
        _dptr(workspace, "workspace", torch.uint8), ctypes.byref(ws), _dptr(dev_status, "dev_status", torch.int32),
        _stream_ptr(stream))
    _check("oscar_decode_attn", st)


NOALLOC_SCRATCH_BYTES = 64 << 20


def oscar_decode_attn_noalloc(shape: oscar_shape, q, bf16_kv, bf16_len, pool, page_table, max_pages: int,
                              num_pages: int, hist_len, U, sm_scale: float, out, dev_status=None,
                              stream=None) -> None:
    """oscar_decode_attn for callers that cannot allocate device memory: the
    scratch is the library's fixed 64 MiB device array (see include/oscar.h
    for the limits, the first-call set-up and why overlapping calls race)."""
    import torch
    B = int(q.shape[0])
    st = lib().oscar_decode_attn_noalloc(
        ctypes.byref(shape), B, _dptr(q, "q", torch.bfloat16), _dptr(bf16_kv, "bf16_kv", torch.bfloat16),
        _dptr(bf16_len, "bf16_len", torch.int32), _dptr(pool, "pool", torch.uint8),
        _dptr(page_table, "page_table", torch.int32), max_pages, num_pages, _dptr(hist_len, "hist_len", torch.int32),
        _dptr(U, "U", torch.float32), ctypes.c_float(sm_scale), _dptr(out, "out", torch.float32),
        _dptr(dev_status, "dev_status", torch.int32), _stream_ptr(stream))
    _check("oscar_decode_attn_noalloc", st)


def oscar_calibrate_workspace_bytes(shape: oscar_shape, n_q: int) -> int:
    ws = ctypes.c_size_t(0)
    st = lib().oscar_calibrate_rotation(ctypes.byref(shape), n_q, None, 1, None, ctypes.c_float(1.0), None, None,
                                        None, ctypes.byref(ws), None, None)
    _check("oscar_calibrate_rotation", st)
    return int(ws.value)


def oscar_calibrate_rotation(shape: oscar_shape, q, kv, sm_scale: float, U, workspace, eigvals=None,
                             dev_status=None, stream=None) -> None:
    """Offline calibration of U from calibration queries q [n_q][Hq][d] and
    tokens kv [n_t][Hk][2][d] (bf16 CUDA tensors) into U [Hk][2][d][d]
    (fp32); see include/oscar.h."""
    import torch
    ws = ctypes.c_size_t(int(workspace.numel()))
    st = lib().oscar_calibrate_rotation(
        ctypes.byref(shape), int(q.shape[0]), _dptr(q, "q", torch.bfloat16), int(kv.shape[0]),
        _dptr(kv, "kv", torch.bfloat16), ctypes.c_float(sm_scale), _dptr(U, "U", torch.float32),
        _dptr(eigvals, "eigvals", torch.float32), _dptr(workspace, "workspace", torch.uint8), ctypes.byref(ws),
        _dptr(dev_status, "dev_status", torch.int32), _stream_ptr(stream))
    _check("oscar_calibrate_rotation", st)


def oscar_calibrate_clip_workspace_bytes(shape: oscar_shape, n_t: int = 1, n_grid: int = 1) -> int:
    need = ctypes.c_size_t(0)
    st = lib().oscar_calibrate_clip(ctypes.byref(shape), n_t, None, None, None, n_grid, None, None, None,
                                    ctypes.byref(need), None)
    _check("oscar_calibrate_clip", st)
    return int(need.value)


def oscar_calibrate_clip(shape: oscar_shape, kv, U, grid, clip, workspace=None, mse=None, stream=None) -> None:
    """Offline clip-ratio search: for each (KV head, K/V) the ratio of grid
    (fp32 CUDA tensor) with the least reconstruction error of the rotated
    calibration tokens kv [n_t][Hk][2][d] under the eviction's quantiser;
    see include/oscar.h.  ``workspace`` defaults to a fresh tensor."""
    import torch
    n_grid = int(grid.numel())
    if workspace is None:
        workspace = torch.zeros(oscar_calibrate_clip_workspace_bytes(shape, int(kv.shape[0]), n_grid),
                                dtype=torch.uint8, device=kv.device)
    ws = ctypes.c_size_t(int(workspace.numel()))
    st = lib().oscar_calibrate_clip(
        ctypes.byref(shape), int(kv.shape[0]), _dptr(kv, "kv", torch.bfloat16), _dptr(U, "U", torch.float32),
        _dptr(grid, "grid", torch.float32), n_grid, _dptr(clip, "clip", torch.float32),
        _dptr(mse, "mse", torch.float32), _dptr(workspace, "workspace", torch.uint8), ctypes.byref(ws),
        _stream_ptr(stream))
    _check("oscar_calibrate_clip", st)


def oscar_evict_quantize_codebook(shape: oscar_shape, src_kv, dst_seq, dst_pos, U, clip, codebook, pool, page_table,
                                  batch: int, max_pages: int, num_pages: int, src_row=None, new_kv=None,
                                  dev_status=None, stream=None) -> None:
    """oscar_evict_quantize with the Lloyd-Max levels {0, a, 3 - a, 3}
    (codebook: fp32 [Hk][2] inner levels a); see include/oscar.h."""
    import torch
    n_tok = int(dst_seq.numel())
    st = lib().oscar_evict_quantize_codebook(
        ctypes.byref(shape), n_tok, _dptr(src_kv, "src_kv", torch.bfloat16), int(src_kv.shape[0]),
        _dptr(src_row, "src_row", torch.int32), _dptr(dst_seq, "dst_seq", torch.int32),
        _dptr(dst_pos, "dst_pos", torch.int32), _dptr(new_kv, "new_kv", torch.bfloat16),
        _dptr(U, "U", torch.float32), _dptr(clip, "clip", torch.float32),
        _dptr(codebook, "codebook", torch.float32), _dptr(pool, "pool", torch.uint8),
        _dptr(page_table, "page_table", torch.int32), batch, max_pages, num_pages,
        _dptr(dev_status, "dev_status", torch.int32), _stream_ptr(stream))
    _check("oscar_evict_quantize_codebook", st)


def oscar_decode_attn_codebook(shape: oscar_shape, q, bf16_kv, bf16_len, pool, page_table, max_pages: int,
                               num_pages: int, hist_len, U, codebook, sm_scale: float, out, workspace,
                               dev_status=None, stream=None) -> None:
    """oscar_decode_attn reading the history with the Lloyd-Max levels
    (codebook: fp32 [Hk][2]).  The workspace size is
    oscar_decode_workspace_bytes's."""
    import torch
    B = int(q.shape[0])
    ws = ctypes.c_size_t(int(workspace.numel()))
    st = lib().oscar_decode_attn_codebook(
        ctypes.byref(shape), B, _dptr(q, "q", torch.bfloat16), _dptr(bf16_kv, "bf16_kv", torch.bfloat16),
        _dptr(bf16_len, "bf16_len", torch.int32), _dptr(pool, "pool", torch.uint8),
        _dptr(page_table, "page_table", torch.int32), max_pages, num_pages, _dptr(hist_len, "hist_len", torch.int32),
        _dptr(U, "U", torch.float32), _dptr(codebook, "codebook", torch.float32), ctypes.c_float(sm_scale),
        _dptr(out, "out", torch.float32), _dptr(workspace, "workspace", torch.uint8), ctypes.byref(ws),
        _dptr(dev_status, "dev_status", torch.int32), _stream_ptr(stream))
    _check("oscar_decode_attn_codebook", st)


def _host_i32(a):
    import numpy as np
    return np.ascontiguousarray(a, np.int32)


def _np_ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p) if a is not None and a.size else None


class Pages:
    """Refcounted history pages with copy-on-write (host logic of the C ABI's
    oscar_pages_* calls; see include/oscar.h)."""

    def __init__(self, num_pages: int):
        h = ctypes.c_void_p()
        _check("oscar_pages_create", lib().oscar_pages_create(int(num_pages), ctypes.byref(h)))
        self._h = h

    def close(self) -> None:
        if self._h:
            lib().oscar_pages_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc(self, n: int):
        import numpy as np
        out = np.zeros(max(int(n), 0), np.int32)
        _check("oscar_pages_alloc", lib().oscar_pages_alloc(self._h, int(n), _np_ptr(out)))
        return out

    def retain(self, pages) -> None:
        a = _host_i32(pages)
        _check("oscar_pages_retain", lib().oscar_pages_retain(self._h, a.size, _np_ptr(a)))

    def release(self, pages) -> None:
        a = _host_i32(pages)
        _check("oscar_pages_release", lib().oscar_pages_release(self._h, a.size, _np_ptr(a)))

    def refcount(self, page: int) -> int:
        return int(lib().oscar_pages_refcount(self._h, int(page)))

    def free_count(self) -> int:
        return int(lib().oscar_pages_free_count(self._h))

    def prepare_write(self, seq, page_index, page_table):
        """Make the target pages of page_table (numpy int32 [batch][max_pages],
        updated in place) private; returns (copy_src, copy_dst)."""
        import numpy as np
        sq, pi = _host_i32(seq), _host_i32(page_index)
        assert page_table.dtype == np.int32 and page_table.flags.c_contiguous
        src = np.zeros(max(sq.size, 1), np.int32)
        dst = np.zeros(max(sq.size, 1), np.int32)
        n = ctypes.c_int32(0)
        st = lib().oscar_pages_prepare_write(self._h, sq.size, _np_ptr(sq), _np_ptr(pi),
                                             page_table.ctypes.data_as(ctypes.c_void_p), page_table.shape[0],
                                             page_table.shape[1], _np_ptr(src), _np_ptr(dst), ctypes.byref(n))
        _check("oscar_pages_prepare_write", st)
        return src[:n.value].copy(), dst[:n.value].copy()


class Radix:
    """Radix prefix cache over history pages (the C ABI's oscar_radix_*; see
    include/oscar.h).  Keeps a reference to its Pages allocator."""

    def __init__(self, pages: Pages):
        h = ctypes.c_void_p()
        _check("oscar_radix_create", lib().oscar_radix_create(pages._h, ctypes.byref(h)))
        self._h, self.pages = h, pages

    def close(self) -> None:
        if self._h:
            lib().oscar_radix_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def insert(self, tokens, pages) -> None:
        t, p = _host_i32(tokens), _host_i32(pages)
        _check("oscar_radix_insert", lib().oscar_radix_insert(self._h, _np_ptr(t), t.size, _np_ptr(p), p.size))

    def match(self, tokens, max_pages: int):
        """Page ids of the longest cached prefix (one reference each for the caller)."""
        import numpy as np
        t = _host_i32(tokens)
        out = np.zeros(max(int(max_pages), 1), np.int32)
        n = ctypes.c_int32(0)
        _check("oscar_radix_match", lib().oscar_radix_match(self._h, _np_ptr(t), t.size, int(max_pages),
                                                            _np_ptr(out), ctypes.byref(n)))
        return out[:n.value].copy()

    def evict(self, n_pages: int) -> int:
        n = ctypes.c_int32(0)
        _check("oscar_radix_evict", lib().oscar_radix_evict(self._h, int(n_pages), ctypes.byref(n)))
        return int(n.value)

    def cached_pages(self) -> int:
        return int(lib().oscar_radix_cached_pages(self._h))


def oscar_pages_copy(shape: oscar_shape, copy_src, copy_dst, pool, boost, num_pages: int, stream=None) -> None:
    """Copy the pool blocks (and boost records) of copy_src pages to copy_dst
    pages on the device (host index arrays)."""
    import torch
    src, dst = _host_i32(copy_src), _host_i32(copy_dst)
    assert src.size == dst.size
    st = lib().oscar_pages_copy(ctypes.byref(shape), src.size, _np_ptr(src), _np_ptr(dst),
                                _dptr(pool, "pool", torch.uint8), _dptr(boost, "boost", torch.uint8), num_pages,
                                _stream_ptr(stream))
    _check("oscar_pages_copy", st)


BOOST_N = 8
BOOST_BLOCK_BYTES = 1024        # per (page, KV head): 64 tokens x 8 entries x 2 bytes


def oscar_evict_quantize_boost(shape: oscar_shape, src_kv, dst_seq, dst_pos, U, clip, pool, boost, page_table,
                               batch: int, max_pages: int, num_pages: int, src_row=None, new_kv=None,
                               dev_status=None, stream=None) -> None:
    """oscar_evict_quantize plus the K channel-boost records (boost: uint8
    [num_pages * Hk * BOOST_BLOCK_BYTES]); see include/oscar.h."""
    import torch
    n_tok = int(dst_seq.numel())
    st = lib().oscar_evict_quantize_boost(
        ctypes.byref(shape), n_tok, _dptr(src_kv, "src_kv", torch.bfloat16), int(src_kv.shape[0]),
        _dptr(src_row, "src_row", torch.int32), _dptr(dst_seq, "dst_seq", torch.int32),
        _dptr(dst_pos, "dst_pos", torch.int32), _dptr(new_kv, "new_kv", torch.bfloat16),
        _dptr(U, "U", torch.float32), _dptr(clip, "clip", torch.float32), _dptr(pool, "pool", torch.uint8),
        _dptr(boost, "boost", torch.uint8), _dptr(page_table, "page_table", torch.int32), batch, max_pages,
        num_pages, _dptr(dev_status, "dev_status", torch.int32), _stream_ptr(stream))
    _check("oscar_evict_quantize_boost", st)


def oscar_decode_attn_boost(shape: oscar_shape, q, bf16_kv, bf16_len, pool, boost, page_table, max_pages: int,
                            num_pages: int, hist_len, U, sm_scale: float, out, workspace, dev_status=None,
                            stream=None) -> None:
    """oscar_decode_attn with the boosted K values.  The workspace size is
    oscar_decode_workspace_bytes's."""
    import torch
    B = int(q.shape[0])
    ws = ctypes.c_size_t(int(workspace.numel()))
    st = lib().oscar_decode_attn_boost(
        ctypes.byref(shape), B, _dptr(q, "q", torch.bfloat16), _dptr(bf16_kv, "bf16_kv", torch.bfloat16),
        _dptr(bf16_len, "bf16_len", torch.int32), _dptr(pool, "pool", torch.uint8), _dptr(boost, "boost", torch.uint8),
        _dptr(page_table, "page_table", torch.int32), max_pages, num_pages, _dptr(hist_len, "hist_len", torch.int32),
        _dptr(U, "U", torch.float32), ctypes.c_float(sm_scale), _dptr(out, "out", torch.float32),
        _dptr(workspace, "workspace", torch.uint8), ctypes.byref(ws), _dptr(dev_status, "dev_status", torch.int32),
        _stream_ptr(stream))
    _check("oscar_decode_attn_boost", st)


def oscar_calibrate_codebook(shape: oscar_shape, kv, U, clip, codebook, workspace=None, stream=None) -> None:
    """Lloyd-Max fit of the codebook inner levels a [Hk][2] (fp32 CUDA tensor,
    out) from calibration tokens kv [n_t][Hk][2][d]; see include/oscar.h."""
    import torch
    n_t = int(kv.shape[0])
    if workspace is None:
        need = ctypes.c_size_t(0)
        st = lib().oscar_calibrate_codebook(ctypes.byref(shape), n_t, None, None, None, None, None,
                                            ctypes.byref(need), None)
        _check("oscar_calibrate_codebook", st)
        workspace = torch.zeros(int(need.value), dtype=torch.uint8, device=kv.device)
    ws = ctypes.c_size_t(int(workspace.numel()))
    st = lib().oscar_calibrate_codebook(
        ctypes.byref(shape), n_t, _dptr(kv, "kv", torch.bfloat16), _dptr(U, "U", torch.float32),
        _dptr(clip, "clip", torch.float32), _dptr(codebook, "codebook", torch.float32),
        _dptr(workspace, "workspace", torch.uint8), ctypes.byref(ws), _stream_ptr(stream))
    _check("oscar_calibrate_codebook", st)


OSCAR_OUT_F32, OSCAR_OUT_BF16 = 0, 1
MAX_COPY_POOLS = 128

# The calls below run once per layer and step, where a launch costs a few
# microseconds: their checks touch each tensor once (_arg), and pointers go to
# ctypes as ints.
_F32 = _BF16 = _I32 = _U8 = _raw_stream = _current_device = None


def _torch_names() -> None:
    global _F32, _BF16, _I32, _U8, _raw_stream, _current_device
    import torch
    torch.cuda.current_device()                     # initialises CUDA once; the raw queries below do not
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _current_device = torch._C._cuda_getDevice
    _BF16, _I32, _U8 = torch.bfloat16, torch.int32, torch.uint8
    _F32 = torch.float32                            # last: other threads take it for the sign that all are set


def _arg(t, what: str, dtype, need: int, dev: int):
    """Address of a contiguous tensor of `dtype` on device `dev` with at least
    `need` elements (None -> NULL)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.get_device() == dev and t.numel() >= need and t.is_contiguous():
            return t.data_ptr()
        if not t.is_cuda:
            raise TypeError(f"{what}: expected a CUDA tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{what}: must be contiguous")
        if t.numel() < need:
            raise ValueError(f"{what}: {t.numel()} elements, {need} are needed")
        raise ValueError(f"{what}: on device {t.get_device()}, the current device is {dev}")
    except AttributeError:
        raise TypeError(f"{what}: expected a CUDA tensor") from None


def _stream_arg(stream, dev: int):
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev)


def _out_type(out) -> int:
    """OSCAR_OUT_* of an output tensor."""
    if _F32 is None:
        _torch_names()
    if out.dtype is _BF16:
        return OSCAR_OUT_BF16
    if out.dtype is _F32:
        return OSCAR_OUT_F32
    raise TypeError(f"out: expected float32 or bfloat16, got {out.dtype}")


def _pool_block(shape: oscar_shape, bits: int) -> int:
    """Block bytes of a pool of a supported shape (the library refuses the
    others): codes of 64 K and V vectors and their pairs."""
    return bits * 2048 + 512 * (128 // max(shape.quant_group, 1))


def block_bytes_int4(shape: oscar_shape) -> int:
    """Bytes of a (page, KV head) block of a 4-bit pool, 0 if unsupported."""
    return int(lib().oscar_block_bytes_int4(ctypes.byref(shape)))


def oscar_evict_quantize_int4(shape: oscar_shape, src_kv, dst_seq, dst_pos, U, clip, pool, page_table, batch: int,
                              max_pages: int, num_pages: int, src_row=None, new_kv=None, dev_status=None,
                              stream=None) -> None:
    """oscar_evict_quantize into a 4-bit pool (num_pages * Hk blocks of
    block_bytes_int4(shape) bytes); see include/oscar.h."""
    if _F32 is None:
        _torch_names()
    dev, n, hk, d = _current_device(), dst_seq.numel(), shape.num_kv_heads, shape.head_dim
    rows, row = src_kv.shape[0], hk * 2 * d
    st = lib().oscar_evict_quantize_int4(
        ctypes.byref(shape), n, _arg(src_kv, "src_kv", _BF16, rows * row, dev), rows,
        _arg(src_row, "src_row", _I32, n, dev), _arg(dst_seq, "dst_seq", _I32, n, dev),
        _arg(dst_pos, "dst_pos", _I32, n, dev), _arg(new_kv, "new_kv", _BF16, n * row, dev),
        _arg(U, "U", _F32, row * d, dev), _arg(clip, "clip", _F32, hk * 2, dev),
        _arg(pool, "pool", _U8, num_pages * hk * _pool_block(shape, 4), dev),
        _arg(page_table, "page_table", _I32, batch * max_pages, dev), batch, max_pages, num_pages,
        _arg(dev_status, "dev_status", _I32, 1, dev), _stream_arg(stream, dev))
    if st:
        _check("oscar_evict_quantize_int4", st)


def oscar_decode_workspace_bytes_int4(shape: oscar_shape, batch: int, max_pages: int) -> int:
    ws = ctypes.c_size_t(0)
    st = lib().oscar_decode_attn_int4(ctypes.byref(shape), batch, None, None, None, None, None, max_pages, 0, None,
                                      None, ctypes.c_float(1.0), None, OSCAR_OUT_F32, None, ctypes.byref(ws), None,
                                      None)
    _check("oscar_decode_attn_int4", st)
    return int(ws.value)


def oscar_decode_attn_int4(shape: oscar_shape, q, bf16_kv, bf16_len, pool, page_table, max_pages: int,
                           num_pages: int, hist_len, U, sm_scale: float, out, workspace, dev_status=None,
                           stream=None) -> None:
    """oscar_decode_attn over a 4-bit pool; out may be float32 or bfloat16 (see
    include/oscar.h).  ``workspace``: CUDA uint8 tensor of at least
    oscar_decode_workspace_bytes_int4(shape, batch, max_pages) bytes."""
    kind = _out_type(out)
    dev, B, hk, d = _current_device(), q.shape[0], shape.num_kv_heads, shape.head_dim
    rows, slots = B * shape.num_q_heads * d, shape.sink + shape.recent
    st = lib().oscar_decode_attn_int4(
        ctypes.byref(shape), B, _arg(q, "q", _BF16, rows, dev),
        _arg(bf16_kv, "bf16_kv", _BF16, B * slots * hk * 2 * d, dev), _arg(bf16_len, "bf16_len", _I32, B, dev),
        _arg(pool, "pool", _U8, num_pages * hk * _pool_block(shape, 4), dev),
        _arg(page_table, "page_table", _I32, B * max_pages, dev), max_pages, num_pages,
        _arg(hist_len, "hist_len", _I32, B, dev), _arg(U, "U", _F32, hk * 2 * d * d, dev), sm_scale,
        _arg(out, "out", out.dtype, rows, dev), kind, _arg(workspace, "workspace", _U8, 1 if B else 0, dev),
        ctypes.byref(ctypes.c_size_t(workspace.numel())), _arg(dev_status, "dev_status", _I32, 1, dev),
        _stream_arg(stream, dev))
    if st:
        _check("oscar_decode_attn_int4", st)


def oscar_history_read(shape: oscar_shape, bits: int, seq, pos, pool, page_table, batch: int, max_pages: int,
                       num_pages: int, out, dev_status=None, stream=None) -> None:
    """Stored tokens (seq, pos: int32 [n]) as rows out [n][Hk][2][d] (float32 or
    bfloat16) in the rotated domain; bits: 2 (uniform levels: not for a Lloyd-Max
    pool) or 4, the pool's codes; see include/oscar.h."""
    kind = _out_type(out)
    dev, n, hk = _current_device(), seq.numel(), shape.num_kv_heads
    st = lib().oscar_history_read(
        ctypes.byref(shape), bits, n, _arg(seq, "seq", _I32, n, dev), _arg(pos, "pos", _I32, n, dev),
        _arg(pool, "pool", _U8, num_pages * hk * _pool_block(shape, bits), dev),
        _arg(page_table, "page_table", _I32, batch * max_pages, dev), batch, max_pages, num_pages,
        _arg(out, "out", out.dtype, n * hk * 2 * shape.head_dim, dev), kind,
        _arg(dev_status, "dev_status", _I32, 1, dev), _stream_arg(stream, dev))
    if st:
        _check("oscar_history_read", st)


def oscar_history_gather(shape: oscar_shape, bits: int, pool, src_table, dst_table, keep, n_keep, num_pages: int,
                         boost=None, dev_status=None, stream=None) -> None:
    """The kept tokens (keep: int32 [B][stride] source positions, the first
    n_keep[b] of row b) of each history moved to positions 0, 1, ... of its
    row of dst_table (int32 [B][pages], fresh pages); see include/oscar.h."""
    if _F32 is None:
        _torch_names()
    (B, smax), (B2, dmax), (B3, stride) = src_table.shape, dst_table.shape, keep.shape
    if B2 != B or B3 != B:
        raise ValueError("src_table, dst_table and keep: one row per sequence")
    dev, hk = _current_device(), shape.num_kv_heads
    st = lib().oscar_history_gather(
        ctypes.byref(shape), bits, B, _arg(pool, "pool", _U8, num_pages * hk * _pool_block(shape, bits), dev),
        _arg(boost, "boost", _U8, num_pages * hk * BOOST_BLOCK_BYTES, dev), _arg(src_table, "src_table", _I32, 0, dev),
        smax, _arg(dst_table, "dst_table", _I32, 0, dev), dmax, _arg(keep, "keep", _I32, 0, dev), stride,
        _arg(n_keep, "n_keep", _I32, B, dev), num_pages, _arg(dev_status, "dev_status", _I32, 1, dev),
        _stream_arg(stream, dev))
    if st:
        _check("oscar_history_gather", st)


def _pool_args(pools, need: int, dev: int) -> list:
    """Addresses of the pools of a copy.  The usual case is checked by loops in
    C (36 layers: half the time of as many _arg calls); anything else goes
    through _arg, which says what is wrong."""
    import torch
    T = torch.Tensor
    try:
        if ({t.dtype for t in pools} <= {_U8} and set(map(T.get_device, pools)) <= {dev}
                and min(map(T.numel, pools), default=need) >= need and all(map(T.is_contiguous, pools))):
            return list(map(T.data_ptr, pools))
    except (AttributeError, TypeError):
        pass
    return [_arg(t, "pools", _U8, need, dev) for t in pools]


def oscar_pages_copy_device(page_bytes: int, src, dst, pools, num_pages: int, dev_status=None, stream=None) -> None:
    """Page src[i] copied to page dst[i] (int32 CUDA tensors) in every pool of
    the list (uint8 CUDA tensors of num_pages pages of page_bytes each) by
    one launch; see include/oscar.h."""
    if _F32 is None:
        _torch_names()
    dev, n, need = _current_device(), src.numel(), num_pages * page_bytes
    if len(pools) > MAX_COPY_POOLS:
        raise ValueError(f"pools: {len(pools)}, at most {MAX_COPY_POOLS}")
    ptrs = array.array("Q", _pool_args(pools, need, dev))
    st = lib().oscar_pages_copy_device(
        page_bytes, n, _arg(src, "src", _I32, n, dev), _arg(dst, "dst", _I32, n, dev),
        ptrs.buffer_info()[0], len(pools), num_pages,
        _arg(dev_status, "dev_status", _I32, 1, dev), _stream_arg(stream, dev))
    if st:
        _check("oscar_pages_copy_device", st)


def oscar_decode_workspace_bytes_weights(shape: oscar_shape, bits: int, batch: int, max_pages: int) -> int:
    ws = ctypes.c_size_t(0)
    st = lib().oscar_decode_attn_weights(ctypes.byref(shape), bits, batch, None, None, None, None, None, max_pages, 0,
                                         None, None, 1.0, None, OSCAR_OUT_F32, None, 0, None, 1.0, None,
                                         ctypes.byref(ws), None, None)
    _check("oscar_decode_attn_weights", st)
    return int(ws.value)


def oscar_decode_attn_weights(shape: oscar_shape, bits: int, q, bf16_kv, bf16_len, pool, page_table, max_pages: int,
                              num_pages: int, hist_len, U, sm_scale: float, out, weight, workspace, slot_weight=None,
                              decay: float = 1.0, dev_status=None, stream=None) -> None:
    """oscar_decode_attn (bits 2) or oscar_decode_attn_int4 (bits 4) with each
    token's attention weight, summed over the query heads, added to decay times
    its score: weight float32 [B][>= 64 max_pages] for the history,
    slot_weight float32 [B][sink + recent] for the windows; see
    include/oscar.h.  ``workspace``: CUDA uint8 tensor of at least
    oscar_decode_workspace_bytes_weights(shape, bits, batch, max_pages) bytes."""
    kind = _out_type(out)
    dev, B, hk, d = _current_device(), q.shape[0], shape.num_kv_heads, shape.head_dim
    rows, slots = B * shape.num_q_heads * d, shape.sink + shape.recent
    if weight.dim() != 2 or weight.shape[0] != B:
        raise ValueError("weight: one row per sequence")
    st = lib().oscar_decode_attn_weights(
        ctypes.byref(shape), bits, B, _arg(q, "q", _BF16, rows, dev),
        _arg(bf16_kv, "bf16_kv", _BF16, B * slots * hk * 2 * d, dev), _arg(bf16_len, "bf16_len", _I32, B, dev),
        _arg(pool, "pool", _U8, num_pages * hk * _pool_block(shape, bits), dev),
        _arg(page_table, "page_table", _I32, B * max_pages, dev), max_pages, num_pages,
        _arg(hist_len, "hist_len", _I32, B, dev), _arg(U, "U", _F32, hk * 2 * d * d, dev), sm_scale,
        _arg(out, "out", out.dtype, rows, dev), kind, _arg(weight, "weight", _F32, 0, dev), weight.shape[1],
        _arg(slot_weight, "slot_weight", _F32, B * slots, dev), decay,
        _arg(workspace, "workspace", _U8, 1 if B else 0, dev), ctypes.byref(ctypes.c_size_t(workspace.numel())),
        _arg(dev_status, "dev_status", _I32, 1, dev), _stream_arg(stream, dev))
    if st:
        _check("oscar_decode_attn_weights", st)


def oscar_history_select(weight, hist_len, budget, keep, n_keep, protect: int = 0, kept_weight=None, dev_status=None,
                         stream=None) -> None:
    """The tokens of each history that stay under budget (int32 [B]) by their
    scores weight (float32 [B][stride]), the newest ``protect`` first: their
    positions in increasing order into keep (int32 [B][stride]), their number
    into n_keep (int32 [B]), their scores into kept_weight (float32 [B][stride]);
    see include/oscar.h.  The lists are those that oscar_history_gather takes."""
    if _F32 is None:
        _torch_names()
    (B, stride), (B2, kstride) = weight.shape, keep.shape
    if B2 != B or (kept_weight is not None and (kept_weight.dim() != 2 or kept_weight.shape[0] != B)):
        raise ValueError("weight, keep and kept_weight: one row per sequence")
    dev = _current_device()
    st = lib().oscar_history_select(
        B, _arg(weight, "weight", _F32, 0, dev), stride, _arg(hist_len, "hist_len", _I32, B, dev),
        _arg(budget, "budget", _I32, B, dev), protect, _arg(keep, "keep", _I32, 0, dev), kstride,
        _arg(n_keep, "n_keep", _I32, B, dev), _arg(kept_weight, "kept_weight", _F32, 0, dev),
        0 if kept_weight is None else kept_weight.shape[1], _arg(dev_status, "dev_status", _I32, 1, dev),
        _stream_arg(stream, dev))
    if st:
        _check("oscar_history_select", st)


def oscar_decode_workspace_bytes_shared(shape: oscar_shape, bits: int, batch: int, max_pages: int, n_groups: int) -> int:
    ws = ctypes.c_size_t(0)
    st = lib().oscar_decode_attn_shared(ctypes.byref(shape), bits, batch, None, None, None, None, None, max_pages, 0, None,
                                        None, n_groups, None, 0, None, 1.0, None, OSCAR_OUT_F32, None, ctypes.byref(ws),
                                        None, None)
    _check("oscar_decode_attn_shared", st)
    return int(ws.value)


def oscar_decode_attn_shared(shape: oscar_shape, bits: int, q, bf16_kv, bf16_len, pool, page_table, max_pages: int,
                             num_pages: int, hist_len, prefix_group, group_pages, U, sm_scale: float, out, workspace,
                             min_members: int = 0, dev_status=None, stream=None) -> None:
    """oscar_decode_attn (bits 2) or oscar_decode_attn_int4 (bits 4) with the
    first group_pages[g] (int32 [n_groups]) pages of the sequences whose
    prefix_group (int32 [B]; negative: none) is g read once for all of them, if
    they are at least min_members (0: where it is faster); out may be float32 or bfloat16; see include/oscar.h.  ``workspace``: CUDA
    uint8 tensor of at least oscar_decode_workspace_bytes_shared(shape, bits,
    batch, max_pages, n_groups) bytes."""
    kind = _out_type(out)
    dev, B, hk, d = _current_device(), q.shape[0], shape.num_kv_heads, shape.head_dim
    rows, slots, n_groups = B * shape.num_q_heads * d, shape.sink + shape.recent, group_pages.numel()
    st = lib().oscar_decode_attn_shared(
        ctypes.byref(shape), bits, B, _arg(q, "q", _BF16, rows, dev),
        _arg(bf16_kv, "bf16_kv", _BF16, B * slots * hk * 2 * d, dev), _arg(bf16_len, "bf16_len", _I32, B, dev),
        _arg(pool, "pool", _U8, num_pages * hk * _pool_block(shape, bits), dev),
        _arg(page_table, "page_table", _I32, B * max_pages, dev), max_pages, num_pages,
        _arg(hist_len, "hist_len", _I32, B, dev), _arg(prefix_group, "prefix_group", _I32, B, dev), n_groups,
        _arg(group_pages, "group_pages", _I32, n_groups, dev), min_members, _arg(U, "U", _F32, hk * 2 * d * d, dev),
        sm_scale, _arg(out, "out", out.dtype, rows, dev), kind, _arg(workspace, "workspace", _U8, 1 if B else 0, dev),
        ctypes.byref(ctypes.c_size_t(workspace.numel())), _arg(dev_status, "dev_status", _I32, 1, dev),
        _stream_arg(stream, dev))
    if st:
        _check("oscar_decode_attn_shared", st)
