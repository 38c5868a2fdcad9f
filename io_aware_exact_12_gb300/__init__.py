"""GB300 (sm_103a) fused exact attention: Python binding of the C ABI in
``include/attn.h``.

This module only marshals arguments: it checks tensor shapes/dtypes, allocates
outputs with torch (device memory and streams are the only things torch is
used for), and calls the same-named C entry points of ``libattn.so`` through
ctypes.  Every step of the computation runs in the library's CUDA kernels.
There is no fallback: if the library is missing or fails to load, every call
raises.

Layout: q, k, v, o, do and the gradients are contiguous [B, H, N, d] tensors
(bf16 or fp16) on one CUDA device; lse is fp32 [B, H, N].  The windowed calls
take [B, heads, N, d] tensors of any strides whose channels are contiguous, and
fewer key/value heads than query heads.  The paged-cache calls take token-major
rows [rows, heads, d] and a ``PagedKV``.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

__all__ = ["attention", "attn_fwd", "attn_bwd", "attn_fwd_dropout", "attn_bwd_dropout", "attn_decode", "attn_fwd_fp8", "attn_fwd_blocksparse", "attn_bwd_blocksparse",
           "attn_fwd_blocksparse_dropout", "attn_bwd_blocksparse_dropout", "attn_fwd_window", "attn_bwd_window", "PagedKV",
           "attn_paged_assign", "attn_paged_append", "attn_paged_decode", "attn_paged_decode_window", "attn_paged_select",
           "rotation_tables", "sync_status", "status_string", "last_launch_count", "lib",
           "AttnError", "LIB_PATH", "STATUS"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libattn.so")

STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_CUDA",
          4: "ATTN_ERR_TIMEOUT", 5: "ATTN_ERR_ARCH", 6: "ATTN_ERR_DEVICE_CHECK"}


class AttnError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__("%s failed: %s (%d)" % (fn, STATUS.get(code, "?"), code))
        self.code = code


class _PagedKvStruct(ctypes.Structure):  # attn_paged_kv_t
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_strides", ctypes.c_longlong * 3), ("v_strides", ctypes.c_longlong * 3),
                ("k_min", ctypes.c_void_p), ("k_max", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("table_stride", ctypes.c_longlong),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("max_pages", ctypes.c_int), ("B", ctypes.c_int),
                ("type", ctypes.c_int), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class _CacheStruct(ctypes.Structure):  # what the compiled binding reads
    _fields_ = [("kv", _PagedKvStruct), ("device", ctypes.c_int)]


class _RowsStruct(ctypes.Structure):  # attn_rows_t
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


class _BhndStruct(ctypes.Structure):  # attn_bhnd_t
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong),
                ("row_stride", ctypes.c_longlong)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libattn.so not built; run `python -m io_aware_exact_12_gb300.build` "
                              "(or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, F, I, P]
        L.attn_fwd_f16.argtypes = L.attn_fwd.argtypes
        L.attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, F, I, P]
        L.attn_bwd_f16.argtypes = L.attn_bwd.argtypes
        for f in (L.attn_fwd, L.attn_fwd_f16, L.attn_bwd, L.attn_bwd_f16):
            f.restype = I
        U64, U32 = ctypes.c_ulonglong, ctypes.c_uint
        for f in (L.attn_fwd_dropout, L.attn_fwd_dropout_f16):
            f.argtypes = [P, P, P, P, P, I, I, I, I, F, I, F, U64, U32, P]
            f.restype = I
        for f in (L.attn_bwd_dropout, L.attn_bwd_dropout_f16):
            f.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, F, I, F, U64, U32, P]
            f.restype = I
        for f in (L.attn_fwd_blocksparse, L.attn_fwd_blocksparse_f16):
            f.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, I, P]
            f.restype = I
        for f in (L.attn_bwd_blocksparse, L.attn_bwd_blocksparse_f16):
            f.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, F, I, P]
            f.restype = I
        for f in (L.attn_fwd_blocksparse_dropout, L.attn_fwd_blocksparse_dropout_f16):
            f.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, I, F, U64, U32, P]
            f.restype = I
        for f in (L.attn_bwd_blocksparse_dropout, L.attn_bwd_blocksparse_dropout_f16):
            f.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, F, I, F, U64, U32, P]
            f.restype = I
        L.attn_fwd_fp8.argtypes = [P, P, P, F, F, F, P, P, I, I, I, I, F, I, P]
        L.attn_fwd_fp8.restype = I
        L.attn_decode.argtypes = [P, P, P, P, P, I, I, I, I, F, P]
        L.attn_decode.restype = I
        L.attn_paged_append.argtypes = [P, P, P, P, P, I, I, P, P, P, I, I, I, I, P]
        L.attn_paged_decode.argtypes = [P, P, I, P, P, P, I, F, I, P, P]
        L.attn_paged_select.argtypes = [P, P, I, P, I, I, I, I, P, P]
        L.attn_paged_decode_window.argtypes = [P, P, I, P, P, I, I, F, I, P, P]
        L.attn_paged_assign.argtypes = [P, P, P, P, I, P, P, P, P, I, I, I, P, P]
        L.attn_fwd_window.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, P]
        L.attn_bwd_window.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, P, P]
        L.attn_bwd_window_workspace.argtypes = [I, I, I, I, I, I, I, I]
        L.attn_bwd_window_workspace.restype = ctypes.c_longlong
        for f in (L.attn_paged_append, L.attn_paged_decode, L.attn_paged_select, L.attn_paged_decode_window,
                  L.attn_paged_assign, L.attn_fwd_window, L.attn_bwd_window):
            f.restype = I
        L.attn_paged_decode_workspace.argtypes = [P, I, I]
        L.attn_paged_decode_window_workspace.argtypes = [P, I, I, I]
        L.attn_paged_select_workspace.argtypes = [P]
        L.attn_paged_assign_workspace.argtypes = [P]
        for f in (L.attn_paged_decode_workspace, L.attn_paged_decode_window_workspace, L.attn_paged_select_workspace,
                  L.attn_paged_assign_workspace):
            f.restype = ctypes.c_longlong
        L.attn_sync_status.argtypes = [P]
        L.attn_sync_status.restype = I
        L.attn_status_string.argtypes = [I]
        L.attn_status_string.restype = ctypes.c_char_p
        L.attn_last_launch_count.argtypes = []
        L.attn_last_launch_count.restype = I
        L.attn_probe_ex2.argtypes = [P, I, I, P]
        L.attn_probe_ex2.restype = I
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().attn_status_string(int(code)).decode()


def last_launch_count() -> int:
    return lib().attn_last_launch_count()


EX2_PROBE_THREADS = 256
EX2_PROBE_CHAINS = 8


def probe_ex2(sink, blocks, iters, stream=None):
    """Enqueue the exponential-unit throughput probe (attn_probe_ex2) writing
    one float per thread into `sink` (a float32 CUDA tensor of at least
    blocks * 256 elements).  Returns the number of exponentials it computes."""
    if not isinstance(sink, torch.Tensor) or not sink.is_cuda or sink.dtype != torch.float32:
        raise TypeError("sink must be a float32 CUDA tensor")
    if not sink.is_contiguous() or sink.numel() < blocks * EX2_PROBE_THREADS:
        raise ValueError("sink must be contiguous with at least blocks * 256 elements")
    with _on_device(sink):
        rc = lib().attn_probe_ex2(sink.data_ptr(), int(blocks), int(iters), _stream_handle(stream))
    if rc != 0:
        raise RuntimeError("attn_probe_ex2: %s" % status_string(rc))
    return blocks * EX2_PROBE_THREADS * iters * EX2_PROBE_CHAINS


class _Nothing:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NOTHING = _Nothing()


def _on_device(t):
    """The C ABI works on the current device: switch to t's device only when
    it is not already current (entering torch.cuda.device costs several us)."""
    idx = t.device.index
    if idx is None or idx == torch.cuda.current_device():
        return _NOTHING
    return torch.cuda.device(t.device)


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _check(name, t, like=None, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous [B, H, N, d]" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    if like is not None and (t.shape != like.shape or t.device != like.device):
        raise ValueError("%s must match q's shape/device" % name)


def _dims(q):
    if q.dim() != 4:
        raise ValueError("q must be [B, H, N, d]")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("q must be bf16 or fp16")
    return tuple(int(x) for x in q.shape)


def attn_fwd(q, k, v, scale=None, causal=False, o=None, lse=None, stream=None):
    """O, LSE = exact softmax(scale q k^T [+ causal]) v.  Returns (o, lse)."""
    B, H, N, d = _dims(q)
    _check("q", q)
    _check("k", k, q, q.dtype)
    _check("v", v, q, q.dtype)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check("o", o, q, q.dtype)
    _check("lse", lse, None, torch.float32)
    fn = lib().attn_fwd if q.dtype == torch.bfloat16 else lib().attn_fwd_f16
    with _on_device(q):
        rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
                float(scale), int(bool(causal)), _stream_handle(stream))
    if rc:
        raise AttnError("attn_fwd", rc)
    return o, lse


def attn_bwd(q, k, v, o, do, lse, scale=None, causal=False, dq=None, dk=None, dv=None, stream=None):
    """dQ, dK, dV of L = <O, dO> by recomputation from LSE.  Returns (dq, dk, dv)."""
    B, H, N, d = _dims(q)
    _check("q", q)
    for name, t in (("k", k), ("v", v), ("o", o), ("do", do)):
        _check(name, t, q, q.dtype)
    _check("lse", lse, None, torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check(name, t, q, q.dtype)
    fn = lib().attn_bwd if q.dtype == torch.bfloat16 else lib().attn_bwd_f16
    with _on_device(q):
        rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, float(scale), int(bool(causal)),
                _stream_handle(stream))
    if rc:
        raise AttnError("attn_bwd", rc)
    return dq, dk, dv


def attn_fwd_dropout(q, k, v, p_drop, seed, offset=0, scale=None, causal=False, o=None, lse=None, stream=None):
    """attn_fwd with inverted dropout of probability ``p_drop`` on P, the keep
    decisions drawn in the kernel from Philox4x32-10 keyed by ``seed`` (64-bit)
    with ``offset`` (32-bit) as the fourth counter word.  bf16 or fp16.
    Returns (o, lse); lse is that of the undropped softmax."""
    B, H, N, d = _dims(q)
    _check("q", q)
    _check("k", k, q, q.dtype)
    _check("v", v, q, q.dtype)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q) if o is None else o
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check("o", o, q, q.dtype)
    _check("lse", lse, None, torch.float32)
    with _on_device(q):
        fn = lib().attn_fwd_dropout if q.dtype == torch.bfloat16 else lib().attn_fwd_dropout_f16
        rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H,
                N, d, float(scale), int(bool(causal)), float(p_drop),
                int(seed) & 0xFFFFFFFFFFFFFFFF, int(offset) & 0xFFFFFFFF,
                _stream_handle(stream))
    if rc:
        raise AttnError("attn_fwd_dropout", rc)
    return o, lse


def attn_bwd_dropout(q, k, v, o, do, lse, p_drop, seed, offset=0, scale=None, causal=False, dq=None, dk=None,
                     dv=None, stream=None):
    """Gradients of attn_fwd_dropout's output (same p_drop, seed, offset): the
    keep decisions are drawn again, not stored.  Returns (dq, dk, dv)."""
    B, H, N, d = _dims(q)
    _check("q", q)
    for name, t in (("k", k), ("v", v), ("o", o), ("do", do)):
        _check(name, t, q, q.dtype)
    _check("lse", lse, None, torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check(name, t, q, q.dtype)
    with _on_device(q):
        fn = lib().attn_bwd_dropout if q.dtype == torch.bfloat16 else lib().attn_bwd_dropout_f16
        rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                float(scale), int(bool(causal)), float(p_drop),
                int(seed) & 0xFFFFFFFFFFFFFFFF, int(offset) & 0xFFFFFFFF,
                _stream_handle(stream))
    if rc:
        raise AttnError("attn_bwd_dropout", rc)
    return dq, dk, dv


def attn_decode(q, k, v, scale=None, o=None, lse=None, stream=None):
    """One decode step: q [B, H, d] (or [B, H, 1, d]) against the cache k, v
    [B, H, L, d], bf16; every key visible.  Returns (o [B, H, d], lse [B, H])."""
    if q.dim() == 4:
        if q.shape[2] != 1:
            raise ValueError("decode takes one query token per (batch, head)")
        q = q.reshape(q.shape[0], q.shape[1], q.shape[3])
    if q.dim() != 3 or k.dim() != 4:
        raise ValueError("q must be [B, H, d] and k, v [B, H, L, d]")
    B, H, d = (int(x) for x in q.shape)
    Lk = int(k.shape[2])
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(name, t, None, torch.bfloat16)
    if tuple(k.shape) != (B, H, Lk, d) or tuple(v.shape) != (B, H, Lk, d):
        raise ValueError("k and v must be [B, H, L, d] matching q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H), dtype=torch.float32, device=q.device) if lse is None else lse
    _check("o", o, q, torch.bfloat16)
    _check("lse", lse, None, torch.float32)
    with _on_device(q):
        rc = lib().attn_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, Lk,
                               d, float(scale), _stream_handle(stream))
    if rc:
        raise AttnError("attn_decode", rc)
    return o, lse


_TYPE_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}


class PagedKV:
    """A paged key/value cache (attn_paged_kv_t): the caller's tensors, checked
    once, and what the paged calls need to know of them.

    k_pages, v_pages : [num_pages, kv_heads, page_size, d] bf16, fp16 or
        float8_e4m3fn; any strides whose channels are contiguous and whose rows
        do not overlap (pages stored as [page_size, kv_heads, d] come in as
        ``t.permute(0, 2, 1, 3)``).
    block_table : [B, max_pages] int32; seq_lens : [B] int32.  Both are read by
        the kernels, so a program updates them in place, also between replays of
        a captured graph.
    k_scale, v_scale : value of one unit of an e4m3 cache (1 otherwise).
    k_min, k_max : [num_pages, kv_heads, d] of the cache's type, contiguous: key
        summaries for attn_paged_select, kept by attn_paged_append.

    The object holds references to the tensors and no data of its own.  Its
    attributes cannot be assigned: the calls go by what it was built with, so new
    lengths or tables are written into the tensors, and other tensors want
    another PagedKV."""

    __slots__ = ("k_pages", "v_pages", "block_table", "seq_lens", "k_min", "k_max", "k_scale", "v_scale", "device",
                 "B", "kv_heads", "page_size", "head_dim", "max_pages", "dtype", "_struct", "_address")

    def __init__(self, k_pages, v_pages, block_table, seq_lens, k_scale=1.0, v_scale=1.0, k_min=None, k_max=None):
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError("%s must be a CUDA tensor" % name)
            if t.dtype not in _TYPE_CODES:
                raise TypeError("%s must be bf16, fp16 or float8_e4m3fn" % name)
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError("%s must be [num_pages, kv_heads, page_size, d] with contiguous channels" % name)
        dev = k_pages.device
        if v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype or v_pages.device != dev:
            raise ValueError("v_pages must match k_pages' shape, type and device")
        for name, t, dim in (("block_table", block_table, 2), ("seq_lens", seq_lens, 1)):
            if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != torch.int32:
                raise TypeError("%s must be an int32 tensor on the cache's device" % name)
            if t.dim() != dim or (t.shape[-1] > 1 and t.stride(-1) != 1):
                raise ValueError("%s must have %d dimension(s), the last contiguous" % (name, dim))
        if seq_lens.shape[0] != block_table.shape[0]:
            raise ValueError("block_table and seq_lens must have one row per sequence")
        if (k_min is None) != (k_max is None):
            raise ValueError("k_min and k_max come together")
        P, H, page, d = (int(x) for x in k_pages.shape)
        for name, t in (("k_min", k_min), ("k_max", k_max)):
            if t is None:
                continue
            if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype != k_pages.dtype:
                raise TypeError("%s must be of the cache's type on its device" % name)
            if tuple(t.shape) != (P, H, d) or not t.is_contiguous():
                raise ValueError("%s must be a contiguous [num_pages, kv_heads, d]" % name)
        three = ctypes.c_longlong * 3
        B, max_pages, k_scale, v_scale = int(block_table.shape[0]), int(block_table.shape[1]), float(k_scale), float(v_scale)
        struct = _CacheStruct(_PagedKvStruct(
            k_pages.data_ptr(), v_pages.data_ptr(), three(*k_pages.stride()[:3]), three(*v_pages.stride()[:3]),
            k_min.data_ptr() if k_min is not None else None, k_max.data_ptr() if k_max is not None else None,
            block_table.data_ptr(), seq_lens.data_ptr(), int(block_table.stride(0)), P, page, H, d, max_pages,
            B, _TYPE_CODES[k_pages.dtype], k_scale, v_scale), dev.index)
        for name, value in (("k_pages", k_pages), ("v_pages", v_pages), ("block_table", block_table), ("seq_lens", seq_lens),
                            ("k_min", k_min), ("k_max", k_max), ("k_scale", k_scale), ("v_scale", v_scale), ("device", dev),
                            ("B", B), ("kv_heads", H), ("page_size", page), ("head_dim", d), ("max_pages", max_pages),
                            ("dtype", k_pages.dtype), ("_struct", struct), ("_address", ctypes.addressof(struct))):
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError("a PagedKV cannot be changed (%s): write into its tensors, or build another" % name)

    def __delattr__(self, name):
        raise AttributeError("a PagedKV cannot be changed (%s)" % name)

    def __copy__(self):
        return self


_native_module = None


def _native():
    """The compiled marshalling of the paged and windowed calls (raises if it has not been built)."""
    global _native_module
    if _native_module is None:
        lib()  # says how to build where that has not been done
        from . import _paged
        _native_module = _paged
    return _native_module


class _OnStream:
    """A stream of the cache's (or q's) device as the current one: what a call
    allocates then belongs to the stream that it runs on."""

    def __init__(self, on, stream):
        if stream.device != on.device:
            raise ValueError("the stream must be of the tensors' device")
        self.stream = torch.cuda.stream(stream)

    def __enter__(self):
        self.stream.__enter__()

    def __exit__(self, *exc):
        self.stream.__exit__(*exc)
        return False


def _paged_call(name, kv, stream, *args):
    if not isinstance(kv, PagedKV):
        raise TypeError("kv must be a PagedKV")
    f = getattr(_native_module or _native(), name)
    if stream is None:
        r = f(kv._address, *args)
    else:
        with _OnStream(kv, stream):
            r = f(kv._address, *args)
    if type(r) is int:
        raise AttnError("attn_paged_" + name, r)
    return r


def rotation_tables(positions, rot_dim, base=10000.0, device=None):
    """cos and sin [positions, rot_dim / 2] (fp32) of the angles
    p * base^(-2 i / rot_dim), computed in 64 bits, for attn_paged_append."""
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return angle.cos().float(), angle.sin().float()


def attn_paged_append(kv, k, v, q=None, q_out=None, token_start=None, cos=None, sin=None, interleaved=False,
                      stream=None):
    """Append new tokens' k, v [rows, kv_heads, d] to the cache, rotated by the
    tables cos, sin [positions, rot_dim / 2] (none: not rotated), and rotate q
    [rows, q_heads, d] with them.  kv.seq_lens counts the new tokens already;
    token_start [B + 1] int32 gives each sequence's rows (None: one row per
    sequence).  Returns q_out (allocated where None; may be q itself), or None
    without q.  Rows of padding and empty slots are left as they are."""
    return _paged_call("append", kv, stream, k, v, q, q_out, token_start, cos, sin, interleaved)


def attn_paged_decode(kv, q, pages=None, scale=None, o=None, lse=None, stream=None):
    """One decode step over the paged cache: q [B, q_heads, d] (query heads in
    groups of q_heads / kv_heads share a key/value head) against each
    sequence's seq_lens tokens, or the tokens of the listed ``pages``
    [B, kv_heads, n] (attn_paged_select).  Returns (o [B, q_heads, d],
    lse [B, q_heads]); an empty sequence gets o = 0, lse = -inf."""
    return _paged_call("decode", kv, stream, q, pages, scale, o, lse)


def attn_paged_select(kv, q, n_select, keep_first=1, keep_last=1, pages=None, stream=None):
    """The ``n_select`` pages of each sequence and key/value head on which q
    [B, q_heads, d] can have its largest logits (scale > 0), by the bound that
    the cache's key summaries give; the first keep_first and last keep_last
    pages always, equal scores by the lower index.  Returns int32
    [B, kv_heads, n_select] page indices, ascending, -1 behind the pages of a
    shorter sequence, for attn_paged_decode."""
    if isinstance(kv, PagedKV) and kv.k_min is None:
        raise ValueError("the cache has no key summaries (k_min, k_max)")
    return _paged_call("select", kv, stream, q, n_select, keep_first, keep_last, pages)


def attn_paged_decode_window(kv, q, window, sinks=0, scale=None, o=None, lse=None, stream=None):
    """attn_paged_decode for a model with a sliding window: each sequence's new
    token sees its last ``window`` tokens (itself among them) and the first
    ``sinks`` ones.  Pages of other tokens are neither looked up nor read."""
    return _paged_call("decode_window", kv, stream, q, window, sinks, scale, o, lse)


def attn_paged_assign(kv, n_new, free_pages, free_state, lens=None, free_out=None, token_start=None, slots=None,
                      rows=None, window=0, sinks=0, stream=None):
    """Bookkeeping of a step on the device: writes kv.seq_lens and the new
    entries of kv.block_table for n_new [B] int32 new tokens of each sequence (-1:
    the sequence is over), and returns token_start [B + 1] for attn_paged_append.

    free_pages (int32) is a ring of free page numbers, free_state [2] int32 the
    position of its first and their number; free_out gets the new state and lens
    [B] is the tokens before the step (None: both in place).  slots (int64) gets
    each new row's slot in the cache, page * page_size + place, or -1 behind the
    last.  rows is the most new tokens there may be (None: slots' size, or one
    per sequence).  With a window (and sinks) a sequence keeps the pages that
    they need and writes them again in turns.  A step that cannot be done whole is
    not done at all, and sync_status() says so: too few free pages or rows, a
    length or count out of range, or a ring without room for the pages that are free
    before the step and those that come back in it (one of all pages has it)."""
    return _paged_call("assign", kv, stream, n_new, free_pages, free_state, lens, free_out, token_start, slots, rows, window,
                       sinks)


def _window_call(name, q, stream, *args):
    f = getattr(_native_module or _native(), name)
    if stream is None or not isinstance(q, torch.Tensor):
        r = f(q, *args)
    else:
        with _OnStream(q, stream):
            r = f(q, *args)
    if type(r) is int:
        raise AttnError("attn_" + name, r)
    return r


def attn_fwd_window(q, k, v, window, sinks=0, scale=None, o=None, lse=None, stream=None):
    """Causal attention with a sliding window: q [B, q_heads, Nq, d] are the last
    Nq of the Nk positions of k, v [B, kv_heads, Nk, d]; the query at position p
    sees the keys p - window + 1 .. p and the first ``sinks`` ones up to p.  Query heads
    in groups of q_heads / kv_heads share a key/value head.  bf16 or fp16, any
    strides whose channels are contiguous and whose rows do not overlap.
    Returns (o, lse); o is dense, token-major where q is."""
    return _window_call("fwd_window", q, stream, k, v, window, sinks, scale, o, lse)


def attn_bwd_window(q, k, v, o, do, lse, window, sinks=0, scale=None, dq=None, dk=None, dv=None, stream=None):
    """Gradients of attn_fwd_window's output for the same window, sinks and scale,
    dk and dv summed over the query heads of a key/value head.  Returns (dq, dk, dv)."""
    return _window_call("bwd_window", q, stream, k, v, o, do, lse, window, sinks, scale, dq, dk, dv)


def _check_block_mask(block_mask, H, N):
    nb = (N + 127) // 128
    if (not isinstance(block_mask, torch.Tensor) or not block_mask.is_cuda or block_mask.dtype != torch.uint8
            or not block_mask.is_contiguous() or block_mask.dim() != 3
            or tuple(block_mask.shape[1:]) != (nb, nb) or block_mask.shape[0] not in (1, H)):
        raise ValueError("block_mask must be a contiguous uint8 CUDA tensor [H or 1, %d, %d]" % (nb, nb))


def _fwd_blocksparse(name, q, k, v, block_mask, scale, causal, o, lse, stream, drop=None):
    B, H, N, d = _dims(q)
    _check("q", q)
    _check("k", k, q, q.dtype)
    _check("v", v, q, q.dtype)
    _check_block_mask(block_mask, H, N)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _check("o", o, q, q.dtype)
    _check("lse", lse, None, torch.float32)
    args = [q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
            block_mask.data_ptr(), int(block_mask.shape[0]), B, H, N, d, float(scale), int(bool(causal))]
    if drop is not None:
        p_drop, seed, offset = drop
        args += [float(p_drop), int(seed) & 0xFFFFFFFFFFFFFFFF, int(offset) & 0xFFFFFFFF]
    with _on_device(q):
        fn = getattr(lib(), name if q.dtype == torch.bfloat16 else name + "_f16")
        rc = fn(*args, _stream_handle(stream))
    if rc:
        raise AttnError(name, rc)
    return o, lse


def _bwd_blocksparse(name, q, k, v, o, do, lse, block_mask, scale, causal, dq, dk, dv, stream, drop=None):
    B, H, N, d = _dims(q)
    _check("q", q)
    for n, t in (("k", k), ("v", v), ("o", o), ("do", do)):
        _check(n, t, q, q.dtype)
    _check("lse", lse, None, torch.float32)
    _check_block_mask(block_mask, H, N)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check(n, t, q, q.dtype)
    args = [q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), block_mask.data_ptr(), int(block_mask.shape[0]),
            B, H, N, d, float(scale), int(bool(causal))]
    if drop is not None:
        p_drop, seed, offset = drop
        args += [float(p_drop), int(seed) & 0xFFFFFFFFFFFFFFFF, int(offset) & 0xFFFFFFFF]
    with _on_device(q):
        fn = getattr(lib(), name if q.dtype == torch.bfloat16 else name + "_f16")
        rc = fn(*args, _stream_handle(stream))
    if rc:
        raise AttnError(name, rc)
    return dq, dk, dv


def attn_fwd_blocksparse(q, k, v, block_mask, scale=None, causal=False, o=None, lse=None, stream=None):
    """Forward restricted by a block mask: block_mask is a uint8 CUDA tensor
    [H or 1, ceil(N/128), ceil(N/128)]; key j is visible to query i iff
    block_mask[h][i // 128][j // 128] != 0 (and j <= i if causal).
    bf16 or fp16.  Returns (o, lse); rows that see no key get O = 0,
    LSE = -inf."""
    return _fwd_blocksparse("attn_fwd_blocksparse", q, k, v, block_mask, scale, causal, o, lse, stream)


def attn_bwd_blocksparse(q, k, v, o, do, lse, block_mask, scale=None, causal=False, dq=None, dk=None, dv=None,
                         stream=None):
    """Gradients of attn_fwd_blocksparse's output for the same block_mask and
    causal flag.  Returns (dq, dk, dv)."""
    return _bwd_blocksparse("attn_bwd_blocksparse", q, k, v, o, do, lse, block_mask, scale, causal, dq, dk, dv,
                            stream)


def attn_fwd_blocksparse_dropout(q, k, v, block_mask, p_drop, seed, offset=0, scale=None, causal=False, o=None,
                                 lse=None, stream=None):
    """attn_fwd_blocksparse with the dropout of attn_fwd_dropout on the keys
    the mask leaves visible (the keep decisions do not depend on the mask).
    Returns (o, lse); lse is that of the undropped softmax."""
    return _fwd_blocksparse("attn_fwd_blocksparse_dropout", q, k, v, block_mask, scale, causal, o, lse, stream,
                            (p_drop, seed, offset))


def attn_bwd_blocksparse_dropout(q, k, v, o, do, lse, block_mask, p_drop, seed, offset=0, scale=None,
                                 causal=False, dq=None, dk=None, dv=None, stream=None):
    """Gradients of attn_fwd_blocksparse_dropout's output (same mask, causal
    flag, p_drop, seed, offset).  Returns (dq, dk, dv)."""
    return _bwd_blocksparse("attn_bwd_blocksparse_dropout", q, k, v, o, do, lse, block_mask, scale, causal,
                            dq, dk, dv, stream, (p_drop, seed, offset))


def attn_fwd_fp8(q, k, v, descale_q, descale_k, descale_v, scale=None, causal=False, o=None, lse=None,
                 stream=None):
    """Forward with e4m3 inputs (torch.float8_e4m3fn or uint8 views) and
    per-tensor descale factors.  Returns (o bf16, lse fp32)."""
    if q.dim() != 4:
        raise ValueError("q must be [B, H, N, d]")
    B, H, N, d = (int(x) for x in q.shape)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(name, t, q)
        if t.element_size() != 1:
            raise TypeError("%s must hold one-byte e4m3 values" % name)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q.device) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _check("o", o, None, torch.bfloat16)
    _check("lse", lse, None, torch.float32)
    with _on_device(q):
        rc = lib().attn_fwd_fp8(q.data_ptr(), k.data_ptr(), v.data_ptr(), float(descale_q), float(descale_k),
                                float(descale_v), o.data_ptr(), lse.data_ptr(), B, H, N, d, float(scale),
                                int(bool(causal)), _stream_handle(stream))
    if rc:
        raise AttnError("attn_fwd_fp8", rc)
    return o, lse


class _Attention(torch.autograd.Function):
    """Differentiable exact attention: forward through attn_fwd (or its
    dropout / block-mask variants), backward through the matching attn_bwd*
    from the saved O and LSE (P is recomputed, never stored)."""

    @staticmethod
    def forward(ctx, q, k, v, scale, causal, p_drop, seed, offset, block_mask):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        if block_mask is not None and p_drop > 0.0:
            o, lse = attn_fwd_blocksparse_dropout(q, k, v, block_mask, p_drop, seed, offset, scale=scale,
                                                  causal=causal)
        elif block_mask is not None:
            o, lse = attn_fwd_blocksparse(q, k, v, block_mask, scale=scale, causal=causal)
        elif p_drop > 0.0:
            o, lse = attn_fwd_dropout(q, k, v, p_drop, seed, offset, scale=scale, causal=causal)
        else:
            o, lse = attn_fwd(q, k, v, scale=scale, causal=causal)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.args = (scale, causal, p_drop, seed, offset, block_mask)
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        scale, causal, p_drop, seed, offset, block_mask = ctx.args
        do = do.contiguous()
        if block_mask is not None and p_drop > 0.0:
            dq, dk, dv = attn_bwd_blocksparse_dropout(q, k, v, o, do, lse, block_mask, p_drop, seed, offset,
                                                      scale=scale, causal=causal)
        elif block_mask is not None:
            dq, dk, dv = attn_bwd_blocksparse(q, k, v, o, do, lse, block_mask, scale=scale, causal=causal)
        elif p_drop > 0.0:
            dq, dk, dv = attn_bwd_dropout(q, k, v, o, do, lse, p_drop, seed, offset, scale=scale, causal=causal)
        else:
            dq, dk, dv = attn_bwd(q, k, v, o, do, lse, scale=scale, causal=causal)
        return dq, dk, dv, None, None, None, None, None, None


def _laid_out(t):
    """t, or a contiguous copy where the windowed calls do not take its strides."""
    if t.stride(-1) != 1 or t.data_ptr() % 16:
        return t.contiguous()
    span = t.shape[-1]
    for stride, n in sorted((s, n) for s, n in zip(t.stride()[:-1], t.shape[:-1]) if n > 1):
        if stride % 8 or stride < span:
            return t.contiguous()
        span += stride * (n - 1)
    return t


class _WindowAttention(torch.autograd.Function):
    """Differentiable windowed attention: attn_fwd_window, attn_bwd_window."""

    @staticmethod
    def forward(ctx, q, k, v, scale, window, sinks):
        q, k, v = _laid_out(q), _laid_out(k), _laid_out(v)
        o, lse = attn_fwd_window(q, k, v, window, sinks, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.args = (window, sinks, scale)
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        return attn_bwd_window(q, k, v, o, _laid_out(do), lse, *ctx.args) + (None, None, None)


def attention(q, k, v, scale=None, causal=False, dropout_p=0.0, seed=0, offset=0, block_mask=None, window=None, sinks=0):
    """O = softmax(scale q k^T [+ causal mask]) v as a differentiable op on
    [B, H, N, d] CUDA tensors (bf16 or fp16).  Gradients flow to q, k and v
    through the recomputation backward.  With dropout_p > 0 the keep
    decisions come from (seed, offset); use a new offset per step.  With a
    block_mask (uint8 [H or 1, ceil(N/128), ceil(N/128)] on the device) only
    the enabled 128 x 128 tiles are computed, as in attn_fwd_blocksparse.  With a
    window (causal by itself, without dropout or block mask) a query sees the last
    ``window`` keys and the first ``sinks``; k and v may have fewer heads and more
    positions than q, as in attn_fwd_window."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if window is not None:
        if dropout_p or block_mask is not None:
            raise ValueError("a window goes with neither dropout nor a block mask")
        return _WindowAttention.apply(q, k, v, float(scale), window, sinks)
    if sinks:
        raise ValueError("sinks go with a window")
    return _Attention.apply(q, k, v, float(scale), bool(causal), float(dropout_p), int(seed), int(offset),
                            block_mask)


def sync_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the sticky device status."""
    return lib().attn_sync_status(_stream_handle(stream))
