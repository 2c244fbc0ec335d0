"""ctypes binding of include/fa.h (argument marshalling only).

Every compute step runs in the CUDA library; if it is missing this module
raises instead of falling back to anything else.  torch is used for device
memory and streams only.
"""
from __future__ import annotations

import ctypes
import os
from contextlib import nullcontext
from functools import lru_cache
from operator import itemgetter

from .build import LIB_PATH

FA_BF16, FA_FP16 = 0, 1
FA_BWD_DETERMINISTIC = 1
STATUS = {0: "FA_OK", 1: "FA_ERR_INVALID_VALUE", 2: "FA_ERR_MISALIGNED", 3: "FA_ERR_UNSUPPORTED_DEVICE",
          4: "FA_ERR_CUDA", 5: "FA_ERR_DEVICE_TIMEOUT", 6: "FA_ERR_NO_ALLOC_LIMIT"}
EXPORTS = ("fa_bwd", "fa_bwd_band", "fa_bwd_ex", "fa_bwd_sink", "fa_bwd_sink_workspace", "fa_cache_append", "fa_cache_evict", "fa_cache_fwd", "fa_cache_read",
           "fa_cache_weights", "fa_cache_workspace", "fa_fwd", "fa_fwd_band", "fa_fwd_ex", "fa_fwd_noalloc",
           "fa_fwd_qkv", "fa_fwd_sink", "fa_fwd_sink_workspace", "fa_sync_status", "fa_status_string")
SCHEDULES = {"auto": 0, "whole_tiles": 1, "balanced": 2}

_lib = None


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


def load(path: str = LIB_PATH):
    """Load the CUDA library (raises OSError if it has not been built)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"CUDA library not built: {path} is missing (run exact_attention_10_gb300.build)")
    lib = ctypes.CDLL(path)
    vp, c_int = ctypes.c_void_p, ctypes.c_int
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, ctypes.c_float, c_int, vp]
    lib.fa_fwd.restype = c_int
    lib.fa_fwd_ex.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, ctypes.c_float, c_int, c_int, vp]
    lib.fa_fwd_ex.restype = c_int
    lib.fa_fwd_noalloc.argtypes = lib.fa_fwd_ex.argtypes
    lib.fa_fwd_noalloc.restype = c_int
    lib.fa_fwd_qkv.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, ctypes.c_float, c_int,
                               c_int, vp]
    lib.fa_fwd_qkv.restype = c_int
    lib.fa_fwd_band.argtypes = [vp, vp, vp, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, c_int, ctypes.c_float,
                                c_int, c_int, vp]
    lib.fa_fwd_band.restype = c_int
    lib.fa_bwd.argtypes = [vp] * 9 + [c_int] * 5 + [ctypes.c_float, c_int, vp]
    lib.fa_bwd.restype = c_int
    lib.fa_bwd_band.argtypes = [vp] * 9 + [c_int] * 7 + [ctypes.c_float, c_int, vp]
    lib.fa_bwd_band.restype = c_int
    lib.fa_bwd_ex.argtypes = [vp] * 9 + [c_int] * 7 + [ctypes.c_float, c_int, ctypes.c_uint, vp]
    lib.fa_bwd_ex.restype = c_int
    lib.fa_fwd_sink.argtypes = [vp] * 5 + [c_int] * 8 + [ctypes.c_float, c_int, c_int, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_sink.restype = c_int
    lib.fa_fwd_sink_workspace.argtypes = [c_int] * 9 + [ctypes.POINTER(ctypes.c_size_t)]
    lib.fa_fwd_sink_workspace.restype = c_int
    lib.fa_bwd_sink.argtypes = [vp] * 9 + [c_int] * 8 + [ctypes.c_float, c_int, ctypes.c_uint, vp, ctypes.c_size_t, vp]
    lib.fa_bwd_sink.restype = c_int
    lib.fa_bwd_sink_workspace.argtypes = [c_int] * 8 + [ctypes.c_uint, ctypes.POINTER(ctypes.c_size_t)]
    lib.fa_bwd_sink_workspace.restype = c_int
    lib.fa_cache_append.argtypes = [vp] * 8 + [c_int] * 6 + [vp]
    lib.fa_cache_append.restype = c_int
    lib.fa_cache_read.argtypes = [vp] * 8 + [c_int] * 6 + [vp]
    lib.fa_cache_read.restype = c_int
    lib.fa_cache_workspace.argtypes = [c_int] * 6 + [ctypes.POINTER(ctypes.c_size_t)]
    lib.fa_cache_workspace.restype = c_int
    lib.fa_cache_fwd.argtypes = [vp] * 8 + [c_int] * 8 + [ctypes.c_float, c_int, vp, ctypes.c_size_t, vp]
    lib.fa_cache_fwd.restype = c_int
    lib.fa_cache_weights.argtypes = [vp] * 6 + [c_int] * 9 + [ctypes.c_float, c_int, vp]
    lib.fa_cache_weights.restype = c_int
    lib.fa_cache_evict.argtypes = [vp] * 13 + [c_int] * 8 + [vp]
    lib.fa_cache_evict.restype = c_int
    lib.fa_sync_status.argtypes = [vp]
    lib.fa_sync_status.restype = c_int
    lib.fa_status_string.argtypes = [c_int]
    lib.fa_status_string.restype = ctypes.c_char_p
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load().fa_status_string(int(status)).decode()
    except OSError:
        return "library not loaded"


def fwd_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, B: int, H: int, N: int, D: int,
            causal: int, scale: float, dtype: int, stream: int = 0, schedule: int | None = None) -> int:
    """Call fa_fwd (or fa_fwd_ex with a schedule code) with raw integer
    pointers; returns the status code unchanged."""
    if schedule is None:
        return load().fa_fwd(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, N, D, causal, scale, dtype, stream)
    return load().fa_fwd_ex(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, N, D, causal, scale, dtype, schedule, stream)


def sync_status(stream: int = 0) -> int:
    return load().fa_sync_status(stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float16:
        return FA_FP16
    raise TypeError(f"fa_fwd takes bfloat16 or float16 tensors, got {t.dtype}")


def _on(stream, t):
    """Where a call on ``stream`` (None: torch's current one) has torch allocate
    its results and workspace: on that very stream, so that no earlier work of
    another stream still uses the memory, and what is dropped after the call is
    handed on to later work of the same stream only."""
    if stream is None:
        return nullcontext()
    import torch
    if not isinstance(stream, torch.cuda.Stream):   # a handle, or another library's stream with one
        stream = torch.cuda.ExternalStream(_stream_of(stream, t), device=t.device)
    return torch.cuda.stream(stream)


def _workspace(nbytes: int, t):
    """Device memory from torch's allocator (None: none needed)."""
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=t.device) if nbytes else None


def forward(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None, stream=None,
            schedule: str = "auto", window: tuple[int, int] | None = None, sinks: int | None = None):
    """Attention forward on CUDA tensors q [B, H, Nq, D], k and v [B, H, Nkv, D];
    returns (O [B, H, Nq, D], LSE [B, H, Nq]).  With Nq != Nkv the causal mask
    is aligned bottom-right (fa_fwd_qkv).  ``window = (left, right)`` masks
    with a band instead (fa_fwd_band; a negative bound is unbounded; causal
    is ignored then).  With ``sinks`` (0 or more) the mask is the causal
    window (left, 0), without one plain causal, whatever ``causal`` says, in
    which the first ``sinks`` keys stay visible, and k and v may have fewer
    heads, [B, Hkv, Nkv, D] with H a multiple of Hkv (fa_fwd_sink); shared heads
    without sinks take ``sinks=0``, other masks have none.

    ``out`` / ``lse`` may be given to write into existing buffers.
    ``schedule`` is "auto", "whole_tiles" or "balanced" (fa_schedule).
    Raises FAError on any non-OK status.  Asynchronous on ``stream``
    (default: the current torch stream).  In every call here the results that
    are not given are allocated on that stream and belong to it, as in torch:
    another stream waits for it before it uses them (``wait_stream``), and
    holds them by ``record_stream``.
    """
    if sinks is not None:
        return _forward_sink(q, k, v, scale, out, lse, stream, schedule, window, sinks)
    import torch
    if q.dim() != 4 or k.shape != v.shape or k.dim() != 4 or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError("q must be [B, H, Nq, D] and k, v [B, H, Nkv, D]")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous")
    code = _dtype_code(q)
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share a dtype")
    B, H, N, D = q.shape
    if scale is None:
        scale = D ** -0.5
    if out is None or lse is None:
        with _on(stream, q):
            out = torch.empty_like(q) if out is None else out
            lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    st = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if schedule not in SCHEDULES:
        raise ValueError(f"schedule must be one of {sorted(SCHEDULES)}")
    Nkv = k.shape[2]
    if window is not None:
        rc = load().fa_fwd_band(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, N, Nkv,
                                D, int(window[0]), int(window[1]), float(scale), code, SCHEDULES[schedule], st)
    elif Nkv == N:
        rc = fwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, N, D,
                     int(bool(causal)), float(scale), code, st, SCHEDULES[schedule])
    else:
        rc = load().fa_fwd_qkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, N, Nkv,
                               D, int(bool(causal)), float(scale), code, SCHEDULES[schedule], st)
    if rc != 0:
        raise FAError(rc, "fa_fwd")
    return out, lse


@lru_cache(maxsize=4096)
def _sink_workspace(device: int, *sizes) -> int:
    n = ctypes.c_size_t()
    rc = load().fa_fwd_sink_workspace(*sizes, ctypes.byref(n))
    if rc != 0:
        raise FAError(rc, "fa_fwd_sink_workspace")
    return n.value


def _sink_shapes(q, k, v):
    """(B, H, Hkv, Nq, Nkv, D, dtype code) of tensors that go together."""
    sq, sk = q.shape, k.shape
    if len(sq) != 4 or len(sk) != 4 or v.shape != sk or sq[0] != sk[0] or sq[3] != sk[3] or sk[1] < 1 or sq[1] % sk[1]:
        raise ValueError("q must be [B, H, Nq, D] and k, v [B, Hkv, Nkv, D], H a multiple of Hkv")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        raise ValueError("q, k, v must be contiguous")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share a dtype")
    return sq[0], sq[1], sk[1], sq[2], sk[2], sq[3], _dtype_code(q)


def _forward_sink(q, k, v, scale, out, lse, stream, schedule, window, sinks):
    import torch
    B, H, Hkv, Nq, Nkv, D, code = _sink_shapes(q, k, v)
    left = _left_of(window, sinks)
    if schedule not in SCHEDULES:
        raise ValueError(f"schedule must be one of {sorted(SCHEDULES)}")
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous()):
        raise ValueError("out must be contiguous, of q's shape and type")
    if lse is not None and (lse.shape != (B, H, Nq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 [B, H, Nq]")
    sched = SCHEDULES[schedule]
    nbytes = _sink_workspace(q.get_device(), B, H, Hkv, Nq, Nkv, D, left, sinks, sched)
    with _on(stream, q):
        out = torch.empty_like(q) if out is None else out
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
        ws = _workspace(nbytes, q)
    rc = load().fa_fwd_sink(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Hkv, Nq,
                            Nkv, D, left, sinks, D ** -0.5 if scale is None else scale, code, sched,
                            ws.data_ptr() if nbytes else None, nbytes, _stream_of(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_fwd_sink")
    return out, lse


def backward(q, k, v, o, do, lse, causal: bool = False, scale: float | None = None, dq=None, dk=None, dv=None,
             stream=None, window: tuple[int, int] | None = None, deterministic: bool = False, sinks: int | None = None):
    """Attention backward on CUDA tensors: q, o, do [B, H, Nq, D], k, v
    [B, H, Nkv, D] and lse [B, H, Nq] as ``forward`` returned them (same
    causal / window); returns (dQ, dK, dV).  Square unmasked or causal calls
    go to fa_bwd; a window, or Nq != Nkv (bottom-right causal), to fa_bwd_band;
    ``deterministic`` (dQ by the second pass, the same bits on every call) to
    fa_bwd_ex with FA_BWD_DETERMINISTIC; ``sinks`` (k, v [B, Hkv, Nkv, D], the
    mask of ``forward`` with sinks, ``causal`` or not) to fa_bwd_sink.

    ``dq`` / ``dk`` / ``dv`` may be given to write into existing buffers.
    Raises FAError on any non-OK status.  Asynchronous on ``stream``
    (default: the current torch stream).
    """
    if sinks is not None:
        return _backward_sink(q, k, v, o, do, lse, scale, dq, dk, dv, stream, window, deterministic, sinks)
    import torch
    if (q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or o.shape != q.shape or do.shape != q.shape
            or lse.shape != q.shape[:3] or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]):
        raise ValueError("q, o, do must be [B, H, Nq, D], k, v [B, H, Nkv, D] and lse [B, H, Nq]")
    if not all(x.is_contiguous() for x in (q, k, v, o, do, lse)):
        raise ValueError("inputs must be contiguous")
    code = _dtype_code(q)
    if any(x.dtype != q.dtype for x in (k, v, o, do)) or lse.dtype != torch.float32:
        raise TypeError("q, k, v, o, do must share a dtype; lse must be float32")
    B, H, N, D = q.shape
    Nkv = k.shape[2]
    if scale is None:
        scale = D ** -0.5
    if dq is None or dk is None or dv is None:
        with _on(stream, q):
            dq, dk, dv = (torch.empty_like(x) if d is None else d for d, x in ((dq, q), (dk, k), (dv, v)))
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    st = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    ptrs = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr())
    if deterministic:
        left, right = window if window is not None else (-1, 0 if causal else -1)
        rc = load().fa_bwd_ex(*ptrs, B, H, N, Nkv, D, int(left), int(right), float(scale), code, FA_BWD_DETERMINISTIC, st)
    elif window is None and Nkv == N:
        rc = load().fa_bwd(*ptrs, B, H, N, D, int(bool(causal)), float(scale), code, st)
    else:
        left, right = window if window is not None else (-1, 0 if causal else -1)
        rc = load().fa_bwd_band(*ptrs, B, H, N, Nkv, D, int(left), int(right), float(scale), code, st)
    if rc != 0:
        raise FAError(rc, "fa_bwd")
    return dq, dk, dv


@lru_cache(maxsize=4096)
def _sink_bwd_workspace(device: int, *sizes) -> int:
    n = ctypes.c_size_t()
    rc = load().fa_bwd_sink_workspace(*sizes, ctypes.byref(n))
    if rc != 0:
        raise FAError(rc, "fa_bwd_sink_workspace")
    return n.value


def _backward_sink(q, k, v, o, do, lse, scale, dq, dk, dv, stream, window, deterministic, sinks):
    import torch
    B, H, Hkv, Nq, Nkv, D, code = _sink_shapes(q, k, v)
    left = _left_of(window, sinks)
    if o.shape != q.shape or do.shape != q.shape or lse.shape != (B, H, Nq):
        raise ValueError("o, do must be of q's shape and lse [B, H, Nq]")
    if not (o.is_contiguous() and do.is_contiguous() and lse.is_contiguous()):
        raise ValueError("o, do, lse must be contiguous")
    if o.dtype != q.dtype or do.dtype != q.dtype or lse.dtype != torch.float32:
        raise TypeError("o, do must be of q's type, lse float32")
    for d, x in ((dq, q), (dk, k), (dv, v)):
        if d is not None and (d.shape != x.shape or d.dtype != x.dtype or not d.is_contiguous()):
            raise ValueError("dq, dk, dv must be contiguous, of the shapes and type of q, k, v")
    flags = FA_BWD_DETERMINISTIC if deterministic else 0
    nbytes = _sink_bwd_workspace(q.get_device(), B, H, Hkv, Nq, Nkv, D, left, sinks, flags)
    with _on(stream, q):
        outs = [torch.empty_like(x) if d is None else d for d, x in ((dq, q), (dk, k), (dv, v))]
        ws = _workspace(nbytes, q)
    rc = load().fa_bwd_sink(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                            *(d.data_ptr() for d in outs), B, H, Hkv, Nq, Nkv, D, left, sinks,
                            D ** -0.5 if scale is None else scale, code, flags, ws.data_ptr(), nbytes,
                            _stream_of(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_bwd_sink")
    return tuple(outs)


# ---- the 4-bit key/value cache

class PackedCache(tuple):
    """K and V of [B, Hkv, C, D] held in 4 bits: the tensors (k_codes,
    k_params, v_codes, v_params), codes [B, Hkv, C, D/2] uint8 and (scale,
    minimum) [B, Hkv, C, 2] in the model's type (the format is in
    include/fa.h).  Checked when it is made; ``sizes`` is (B, Hkv, C, D, dtype
    code)."""

    k_codes, k_params, v_codes, v_params = (property(itemgetter(i)) for i in range(4))

    def __new__(cls, k_codes, k_params, v_codes, v_params):
        import torch
        shape = k_codes.shape
        if len(shape) != 4 or 0 in shape or v_codes.shape != shape or k_params.shape != v_params.shape or (
                k_params.shape != (*shape[:3], 2)):
            raise ValueError("a cache is codes [B, Hkv, C, D/2] and params [B, Hkv, C, 2] for K and for V, none empty")
        if k_codes.dtype != torch.uint8 or v_codes.dtype != torch.uint8 or k_params.dtype != v_params.dtype:
            raise TypeError("cache codes are uint8, the params of K and V of one type")
        if not (k_codes.is_contiguous() and k_params.is_contiguous() and v_codes.is_contiguous()
                and v_params.is_contiguous()):
            raise ValueError("the cache must be contiguous")
        self = super().__new__(cls, (k_codes, k_params, v_codes, v_params))
        self.sizes = (*shape[:3], 2 * shape[3], _dtype_code(k_params))
        return self

    def __reduce__(self):   # (copying and pickling go through the checks)
        return PackedCache, tuple(self)


def cache_empty(B: int, Hkv: int, C: int, D: int, dtype=None, device="cuda") -> PackedCache:
    """A cache of capacity C for B sequences and Hkv key heads (all codes and
    params zero); ``dtype`` bfloat16 (default) or float16."""
    import torch
    if D not in (64, 128):
        raise ValueError("D must be 64 or 128")
    dtype = torch.bfloat16 if dtype is None else dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"a cache is of bfloat16 or float16, got {dtype}")
    return PackedCache(*(torch.zeros((B, Hkv, C, n), dtype=t, device=device)
                         for n, t in ((D // 2, torch.uint8), (2, dtype)) * 2))


def _ints(t, B: int, name: str) -> int:
    import torch
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.dim() != 1 or t.numel() != B or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{B}]")
    return t.data_ptr()


def _stream_of(stream, t) -> int:
    """The stream's handle; None: torch's current stream on t's device (asked
    for as a plain number: a Stream object would cost more than the launch)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(t.get_device()) if t.is_cuda else 0
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _left_of(window, sinks) -> int:
    """window_left of ``window`` = (left, 0) or None (no window)."""
    if not 0 <= sinks <= 0x7FFFFFFF:
        raise ValueError("sinks must be a 32-bit count")
    if window is None:
        return -1
    if window[1] != 0:
        raise ValueError("this attention is causal: window must be (left, 0)")
    return max(-1, min(int(window[0]), 0x7FFFFFFF))


def cache_append(cache: PackedCache, k, v, start, count=None, stream=None) -> None:
    """Pack tokens k, v [B, Hkv, N, D] into the cache at positions start[b] + i
    (``start`` int32 [B]); with ``count`` (int32 [B]) only the first count[b]
    of a sequence.  Tokens whose place lies outside the cache are not written.
    Raises FAError on any non-OK status.  Asynchronous on ``stream``
    (default: the current torch stream)."""
    kc, kp, vc, vp = cache
    B, Hkv, C, D, code = cache.sizes
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or shape[0] != B or shape[1] != Hkv or shape[3] != D:
        raise ValueError(f"k, v must be [{B}, {Hkv}, N, {D}]")
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k, v must be contiguous")
    if k.dtype != kp.dtype or v.dtype != k.dtype:
        raise TypeError("k, v must be of the cache's type")
    rc = load().fa_cache_append(kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(), k.data_ptr(), v.data_ptr(),
                                _ints(start, B, "start"), None if count is None else _ints(count, B, "count"), B, Hkv,
                                shape[2], C, D, code, _stream_of(stream, k))
    if rc != 0:
        raise FAError(rc, "fa_cache_append")


def cache_read(cache: PackedCache, start, n: int, count=None, stream=None):
    """The values (k, v) [B, Hkv, n, D] that cache tokens start[b] + i stand
    for; rows from count[b] on, or outside the cache, are zeros.
    Asynchronous on ``stream``, which the results belong to (see ``forward``)."""
    if not 1 <= n <= 0x7FFFFFFF:
        raise ValueError("n must be a 32-bit count of at least 1")
    kc, kp, vc, vp = cache
    B, Hkv, C, D, code = cache.sizes
    import torch
    with _on(stream, kp):
        k = torch.empty((B, Hkv, n, D), dtype=kp.dtype, device=kp.device)
        v = torch.empty_like(k)
    rc = load().fa_cache_read(kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(), k.data_ptr(), v.data_ptr(),
                              _ints(start, B, "start"), None if count is None else _ints(count, B, "count"), B, Hkv, n,
                              C, D, code, _stream_of(stream, k))
    if rc != 0:
        raise FAError(rc, "fa_cache_read")
    return k, v


@lru_cache(maxsize=4096)
def _cache_workspace(device: int, *sizes) -> int:
    n = ctypes.c_size_t()
    rc = load().fa_cache_workspace(*sizes, ctypes.byref(n))
    if rc != 0:
        raise FAError(rc, "fa_cache_workspace")
    return n.value


def _cache_queries(q, cache):
    """(H, Nq) of queries that go with the cache."""
    B, Hkv, _, D, _ = cache.sizes
    shape = q.shape
    if len(shape) != 4 or shape[0] != B or shape[3] != D or shape[1] % Hkv != 0:
        raise ValueError(f"q must be [{B}, a multiple of {Hkv}, Nq, {D}]")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    if q.dtype != cache.k_params.dtype:
        raise TypeError("q must be of the cache's type")
    return shape[1], shape[2]


def cache_forward(q, cache: PackedCache, lens, window: tuple[int, int] | None = None, sinks: int = 0,
                  scale: float | None = None, out=None, lse=None, stream=None):
    """Attention of each sequence's last Nq tokens, q [B, H, Nq, D], against
    the cache's first lens[b] tokens (theirs among them; ``lens`` int32 [B]);
    H / Hkv query heads share a key head.  Returns (O [B, H, Nq, D], LSE
    [B, H, Nq]).  ``window = (left, 0)`` limits query position p to tokens
    from p - left on, but for the first ``sinks`` tokens, which stay visible.

    Raises FAError on any non-OK status.  Asynchronous on ``stream``
    (default: the current torch stream), which the results that are not given
    belong to (see ``forward``).
    """
    import torch
    kc, kp, vc, vp = cache
    B, Hkv, C, D, code = cache.sizes
    H, Nq = _cache_queries(q, cache)
    left = _left_of(window, sinks)
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous()):
        raise ValueError("out must be contiguous, of q's shape and type")
    if lse is not None and (lse.shape != (B, H, Nq) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 [B, H, Nq]")
    nbytes = _cache_workspace(q.get_device(), B, H, Hkv, Nq, C, D)
    with _on(stream, q):
        out = torch.empty_like(q) if out is None else out
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
        ws = _workspace(nbytes, q)
    rc = load().fa_cache_fwd(q.data_ptr(), kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(),
                             _ints(lens, B, "lens"), out.data_ptr(), lse.data_ptr(), B, H, Hkv, Nq, C, D, left, sinks,
                             D ** -0.5 if scale is None else scale, code, ws.data_ptr() if nbytes else None, nbytes,
                             _stream_of(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_cache_fwd")
    return out, lse


def cache_weights(q, cache: PackedCache, lse, lens, window: tuple[int, int] | None = None, sinks: int = 0,
                  scale: float | None = None, acc=None, stream=None):
    """What each cached token weighs in ``cache_forward`` of the same arguments
    (``lse`` as it returned it): [B, Hkv, C] float32, the sum over a key
    head's query rows of exp(scale q.k - lse).  With ``acc`` ([B, Hkv, C]
    float32) the weights are added to it in place, and it is returned.
    Asynchronous on ``stream``, which a result that is not given belongs to (see
    ``forward``)."""
    import torch
    kc, kp = cache[:2]
    B, Hkv, C, D, code = cache.sizes
    H, Nq = _cache_queries(q, cache)
    left = _left_of(window, sinks)
    if lse.shape != (B, H, Nq) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous [B, H, Nq]")
    if lse.dtype != torch.float32 or (acc is not None and acc.dtype != torch.float32):
        raise TypeError("lse and acc must be float32")
    if acc is None:
        with _on(stream, q):
            out = torch.empty((B, Hkv, C), dtype=torch.float32, device=q.device)
    elif acc.shape != (B, Hkv, C) or not acc.is_contiguous():
        raise ValueError("acc must be contiguous [B, Hkv, C]")
    else:
        out = acc
    rc = load().fa_cache_weights(q.data_ptr(), kc.data_ptr(), kp.data_ptr(), lse.data_ptr(), _ints(lens, B, "lens"),
                                 out.data_ptr(), int(acc is not None), B, H, Hkv, Nq, C, D, left, sinks,
                                 D ** -0.5 if scale is None else scale, code, _stream_of(stream, q))
    if rc != 0:
        raise FAError(rc, "fa_cache_weights")
    return out


def cache_evict(cache: PackedCache, acc, lens, keep: int, sinks: int = 0, recent: int = 0,
                out: PackedCache | None = None, stream=None):
    """Bring every sequence down to at most ``keep`` tokens per key head: the
    first ``sinks``, the last ``recent`` and the heaviest by ``acc`` [B, Hkv,
    C] float32 between them (ties: the lowest position first), in order.

    Returns (cache, acc, lens, index): another cache (``out``, of any capacity
    from ``keep`` on, or a new one of capacity ``keep``), the kept tokens'
    weights [B, Hkv, capacity] (0 behind them), the new lengths [B] and the
    kept positions [B, Hkv, keep] (-1 behind them).

    The kept tokens move together: in the new cache positions, lengths, windows
    and sinks count them alone (a window hides the kept tokens before it; none
    sees them all).  A new cache is full once a sequence was cut; to append to
    it, give ``out`` a capacity with room (two caches in turn).  Asynchronous on
    ``stream``, which the results belong to (see ``forward``)."""
    import torch
    kc, kp, vc, vp = cache
    B, Hkv, C, D, code = cache.sizes
    if acc.shape != (B, Hkv, C) or not acc.is_contiguous():
        raise ValueError("acc must be contiguous [B, Hkv, C]")
    if acc.dtype != torch.float32:
        raise TypeError("acc must be float32")
    if not 1 <= keep <= 0x7FFFFFFF or sinks < 0 or recent < 0 or sinks + recent > keep:
        raise ValueError("keep must be at least 1 and hold the sinks and the recent tokens")
    if out is None:   # (its rows behind the last kept token are not written)
        with _on(stream, kc):
            codes = torch.empty((B, Hkv, keep, D // 2), dtype=torch.uint8, device=kc.device)
            params = torch.empty((B, Hkv, keep, 2), dtype=kp.dtype, device=kc.device)
            out = PackedCache(codes, params, torch.empty_like(codes), torch.empty_like(params))
    kc2, kp2, vc2, vp2 = out
    B2, Hkv2, C2, D2, code2 = out.sizes
    if (B2, Hkv2, D2, code2) != (B, Hkv, D, code) or C2 < keep:
        raise ValueError("out must be a cache like the first one, of capacity keep at least")
    with _on(stream, kc):
        acc2 = torch.empty((B, Hkv, C2), dtype=torch.float32, device=kc.device)
        lens2 = torch.empty_like(lens)
        index = torch.empty((B, Hkv, keep), dtype=torch.int32, device=kc.device)
    rc = load().fa_cache_evict(kc.data_ptr(), kp.data_ptr(), vc.data_ptr(), vp.data_ptr(), acc.data_ptr(),
                               _ints(lens, B, "lens"), kc2.data_ptr(), kp2.data_ptr(), vc2.data_ptr(), vp2.data_ptr(),
                               acc2.data_ptr(), lens2.data_ptr(), index.data_ptr(), B, Hkv, C, C2, D, keep, sinks,
                               recent, _stream_of(stream, acc))
    if rc != 0:
        raise FAError(rc, "fa_cache_evict")
    return out, acc2, lens2, index
