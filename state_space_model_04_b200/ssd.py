"""Python binding of libssd_b200.so (argument marshalling only).

Every step of the SSD prefill and decode runs in the library's sm_100a kernels; this
module checks tensor dtypes/devices/shapes, allocates outputs and workspaces with torch
(device memory and streams are the only things torch provides) and forwards raw
pointers to the C ABI declared in include/ssd.h.  There is no CPU fallback: if the
library is missing or a call fails, an exception is raised.

Calls run on the current stream, or on `stream`: a torch.cuda.Stream or a raw handle.  What such a call
allocates belongs to that stream; the order between it and the current one, for the operands going in and
the results coming out, is the caller's.  Nothing here takes part in autograd: results carry no graph, and
the backward functions are calls of their own.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssd_b200.so")

SSD_OK = 0
SSD_F32, SSD_BF16 = 0, 1
SSD_ACT_NONE, SSD_ACT_SILU = 0, 1

_i = ctypes.c_int
_ll = ctypes.c_longlong
_sz = ctypes.c_size_t
_vp = ctypes.c_void_p
_INT_MAX = 2**31 - 1  # ctypes cuts larger numbers short


class SSDError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__("%s failed: status %d (%s) %s" % (where, status, status_string(status), detail))
        self.status = status


class _KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int), ("total_ms", ctypes.c_double)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libssd_b200.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libssd_b200.so is not built: run `python -m state_space_model_04_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.ssd_version.restype = _i
        L.ssd_status_string.argtypes = [_i]
        L.ssd_status_string.restype = ctypes.c_char_p
        L.ssd_last_error.restype = ctypes.c_char_p
        L.ssd_prefill_workspace_size.argtypes = [_i] * 8
        L.ssd_prefill_workspace_size.restype = _sz
        L.ssd_prefill.argtypes = [_i] * 8 + [_vp] * 10 + [_sz, _vp]
        L.ssd_prefill.restype = _i
        L.ssd_prefill_dt_raw.argtypes = [_i] * 8 + [_vp] * 3 + [ctypes.c_float] * 2 + [_vp] * 8 + [_sz, _vp]
        L.ssd_prefill_dt_raw.restype = _i
        L.ssd_prefill_check.argtypes = [_vp, _vp]
        L.ssd_prefill_check.restype = _i
        L.ssd_debug_starve_next_prefill.argtypes = [ctypes.c_ulonglong]
        L.ssd_debug_starve_next_prefill.restype = _i
        L.ssd_debug_starve_next_prefill_backward.argtypes = [ctypes.c_ulonglong]
        L.ssd_debug_starve_next_prefill_backward.restype = _i
        L.ssd_debug_lag_next_prefill_backward.argtypes = [_i]
        L.ssd_debug_lag_next_prefill_backward.restype = _i
        L.ssd_prefill_local_state_workspace_size.argtypes = [_i] * 7
        L.ssd_prefill_local_state_workspace_size.restype = _sz
        L.ssd_prefill_local_state.argtypes = [_i] * 7 + [_vp] * 7 + [_sz, _vp]
        L.ssd_prefill_local_state.restype = _i
        L.ssd_prefill_context_scan.argtypes = [_i] * 6 + [_vp] * 5
        L.ssd_prefill_context_scan.restype = _i
        L.ssd_prefill_segments.argtypes = [_i] * 8
        L.ssd_prefill_segments.restype = _i
        L.ssd_prefill_whole_units.argtypes = [_i] * 8
        L.ssd_prefill_whole_units.restype = _i
        L.ssd_debug_decay_precision.argtypes = [_i]
        L.ssd_debug_decay_precision.restype = _i
        L.ssd_debug_force_prefill_split.argtypes = [_i, _i]
        L.ssd_debug_force_prefill_split.restype = _i
        L.ssd_debug_force_prefill_segments.argtypes = [_i]
        L.ssd_debug_force_prefill_segments.restype = _i
        L.ssd_debug_force_fma_prefill.argtypes = [_i]
        L.ssd_debug_force_fma_prefill.restype = _i
        L.ssd_decode_workspace_size.argtypes = [_i] * 3
        L.ssd_decode_workspace_size.restype = _sz
        L.ssd_decode_step.argtypes = [_i] * 9 + [_vp] * 10 + [_sz, _vp]
        L.ssd_decode_step.restype = _i
        L.ssd_decode_plan_create.argtypes = [ctypes.POINTER(_vp)] + [_i] * 9 + [_vp] * 4 + [_i] + [_vp] * 5 + [_i, _vp, _sz]
        L.ssd_decode_plan_create.restype = _i
        L.ssd_decode_plan_launch.argtypes = [_vp, _vp]
        L.ssd_decode_plan_launch.restype = _i
        L.ssd_decode_plan_destroy.argtypes = [_vp]
        L.ssd_decode_plan_destroy.restype = _i
        L.ssd_decode_loop.argtypes = [_i] * 9 + [_vp] * 4 + [_i] + [_vp] * 5 + [_i, _vp, _sz, _vp]
        L.ssd_decode_loop.restype = _i
        L.ssd_decode_step_noalloc.argtypes = [_i] * 9 + [_vp] * 10
        L.ssd_decode_step_noalloc.restype = _i
        f = ctypes.c_float
        L.ssd_prefill_backward_workspace_size.argtypes = [_i] * 7
        L.ssd_prefill_backward_workspace_size.restype = _sz
        L.ssd_prefill_backward.argtypes = [_i] * 7 + [_vp] * 17 + [_sz, _vp]
        L.ssd_prefill_backward.restype = _i
        L.ssd_prefill_backward_dt_raw.argtypes = [_i] * 7 + [_vp] * 4 + [f] * 2 + [_vp] * 15 + [_sz, _vp]
        L.ssd_prefill_backward_dt_raw.restype = _i
        mat = [_vp, _ll]  # pointer, row stride
        L.ssd_norm_backward_workspace_size.argtypes = [_ll, _i, _i]
        L.ssd_norm_backward_workspace_size.restype = _sz
        L.ssd_residual_norm.argtypes = [_ll, _i, _i, _i] + mat * 2 + [f, _vp, f] + mat * 2 + [_vp]
        L.ssd_residual_norm.restype = _i
        L.ssd_residual_norm_backward.argtypes = ([_ll, _i, _i, _i] + mat * 2 + [_vp] + mat + [f, f] + mat * 2 +
                                                 [_vp, _vp, _sz, _vp])
        L.ssd_residual_norm_backward.restype = _i
        L.ssd_gated_norm.argtypes = [_ll] + [_i] * 4 + mat * 2 + [_vp, f] + mat + [_vp]
        L.ssd_gated_norm.restype = _i
        L.ssd_gated_norm_backward.argtypes = [_ll] + [_i] * 4 + mat * 3 + [_vp, f] + mat * 2 + [_vp, _vp, _sz, _vp]
        L.ssd_gated_norm_backward.restype = _i
        L.ssd_launch_count.restype = ctypes.c_uint64
        L.ssd_profile_begin.restype = _i
        L.ssd_profile_end.argtypes = [ctypes.POINTER(_KernelTime), _i]
        L.ssd_profile_end.restype = _i
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ssd_status_string(int(status)).decode()


def last_error() -> str:
    return lib().ssd_last_error().decode()


def launch_count() -> int:
    """Kernels the library has enqueued in this process (decode plans count their steps)."""
    return int(lib().ssd_launch_count())


def profile_begin():
    """Start bracketing every library kernel launch with CUDA events on its stream."""
    _check(lib().ssd_profile_begin(), "ssd_profile_begin")


def profile_end(max_entries=64):
    """Stop and return {kernel name: (launches, summed event milliseconds)}."""
    buf = (_KernelTime * max_entries)()
    n = lib().ssd_profile_end(buf, max_entries)
    if n < 0:
        _check(-n, "ssd_profile_end")
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(n)}


def _check_device(device, **tensors):
    """Every tensor of one call must sit on the GPU of its first operand, and that GPU must be
    the current device: the library launches there and its kernels read these pointers
    directly (a tensor on another GPU would be a peer address)."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError("%s is on %s, the call's other tensors on %s" % (name, t.device, device))
    if device.type == "cuda" and device.index is not None and device.index != torch.cuda.current_device():
        raise ValueError("the tensors are on %s but the current device is cuda:%d (call under "
                         "torch.cuda.device(...))" % (device, torch.cuda.current_device()))


def _check(status: int, where: str):
    if status != SSD_OK:
        raise SSDError(status, where, last_error())


def _ptr(t):
    return None if t is None else t.data_ptr()


# the current stream's handle without building a torch.cuda.Stream (4.7 us of host time a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _checked_stream(first, **others):
    """The current stream, after _check_device: the device numbers are compared first, as small calls
    are bound by the host's time."""
    dev = first.get_device()
    same = dev == torch.cuda.current_device()
    for t in others.values():
        same = same and (t is None or t.get_device() == dev)
    if not same:
        _check_device(first.device, **others)
    return _raw_stream(dev) if _raw_stream is not None else _stream(None)


def _on(stream, call, *args):
    """call(*args) on a stream given by name.  What the call allocates, its workspace and its results,
    comes from that stream's memory: a block of the current stream's could still be in use by work queued
    there, and would be handed out there again while the call runs.  The results are handed over to the
    current stream, so that they may be dropped with its work on them still queued."""
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle == _stream(None):
        return call(*args)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    here = torch.cuda.current_stream()
    torch.cuda.set_stream(stream)
    try:
        results = call(*args)
    finally:
        torch.cuda.set_stream(here)
    for t in results if isinstance(results, tuple) else (results,):
        if t is not None:
            t.record_stream(here)
    return results


def _io(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    if t.dtype == torch.float32:
        return SSD_F32
    raise TypeError("io tensors must be bfloat16 or float32, got %s" % t.dtype)


def _need(t, name, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return t


def prefill_workspace_size(b, T, H, P, N, G, chunk, io_dtype) -> int:
    return int(lib().ssd_prefill_workspace_size(b, T, H, P, N, G, chunk, io_dtype))


def prefill(x, dt, A, B, C, D, chunk=256, h0=None, y=None, h_final=None, workspace=None,
            want_final=True, stream=None, check=False, dt_raw=False, dt_bias=None, dt_min=0.0,
            dt_max=float("inf")):
    """Chunked SSD prefill.  Shapes: x [b,T,H,P], dt [b,T,H] f32, A [H] f32,
    B/C [b,T,G,N], D [H] f32, h0 [b,H,P,N] f32 or None.  Returns (y, h_final).
    dt_raw=True passes dt as the raw step (ssd_prefill_dt_raw): the kernels form
    clamp(softplus(dt + dt_bias[h]), dt_min, dt_max) themselves; dt_bias [H] f32 or None.
    check=True synchronises and raises if a device-side wait recorded an error."""
    if stream is not None:
        return _on(stream, prefill, x, dt, A, B, C, D, chunk, h0, y, h_final, workspace, want_final, None, check, dt_raw,
                   dt_bias, dt_min, dt_max)
    _need(x, "x")
    io = _io(x)
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    _need(dt, "dt", torch.float32, (b, T, H))
    _need(A, "A", torch.float32, (H,))
    _need(D, "D", torch.float32, (H,))
    _need(B, "B", x.dtype, (b, T, G, N))
    _need(C, "C", x.dtype, (b, T, G, N))
    if h0 is not None:
        _need(h0, "h0", torch.float32, (b, H, P, N))
    if y is None:
        y = torch.empty_like(x)
    _need(y, "y", x.dtype, x.shape)
    if h_final is None and want_final:
        h_final = torch.empty((b, H, P, N), dtype=torch.float32, device=x.device)
    if h_final is not None:
        _need(h_final, "h_final", torch.float32, (b, H, P, N))
    if dt_bias is not None:
        _need(dt_bias, "dt_bias", torch.float32, (H,))
    need = prefill_workspace_size(b, T, H, P, N, G, chunk, io)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _check_device(x.device, dt=dt, A=A, B=B, C=C, D=D, h0=h0, y=y, h_final=h_final, dt_bias=dt_bias,
                  workspace=workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if dt_raw:
        st = lib().ssd_prefill_dt_raw(b, T, H, P, N, G, int(chunk), io, _ptr(x), _ptr(dt), _ptr(dt_bias),
                                      float(dt_min), float(dt_max), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                      _ptr(h0), _ptr(y), _ptr(h_final), _ptr(workspace), ws_bytes,
                                      _stream(stream))
        _check(st, "ssd_prefill_dt_raw")
    else:
        if dt_bias is not None:
            raise ValueError("dt_bias applies to the raw step only (pass dt_raw=True)")
        st = lib().ssd_prefill(b, T, H, P, N, G, int(chunk), io, _ptr(x), _ptr(dt), _ptr(A), _ptr(B),
                               _ptr(C), _ptr(D), _ptr(h0), _ptr(y), _ptr(h_final), _ptr(workspace),
                               ws_bytes, _stream(stream))
        _check(st, "ssd_prefill")
    if check and workspace is not None:
        prefill_check(workspace, stream)
    return y, h_final


class PrefillGrads(NamedTuple):
    """What prefill_backward returns; dh0 and ddt_bias are None where they were not asked for."""
    dx: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: torch.Tensor
    dh0: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]


def prefill_backward_workspace_size(b, T, H, P, N, G, io_dtype) -> int:
    return int(lib().ssd_prefill_backward_workspace_size(b, T, H, P, N, G, io_dtype))


def prefill_backward(dy, x, dt, A, B, C, D, h0=None, dh_final=None, grads=None, want_dh0=True, workspace=None,
                     stream=None, check=False, dt_raw=False, dt_bias=None, dt_min=0.0, dt_max=float("inf")):
    """Gradients of prefill(x, dt, A, B, C, D, h0=h0, ...) from dy [b,T,H,P], the gradient of y, and
    dh_final [b,H,P,N] f32, that of h_final (None: zero).  Returns PrefillGrads: dx, dB, dC in x's
    type, ddt [b,T,H], dA, dD [H] and dh0 [b,H,P,N] (None with want_dh0=False) in f32.  With
    dt_raw=True, ddt is the gradient of the raw step and ddt_bias [H] that of the bias (None without
    one).  grads: a PrefillGrads whose tensors take the results instead of new ones.
    check=True synchronises and raises if a device-side wait recorded an error."""
    if stream is not None:
        return _on(stream, prefill_backward, dy, x, dt, A, B, C, D, h0, dh_final, grads, want_dh0, workspace, None, check,
                   dt_raw, dt_bias, dt_min, dt_max)
    _need(x, "x")
    io = _io(x)
    b, T, H, P = x.shape
    _need(B, "B", x.dtype)
    G, N = B.shape[2], B.shape[3]
    _need(dy, "dy", x.dtype, x.shape)
    _need(dt, "dt", torch.float32, (b, T, H))
    _need(A, "A", torch.float32, (H,))
    _need(D, "D", torch.float32, (H,))
    _need(B, "B", x.dtype, (b, T, G, N))
    _need(C, "C", x.dtype, (b, T, G, N))
    if h0 is not None:
        _need(h0, "h0", torch.float32, (b, H, P, N))
    if dh_final is not None:
        _need(dh_final, "dh_final", torch.float32, (b, H, P, N))
    if dt_bias is not None:
        if not dt_raw:
            raise ValueError("dt_bias applies to the raw step only (pass dt_raw=True)")
        _need(dt_bias, "dt_bias", torch.float32, (H,))
    if grads is None:
        grads = PrefillGrads(torch.empty_like(x), torch.empty_like(dt), torch.empty_like(A),
                             torch.empty_like(B), torch.empty_like(C), torch.empty_like(D),
                             dt.new_empty((b, H, P, N)) if want_dh0 else None,
                             None if dt_bias is None else torch.empty_like(dt_bias))
    else:
        _need(grads.dx, "dx", x.dtype, x.shape)
        _need(grads.ddt, "ddt", torch.float32, (b, T, H))
        _need(grads.dA, "dA", torch.float32, (H,))
        _need(grads.dB, "dB", x.dtype, B.shape)
        _need(grads.dC, "dC", x.dtype, C.shape)
        _need(grads.dD, "dD", torch.float32, (H,))
        if grads.dh0 is not None:
            _need(grads.dh0, "dh0", torch.float32, (b, H, P, N))
        if grads.ddt_bias is not None:
            if not dt_raw:
                raise ValueError("ddt_bias belongs to the raw step only (pass dt_raw=True)")
            _need(grads.ddt_bias, "ddt_bias", torch.float32, (H,))
    need = prefill_backward_workspace_size(b, T, H, P, N, G, io)
    if workspace is None and need:
        workspace = x.new_empty(need, dtype=torch.uint8)
    dx, ddt, dA, dB, dC, dD, dh0, ddt_bias = grads
    s = _checked_stream(x, dy=dy, dt=dt, A=A, B=B, C=C, D=D, h0=h0, dh_final=dh_final, dt_bias=dt_bias,
                        workspace=workspace, dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=dD, dh0=dh0, ddt_bias=ddt_bias)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    shape = (b, T, H, P, N, G, io, _ptr(dy), _ptr(x), _ptr(dt))
    rest = (_ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(h0), _ptr(dh_final), _ptr(dx), _ptr(ddt))
    sums = (_ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD), _ptr(dh0), _ptr(workspace), ws_bytes, s)
    if dt_raw:
        st = lib().ssd_prefill_backward_dt_raw(*shape, _ptr(dt_bias), float(dt_min), float(dt_max), *rest,
                                               _ptr(ddt_bias), *sums)
        _check(st, "ssd_prefill_backward_dt_raw")
    else:
        st = lib().ssd_prefill_backward(*shape, *rest, *sums)
        _check(st, "ssd_prefill_backward")
    if check and workspace is not None:
        prefill_check(workspace, stream)
    return grads


def prefill_check(workspace, stream=None):
    """Synchronise and raise if the last prefill on `workspace` recorded a device-side error."""
    _check(lib().ssd_prefill_check(_ptr(workspace), _stream(stream)), "ssd_prefill_check")


def debug_starve_next_prefill(wait_limit_s=0.1):
    """Failure-detection test hook: the next tensor-core prefill issues no loads, so its
    bounded waits expire after `wait_limit_s` and prefill_check raises SSD_ERR_TIMEOUT."""
    _check(lib().ssd_debug_starve_next_prefill(int(wait_limit_s * 1e9)), "ssd_debug_starve_next_prefill")


def debug_starve_next_prefill_backward(wait_limit_s=0.1):
    """The same hook for the next tensor-core prefill_backward."""
    _check(lib().ssd_debug_starve_next_prefill_backward(int(wait_limit_s * 1e9)),
           "ssd_debug_starve_next_prefill_backward")


def debug_lag_next_prefill_backward(role):
    """Test hook: one role of warps of the next tensor-core prefill_backward's main pass is held back at
    every item (0 pair, 1 row, 2 MMA issue, 3 ddt, 4 store, 5 load, 6 <h, dh>); the results are the same."""
    _check(lib().ssd_debug_lag_next_prefill_backward(int(role)), "ssd_debug_lag_next_prefill_backward")


def prefill_local_state(x, dt, A, B, h_local=None, log_decay=None, workspace=None, stream=None):
    """The state these tokens leave when started from zero, and their total log decay
    sum(dt * A), per (sequence, head): returns (h_local [b,H,P,N] f32, log_decay [b,H] f32).
    x [b,T,H,P] bf16, dt [b,T,H] f32, A [H] f32, B [b,T,G,N] bf16 (ssd_prefill_local_state)."""
    if stream is not None:
        return _on(stream, prefill_local_state, x, dt, A, B, h_local, log_decay, workspace)
    _need(x, "x", torch.bfloat16)
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    _need(dt, "dt", torch.float32, (b, T, H))
    _need(A, "A", torch.float32, (H,))
    _need(B, "B", x.dtype, (b, T, G, N))
    if h_local is None:
        h_local = torch.empty((b, H, P, N), dtype=torch.float32, device=x.device)
    if log_decay is None:
        log_decay = torch.empty((b, H), dtype=torch.float32, device=x.device)
    _need(h_local, "h_local", torch.float32, (b, H, P, N))
    _need(log_decay, "log_decay", torch.float32, (b, H))
    need = int(lib().ssd_prefill_local_state_workspace_size(b, T, H, P, N, G, SSD_BF16))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _check_device(x.device, dt=dt, A=A, B=B, h_local=h_local, log_decay=log_decay, workspace=workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().ssd_prefill_local_state(b, T, H, P, N, G, SSD_BF16, _ptr(x), _ptr(dt), _ptr(A), _ptr(B),
                                       _ptr(h_local), _ptr(log_decay), _ptr(workspace), ws_bytes, _stream(stream))
    _check(st, "ssd_prefill_local_state")
    return h_local, log_decay


def prefill_context_scan(rank, h_local_all, log_decay_all, h0=None, h_in=None, stream=None):
    """State entering context shard `rank` from the rank-major gathered local states
    [world,b,H,P,N] and log decays [world,b,H] (ssd_prefill_context_scan)."""
    if stream is not None:
        return _on(stream, prefill_context_scan, rank, h_local_all, log_decay_all, h0, h_in)
    world, b, H, P, N = h_local_all.shape
    _need(h_local_all, "h_local_all", torch.float32)
    _need(log_decay_all, "log_decay_all", torch.float32, (world, b, H))
    if h0 is not None:
        _need(h0, "h0", torch.float32, (b, H, P, N))
    if h_in is None:
        h_in = torch.empty((b, H, P, N), dtype=torch.float32, device=h_local_all.device)
    _need(h_in, "h_in", torch.float32, (b, H, P, N))
    _check_device(h_local_all.device, log_decay_all=log_decay_all, h0=h0, h_in=h_in)
    st = lib().ssd_prefill_context_scan(world, int(rank), b, H, P, N, _ptr(h0), _ptr(h_local_all),
                                        _ptr(log_decay_all), _ptr(h_in), _stream(stream))
    _check(st, "ssd_prefill_context_scan")
    return h_in


def prefill_segments(b, T, H, P, N, G, chunk, io_dtype) -> int:
    """Segments per sequence ssd_prefill uses for this shape (1 = one pass; 0 = invalid)."""
    return int(lib().ssd_prefill_segments(b, T, H, P, N, G, chunk, io_dtype))


def prefill_whole_units(b, T, H, P, N, G, chunk, io_dtype) -> int:
    """(Sequence, head) pairs ssd_prefill runs whole for this shape (-1 = invalid); the rest
    are split into prefill_segments(...) segments each."""
    return int(lib().ssd_prefill_whole_units(b, T, H, P, N, G, chunk, io_dtype))


def debug_decay_precision(mode=0):
    """Decay-precision ablation of the tensor-core prefill: 0 fp32 (default), 1 exponentiated
    decay factors rounded to bf16, 2 log-space prefix sums rounded to bf16 before exp."""
    _check(lib().ssd_debug_decay_precision(int(mode)), "ssd_debug_decay_precision")


def debug_force_prefill_split(n_full, nseg):
    """Test hook: the first n_full (sequence, head) units run whole, the rest are split into
    nseg segments (nseg = 0: the cost model)."""
    _check(lib().ssd_debug_force_prefill_split(int(n_full), int(nseg)), "ssd_debug_force_prefill_split")


def debug_force_fma_prefill(on=False):
    """Measurement hook: route every following prefill through the fp32-FMA path, which uses
    the chunk length as given (the tensor-core kernel always evaluates 128-token chunks)."""
    _check(lib().ssd_debug_force_fma_prefill(1 if on else 0), "ssd_debug_force_fma_prefill")


def debug_force_prefill_segments(nseg=0):
    """Test hook: split every following tensor-core prefill into `nseg` sequence segments
    (0 = let the cost model choose)."""
    _check(lib().ssd_debug_force_prefill_segments(int(nseg)), "ssd_debug_force_prefill_segments")


def decode_workspace_size(layers, b, G) -> int:
    return int(lib().ssd_decode_workspace_size(layers, b, G))


def _decode_shapes(h, conv_state, A, D, conv_w, conv_b, G):
    _need(h, "h", torch.float32)
    layers, b, H, P, N = h.shape
    k = conv_w.shape[-1]
    Dc = H * P + 2 * G * N
    _need(conv_state, "conv_state", torch.float32, (layers, b, Dc, k - 1))
    _need(A, "A", torch.float32, (layers, H))
    _need(D, "D", torch.float32, (layers, H))
    _need(conv_w, "conv_w", torch.float32, (layers, Dc, k))
    _need(conv_b, "conv_b", torch.float32, (layers, Dc))
    return layers, b, H, P, N, k, Dc


def decode_step(h, conv_state, xbc, dt, A, D, conv_w, conv_b, G=1, act=SSD_ACT_SILU, y=None,
                workspace=None, stream=None):
    """One decode step for all layers; h and conv_state are updated in place.  Returns y."""
    if stream is not None:
        return _on(stream, decode_step, h, conv_state, xbc, dt, A, D, conv_w, conv_b, G, act, y, workspace)
    layers, b, H, P, N, k, Dc = _decode_shapes(h, conv_state, A, D, conv_w, conv_b, G)
    _need(xbc, "xbc", None, (layers, b, Dc))
    io = _io(xbc)
    _need(dt, "dt", torch.float32, (layers, b, H))
    if y is None:
        y = torch.empty((layers, b, H, P), dtype=xbc.dtype, device=h.device)
    _need(y, "y", xbc.dtype, (layers, b, H, P))
    if workspace is None:
        workspace = torch.empty(decode_workspace_size(layers, b, G), dtype=torch.uint8, device=h.device)
    _check_device(h.device, conv_state=conv_state, xbc=xbc, dt=dt, A=A, D=D, conv_w=conv_w, conv_b=conv_b, y=y,
                  workspace=workspace)
    st = lib().ssd_decode_step(layers, b, H, P, N, G, k, act, io, _ptr(h), _ptr(conv_state), _ptr(xbc),
                               _ptr(dt), _ptr(A), _ptr(D), _ptr(conv_w), _ptr(conv_b), _ptr(y),
                               _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "ssd_decode_step")
    return y


def decode_step_noalloc(h, conv_state, xbc, dt, A, D, conv_w, conv_b, y, G=1, act=SSD_ACT_SILU,
                        stream=None):
    """decode_step through ssd_decode_step_noalloc: no workspace, and the caller passes
    the output y, so nothing is allocated on this path (for callers that cannot allocate
    device memory).  Calls that overlap on the GPU race on the library's shared scratch."""
    layers, b, H, P, N, k, Dc = _decode_shapes(h, conv_state, A, D, conv_w, conv_b, G)
    _need(xbc, "xbc", None, (layers, b, Dc))
    io = _io(xbc)
    _need(dt, "dt", torch.float32, (layers, b, H))
    _need(y, "y", xbc.dtype, (layers, b, H, P))
    _check_device(h.device, conv_state=conv_state, xbc=xbc, dt=dt, A=A, D=D, conv_w=conv_w, conv_b=conv_b, y=y)
    st = lib().ssd_decode_step_noalloc(layers, b, H, P, N, G, k, act, io, _ptr(h), _ptr(conv_state),
                                       _ptr(xbc), _ptr(dt), _ptr(A), _ptr(D), _ptr(conv_w), _ptr(conv_b),
                                       _ptr(y), _stream(stream))
    _check(st, "ssd_decode_step_noalloc")
    return y


class DecodePlan:
    """n_steps decode steps recorded once as a CUDA graph; launch() runs them all on the
    device with no host round trip.  Step t reads xbc_ring[t % ring], dt_ring[t % ring]
    and writes y_ring[t % ring].  The plan holds references to every tensor it uses."""

    def __init__(self, h, conv_state, xbc_ring, dt_ring, A, D, conv_w, conv_b, n_steps, G=1,
                 act=SSD_ACT_SILU, y_ring=None):
        layers, b, H, P, N, k, Dc = _decode_shapes(h, conv_state, A, D, conv_w, conv_b, G)
        ring = xbc_ring.shape[0]
        _need(xbc_ring, "xbc_ring", None, (ring, layers, b, Dc))
        io = _io(xbc_ring)
        _need(dt_ring, "dt_ring", torch.float32, (ring, layers, b, H))
        if y_ring is None:
            y_ring = torch.empty((ring, layers, b, H, P), dtype=xbc_ring.dtype, device=h.device)
        _need(y_ring, "y_ring", xbc_ring.dtype, (ring, layers, b, H, P))
        _check_device(h.device, conv_state=conv_state, xbc_ring=xbc_ring, dt_ring=dt_ring, A=A, D=D,
                      conv_w=conv_w, conv_b=conv_b, y_ring=y_ring)
        self.workspace = torch.empty(decode_workspace_size(layers, b, G), dtype=torch.uint8, device=h.device)
        self._keep = (h, conv_state, xbc_ring, dt_ring, A, D, conv_w, conv_b, y_ring)
        self.y_ring = y_ring
        self.n_steps = n_steps
        handle = ctypes.c_void_p()
        st = lib().ssd_decode_plan_create(ctypes.byref(handle), layers, b, H, P, N, G, k, act, io,
                                          _ptr(h), _ptr(conv_state), _ptr(xbc_ring), _ptr(dt_ring), ring,
                                          _ptr(A), _ptr(D), _ptr(conv_w), _ptr(conv_b), _ptr(y_ring),
                                          int(n_steps), _ptr(self.workspace), self.workspace.numel())
        _check(st, "ssd_decode_plan_create")
        self._h = handle

    def launch(self, stream=None):
        if self._h is None:
            raise RuntimeError("plan destroyed")
        _check(lib().ssd_decode_plan_launch(self._h, _stream(stream)), "ssd_decode_plan_launch")
        return self.y_ring

    def close(self):
        if getattr(self, "_h", None) is not None:
            _check(lib().ssd_decode_plan_destroy(self._h), "ssd_decode_plan_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def decode_loop(h, conv_state, xbc_ring, dt_ring, A, D, conv_w, conv_b, n_steps, G=1,
                act=SSD_ACT_SILU, stream=None):
    """Run n_steps decode steps as one graph launch (ssd_decode_loop: plan built, launched,
    released, no host synchronisation inside).  Returns y_ring [ring, layers, b, H, P]; the
    call waits for the launch before returning because its workspace is a temporary."""
    if stream is not None:
        return _on(stream, decode_loop, h, conv_state, xbc_ring, dt_ring, A, D, conv_w, conv_b, n_steps, G, act)
    layers, b, H, P, N, k, Dc = _decode_shapes(h, conv_state, A, D, conv_w, conv_b, G)
    ring = xbc_ring.shape[0]
    _need(xbc_ring, "xbc_ring", None, (ring, layers, b, Dc))
    io = _io(xbc_ring)
    _need(dt_ring, "dt_ring", torch.float32, (ring, layers, b, H))
    _check_device(h.device, conv_state=conv_state, xbc_ring=xbc_ring, dt_ring=dt_ring, A=A, D=D,
                  conv_w=conv_w, conv_b=conv_b)
    y_ring = torch.empty((ring, layers, b, H, P), dtype=xbc_ring.dtype, device=h.device)
    ws = torch.empty(decode_workspace_size(layers, b, G), dtype=torch.uint8, device=h.device)
    st = lib().ssd_decode_loop(layers, b, H, P, N, G, k, act, io, _ptr(h), _ptr(conv_state), _ptr(xbc_ring),
                               _ptr(dt_ring), ring, _ptr(A), _ptr(D), _ptr(conv_w), _ptr(conv_b), _ptr(y_ring),
                               int(n_steps), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "ssd_decode_loop")
    torch.cuda.current_stream().synchronize()
    return y_ring


def _rows(t, name, dtype=None, shape=None):
    """A norm operand as (rows, D, row stride): CUDA, last index contiguous, the leading indices
    evenly spaced (a slice of a wider row is fine)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (no CPU path exists)" % name)
    if t.dim() < 1:
        raise ValueError("%s must have at least one dimension" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    D = t.shape[-1]
    if D > _INT_MAX:
        raise ValueError("%s: rows of %d elements" % (name, D))
    rows = t.numel() // D if D else 0
    if rows == 0 or t.is_contiguous():
        return rows, D, D
    if D > 1 and t.stride(-1) != 1:
        raise ValueError("%s must be contiguous along its last dimension" % name)
    ld = None  # leading indices of size 1 have no say in the spacing
    for i in range(t.dim() - 2, -1, -1):
        if t.shape[i] == 1:
            continue
        if ld is None:
            ld, span = t.stride(i), t.stride(i) * t.shape[i]
        elif t.stride(i) != span:
            raise ValueError("%s: its rows are not evenly spaced" % name)
        else:
            span *= t.shape[i]
    ld = D if ld is None else ld
    if ld < D:
        raise ValueError("%s: its rows overlap (row stride %d, %d elements)" % (name, ld, D))
    return rows, D, ld


def _groups(groups):
    if not 1 <= groups <= _INT_MAX:
        raise ValueError("groups=%r" % (groups,))
    return int(groups)


def _new_rows(like, dtype):
    """A new contiguous tensor of like's shape."""
    if dtype == like.dtype and like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(like.shape, dtype=dtype, device=like.device)


@functools.lru_cache(maxsize=1024)  # a function of its arguments and the GPU model
def norm_backward_workspace_size(rows, D, groups=1) -> int:
    return int(lib().ssd_norm_backward_workspace_size(rows, D, groups))


def _norm_workspace(workspace, rows, D, groups, like):
    if workspace is None:
        need = norm_backward_workspace_size(rows, D, groups)
        return (like.new_empty(need, dtype=torch.uint8) if need else None), need
    return workspace, workspace.numel() * workspace.element_size()


def residual_norm(x, weight, residual=None, scale=1.0, eps=1e-5, out=None, residual_out=None, stream=None):
    """The norm ahead of a block, with the residual add in it: r = residual + scale * x,
    out = r * (mean(r^2) + eps)^(-1/2) * weight over the last dimension.  x [..., D] bf16 or fp32,
    weight [D] fp32, residual [..., D] fp32 (or bf16 beside bf16 x) or None (r = scale * x).
    Returns (out, r): out in x's type, r in the residual's (fp32 without one, or residual_out's).
    residual_out may be the residual itself (updated in place).  Operands may be slices of wider rows."""
    if stream is not None:
        return _on(stream, residual_norm, x, weight, residual, scale, eps, out, residual_out)
    rows, D, ld_x = _rows(x, "x")
    io = _io(x)
    _need(weight, "weight", torch.float32, (D,))
    ld_res = 0
    if residual is not None:
        _, _, ld_res = _rows(residual, "residual", None, x.shape)
    ld_ro = ld_out = D
    if residual_out is None:
        residual_out = _new_rows(x if residual is None else residual, torch.float32 if residual is None else residual.dtype)
    else:
        _, _, ld_ro = _rows(residual_out, "residual_out", None if residual is None else residual.dtype, x.shape)
    if out is None:
        out = _new_rows(x, x.dtype)
    else:
        _, _, ld_out = _rows(out, "out", x.dtype, x.shape)
    s = _checked_stream(x, weight=weight, residual=residual, out=out, residual_out=residual_out)
    st = lib().ssd_residual_norm(rows, D, io, _io(residual_out), _ptr(x), ld_x, _ptr(residual), ld_res, float(scale),
                                 _ptr(weight), float(eps), _ptr(out), ld_out, _ptr(residual_out), ld_ro, s)
    _check(st, "ssd_residual_norm")
    return out, residual_out


def residual_norm_backward(dout, r, weight, dresidual_out=None, scale=1.0, eps=1e-5, dx=None, dresidual=None,
                           dweight=None, want_dresidual=True, workspace=None, stream=None):
    """Gradients of residual_norm from r as it returned it: dout the gradient of out, dresidual_out
    that of r (None: zero).  Returns (dx, dresidual, dweight): dx in dout's type, dresidual in r's
    (None with want_dresidual=False), dweight [D] fp32.  dresidual may be dresidual_out itself."""
    if stream is not None:
        return _on(stream, residual_norm_backward, dout, r, weight, dresidual_out, scale, eps, dx, dresidual, dweight,
                   want_dresidual, workspace)
    rows, D, ld_do = _rows(dout, "dout")
    io = _io(dout)
    _, _, ld_r = _rows(r, "r", None, dout.shape)
    _need(weight, "weight", torch.float32, (D,))
    ld_dro = ld_dres = 0
    if dresidual_out is not None:
        _, _, ld_dro = _rows(dresidual_out, "dresidual_out", r.dtype, r.shape)
    ld_dx = D
    if dx is None:
        dx = _new_rows(dout, dout.dtype)
    else:
        _, _, ld_dx = _rows(dx, "dx", dout.dtype, dout.shape)
    if dresidual is not None:
        _, _, ld_dres = _rows(dresidual, "dresidual", r.dtype, r.shape)
    elif want_dresidual:
        dresidual, ld_dres = _new_rows(r, r.dtype), D
    if dweight is None:
        dweight = torch.empty_like(weight)
    else:
        _need(dweight, "dweight", torch.float32, (D,))
    workspace, ws_bytes = _norm_workspace(workspace, rows, D, 1, weight)
    s = _checked_stream(dout, r=r, weight=weight, dresidual_out=dresidual_out, dx=dx, dresidual=dresidual,
                     dweight=dweight, workspace=workspace)
    st = lib().ssd_residual_norm_backward(rows, D, io, _io(r), _ptr(dout), ld_do, _ptr(r), ld_r, _ptr(weight),
                                          _ptr(dresidual_out), ld_dro, float(scale), float(eps), _ptr(dx), ld_dx,
                                          _ptr(dresidual), ld_dres, _ptr(dweight), _ptr(workspace), ws_bytes, s)
    _check(st, "ssd_residual_norm_backward")
    return dx, dresidual, dweight


def gated_norm(y, z, weight, groups=1, eps=1e-5, norm_before_gate=False, out=None, stream=None):
    """The norm behind the SSD with its SiLU gate, over groups of D / groups elements of the last
    dimension: norm(y * silu(z)) * weight, or norm(y) * weight * silu(z) with norm_before_gate.
    y, z [..., D] bf16 or fp32 (either may be a slice of a wider row), weight [D] fp32."""
    if stream is not None:
        return _on(stream, gated_norm, y, z, weight, groups, eps, norm_before_gate, out)
    rows, D, ld_y = _rows(y, "y")
    groups = _groups(groups)
    io = _io(y)
    _, _, ld_z = _rows(z, "z", y.dtype, y.shape)
    _need(weight, "weight", torch.float32, (D,))
    ld_out = D
    if out is None:
        out = _new_rows(y, y.dtype)
    else:
        _, _, ld_out = _rows(out, "out", y.dtype, y.shape)
    s = _checked_stream(y, z=z, weight=weight, out=out)
    st = lib().ssd_gated_norm(rows, D, groups, io, int(bool(norm_before_gate)), _ptr(y), ld_y, _ptr(z), ld_z,
                              _ptr(weight), float(eps), _ptr(out), ld_out, s)
    _check(st, "ssd_gated_norm")
    return out


def gated_norm_backward(dout, y, z, weight, groups=1, eps=1e-5, norm_before_gate=False, dy=None, dz=None,
                        dweight=None, workspace=None, stream=None):
    """Gradients of gated_norm: returns (dy, dz, dweight), dweight [D] fp32.  dy and dz may be
    slices of wider rows (the input projection's gradient)."""
    if stream is not None:
        return _on(stream, gated_norm_backward, dout, y, z, weight, groups, eps, norm_before_gate, dy, dz, dweight,
                   workspace)
    rows, D, ld_do = _rows(dout, "dout")
    groups = _groups(groups)
    io = _io(dout)
    _, _, ld_y = _rows(y, "y", dout.dtype, dout.shape)
    _, _, ld_z = _rows(z, "z", dout.dtype, dout.shape)
    _need(weight, "weight", torch.float32, (D,))
    ld_dy = ld_dz = D
    if dy is None:
        dy = _new_rows(y, y.dtype)
    else:
        _, _, ld_dy = _rows(dy, "dy", y.dtype, y.shape)
    if dz is None:
        dz = _new_rows(y, y.dtype)
    else:
        _, _, ld_dz = _rows(dz, "dz", y.dtype, y.shape)
    if dweight is None:
        dweight = torch.empty_like(weight)
    else:
        _need(dweight, "dweight", torch.float32, (D,))
    workspace, ws_bytes = _norm_workspace(workspace, rows, D, groups, weight)
    s = _checked_stream(dout, y=y, z=z, weight=weight, dy=dy, dz=dz, dweight=dweight, workspace=workspace)
    st = lib().ssd_gated_norm_backward(rows, D, groups, io, int(bool(norm_before_gate)), _ptr(dout), ld_do,
                                       _ptr(y), ld_y, _ptr(z), ld_z, _ptr(weight), float(eps), _ptr(dy), ld_dy,
                                       _ptr(dz), ld_dz, _ptr(dweight), _ptr(workspace), ws_bytes, s)
    _check(st, "ssd_gated_norm_backward")
    return dy, dz, dweight
