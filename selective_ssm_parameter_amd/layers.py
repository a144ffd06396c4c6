"""Python binding of the layers around the mixer (``include/swimba_layers.h``).

Argument marshalling only, as in :mod:`.binding`: every step runs in the HIP
kernels of ``libswimba.so``. Tensors are contiguous, but for the inputs and
gradients of the gated scan, which may be column ranges of a wider tensor
(unit stride along the channels, one row stride for all of them). All tensors
of a call must lie on the current device, have the header's element types
(``seq_lens`` int32) and hold at least the elements that ``dims`` asks for, else
ValueError; work goes to that device's current stream unless ``stream`` (one of
the same device) is given.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as sb
from .binding import SwimbaError, _check  # noqa: F401  (SwimbaError: what calls raise)

ACT_SILU, ACT_GELU = 0, 1
(LAYER_NORM_BACKWARD, LAYER_GATED_SCAN, LAYER_GATED_SCAN_BACKWARD, LAYER_GATED_PROJECT_BACKWARD,
 LAYER_OUTPUT_PROJECT_BACKWARD) = range(5)

EXPORTS = (
    "swimba_layer_workspace_size", "swimba_layer_norm", "swimba_layer_norm_backward",
    "swimba_gated_scan", "swimba_gated_scan_carry_size", "swimba_gated_scan_backward",
    "swimba_gated_step", "swimba_gated_project", "swimba_gated_project_backward",
    "swimba_output_project_backward",
)

_lib = None


def lib() -> ctypes.CDLL:
    """libswimba.so with the layer calls' signatures (loaded once)."""
    global _lib
    if _lib is not None:
        return _lib
    L = sb.lib()
    P, I32, I64, SZ, F = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                          ctypes.c_float)
    D = ctypes.POINTER(sb.Dims)
    for name, res, args in (
            ("swimba_layer_workspace_size", SZ, [D, I32]),
            ("swimba_gated_scan_carry_size", SZ, [D]),
            ("swimba_layer_norm", I32, [D, P, P, P, P, F, P, P, P, P, P]),
            ("swimba_layer_norm_backward", I32,
             [D, P, P, P, P, P, I32, P, P, P, P, P, SZ, P]),
            ("swimba_gated_scan", I32, [D, P, P, P, I64, P, P, P, P, P, P, SZ, P]),
            ("swimba_gated_scan_backward", I32,
             [D, P, P, P, I64, P, P, P, P, P, P, P, I64, P, P, SZ, P]),
            ("swimba_gated_step", I32, [D, P, P, P, I64, P, P, P, P]),
            ("swimba_gated_project", I32, [D, P, P, I32, P, P, P]),
            ("swimba_gated_project_backward", I32,
             [D, P, P, P, I32, P, P, P, SZ, P]),
            ("swimba_output_project_backward", I32, [D, P, P, P, P, P, P, SZ, P])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    _lib = L
    return L


def layer_dims(batch, seqlen, d_model, inner, dtype) -> sb.Dims:
    """Dims of a layer: ``inner`` = F or C (the header's nheads * headdim)."""
    return sb.make_dims(batch, seqlen, d_model, 1, inner, 1, 1, 1, 1, 1, dtype)


def layer_workspace_size(dims, call: int) -> int:
    return lib().swimba_layer_workspace_size(ctypes.byref(dims), call)


def layer_workspace(dims, call: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(layer_workspace_size(dims, call), 16), dtype=torch.uint8, device=device)


def gated_scan_carry(dims, device="cuda") -> torch.Tensor:
    """The tensor that swimba_gated_scan leaves its backward's states in."""
    n = lib().swimba_gated_scan_carry_size(ctypes.byref(dims))
    return torch.empty(max(n // 4, 4), dtype=torch.float32, device=device)


# A decode step is a few microseconds on the GPU, so the marshalling below asks
# torch for no more than it needs.

def _device():
    """The current device's index. Before CUDA is initialised no tensor lies on
    the GPU (and a host tensor's index, -1, must not pass for a device's)."""
    if not torch.cuda.is_initialized():
        raise ValueError("CUDA is not initialised: the tensors cannot lie on the current device")
    return torch._C._cuda_getDevice()


# The element type of dims.dtype.
_TYPES = {sb.F32: torch.float32, sb.BF16: torch.bfloat16}
_F32 = torch.float32


def _refuse(t, dev, dt=None, n=0):
    if n > 0 and dt is not None and t.dtype is not dt:
        raise ValueError(f"tensor of {t.dtype}, but the call takes it as {dt}")
    if t.numel() < n:
        raise ValueError(f"tensor of {t.numel()} elements, but the call takes {n}")
    if t.get_device() != dev:
        raise ValueError(f"tensor on {t.device}, but the current device is cuda:{dev}")
    raise ValueError("tensors passed to the Swimba library must be contiguous")


def _ptrs(dev, *tensors):
    """Device pointers of contiguous tensors on device dev (None stays None)."""
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
        elif t.get_device() == dev and t.is_contiguous():
            out.append(t.data_ptr())
        else:
            _refuse(t, dev)
    return out


def _ptr(dev, dt, t, n):
    """The pointer of one that holds n elements of dt or more. (Where n is 0, for
    want of tokens, nothing is read and any type will do; an element type that
    the library does not know, None here, is refused there.)"""
    if t is None:
        return None
    if t.dtype is dt and t.numel() >= n and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if (n <= 0 or dt is None) and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _refuse(t, dev, dt, n)


def _rows(dev, *tensors, dt=None, M=0, C=0):
    """Pointers of [M, C] tensors whose rows are equally far apart, and that distance."""
    ld, ptrs = None, []
    for t in tensors:
        if t is None:
            ptrs.append(None)
            continue
        stride = t.stride()
        if len(stride) != 2:
            t = t.view(-1, t.shape[-1])
            stride = t.stride()
        rows, cols = t.shape
        if ld is None:
            single = rows <= 1  # whatever its stride is, no row follows
            ld = cols if single else stride[0]
        elif stride[0] != ld and not single:
            raise ValueError("the gated scan's tensors must have one row stride")
        if stride[1] != 1 and cols > 1:
            raise ValueError("rows of the gated scan must have unit stride along the channels")
        if t.dtype is not dt and M > 0 and dt is not None:
            _refuse(t, dev, dt, 1)
        if rows < M or cols < C:
            raise ValueError(f"tensor of {rows} rows of {cols}, but the call takes {M} of {C}")
        if t.get_device() != dev:
            _refuse(t, dev)
        ptrs.append(t.data_ptr())
    return ptrs, ld


# (a torch without GPU support lacks it, and loads this file all the same)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    if isinstance(stream, int):
        return stream
    of = getattr(stream, "device_index", dev)
    if of != dev:
        raise ValueError(f"stream of device {of}, but the current device is cuda:{dev}")
    return stream.cuda_stream


def _ws(ws, ws_bytes):
    have = ws.numel() * ws.element_size() if ws is not None else 0
    if ws_bytes is None:
        return have
    if ws_bytes > have:
        raise ValueError(f"workspace of {have} bytes passed as one of {ws_bytes}")
    return ws_bytes


# ----------------------------------------------------------------- raw calls

def swimba_layer_norm(dims, x, residual, weight, bias, eps, sum, y, mean=None, rstd=None,
                      stream=None):
    dev, dt, M, D = _device(), _TYPES.get(dims.dtype), dims.batch * dims.seqlen, dims.d_model
    n = M * D
    st = lib().swimba_layer_norm(
        dims, _ptr(dev, dt, x, n), _ptr(dev, dt, residual, n), _ptr(dev, dt, weight, D),
        _ptr(dev, dt, bias, D), eps, _ptr(dev, dt, sum, 0 if residual is None else n),
        _ptr(dev, dt, y, n), None if mean is None else _ptr(dev, _F32, mean, M),
        None if rstd is None else _ptr(dev, _F32, rstd, M),
        _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check(st)


def swimba_layer_norm_backward(dims, s, weight, mean, rstd, dy, dres, dx, dweight, dbias, ws,
                               ws_bytes=None, stream=None):
    if dy is not None and dy.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"dy of {dy.dtype}: bfloat16 or float32")
    dev, dt, M, D = _device(), _TYPES.get(dims.dtype), dims.batch * dims.seqlen, dims.d_model
    n = M * D
    dy_dtype = sb.BF16 if dy is not None and dy.dtype == torch.bfloat16 else sb.F32
    _check(lib().swimba_layer_norm_backward(
        dims, _ptr(dev, dt, s, n), _ptr(dev, dt, weight, D), _ptr(dev, _F32, mean, M),
        _ptr(dev, _F32, rstd, M), _ptr(dev, _TYPES[dy_dtype], dy, n), dy_dtype,
        _ptr(dev, _F32, dres, n), _ptr(dev, _F32, dx, n), _ptr(dev, _F32, dweight, D),
        _ptr(dev, _F32, dbias, D), *_ptrs(dev, ws), _ws(ws, ws_bytes), _stream(stream, dev)))


def _carry_ptr(dev, dims, carry):
    return None if carry is None else \
        _ptr(dev, _F32, carry, lib().swimba_gated_scan_carry_size(dims) // 4)


def swimba_gated_scan(dims, x, forget, gate, seq_lens, h_init, y, h_final, carry, ws,
                      ws_bytes=None, stream=None):
    dev, dt, B, C = _device(), _TYPES.get(dims.dtype), dims.batch, dims.nheads * dims.headdim
    M, n = B * dims.seqlen, B * C
    rows, ld = _rows(dev, x, forget, gate, dt=dt, M=M, C=C)
    _check(lib().swimba_gated_scan(
        dims, *rows, ld, _ptr(dev, torch.int32, seq_lens, B if M else 0),
        _ptr(dev, _F32, h_init, n), _ptr(dev, dt, y, M * C), _ptr(dev, _F32, h_final, n),
        _carry_ptr(dev, dims, carry), *_ptrs(dev, ws), _ws(ws, ws_bytes), _stream(stream, dev)))


def swimba_gated_scan_backward(dims, x, forget, gate, seq_lens, carry, dy, dh_final, dx, dforget,
                               dgate, dh_init, ws, ws_bytes=None, stream=None):
    dev, dt, B, C = _device(), _TYPES.get(dims.dtype), dims.batch, dims.nheads * dims.headdim
    M, n = B * dims.seqlen, B * C
    rows, ld = _rows(dev, x, forget, gate, dt=dt, M=M, C=C)
    drows, ldd = _rows(dev, dx, dforget, dgate if gate is not None else None, dt=dt, M=M, C=C)
    _check(lib().swimba_gated_scan_backward(
        dims, *rows, ld, _ptr(dev, torch.int32, seq_lens, B if M else 0),
        _carry_ptr(dev, dims, carry), _ptr(dev, dt, dy, M * C), _ptr(dev, _F32, dh_final, n),
        *drows, ldd, _ptr(dev, _F32, dh_init, n), *_ptrs(dev, ws), _ws(ws, ws_bytes),
        _stream(stream, dev)))


def swimba_gated_step(dims, x, forget, gate, h_prev, h, y, stream=None):
    dev, dt, B, C = _device(), _TYPES.get(dims.dtype), dims.batch, dims.nheads * dims.headdim
    n = B * C
    (px, pf, po), ld = _rows(dev, x, forget, gate, dt=dt, M=B, C=C)
    st = lib().swimba_gated_step(
        dims, px, pf, po, ld, _ptr(dev, _F32, h_prev, n), _ptr(dev, _F32, h, n),
        _ptr(dev, dt, y, n), _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check(st)


def _project_sizes(dims):
    """The element type and the elements of [M, D], [M, F] and [F, D]."""
    M, D, F = dims.batch * dims.seqlen, dims.d_model, dims.nheads * dims.headdim
    return _TYPES.get(dims.dtype), M * D, M * F, F * D


def swimba_gated_project(dims, x, w_in, act, z, h, stream=None):
    dev = _device()
    dt, nx, nh, nw = _project_sizes(dims)
    st = lib().swimba_gated_project(
        dims, _ptr(dev, dt, x, nx), _ptr(dev, dt, w_in, 2 * nw), act, _ptr(dev, dt, z, 2 * nh),
        _ptr(dev, dt, h, nh), _raw_stream(dev) if stream is None else _stream(stream, dev))
    if st:
        _check(st)


def swimba_gated_project_backward(dims, x, w_in, dh, act, dx, dw_in, ws, ws_bytes=None,
                                  stream=None):
    dev = _device()
    dt, nx, nh, nw = _project_sizes(dims)
    _check(lib().swimba_gated_project_backward(
        dims, _ptr(dev, dt, x, nx), _ptr(dev, dt, w_in, 2 * nw), _ptr(dev, dt, dh, nh), act,
        _ptr(dev, _F32, dx, nx), _ptr(dev, _F32, dw_in, 2 * nw), *_ptrs(dev, ws),
        _ws(ws, ws_bytes), _stream(stream, dev)))


def swimba_output_project_backward(dims, y, w_out, dout, dy, dw_out, ws, ws_bytes=None,
                                   stream=None):
    dev = _device()
    dt, nx, ny, nw = _project_sizes(dims)
    _check(lib().swimba_output_project_backward(
        dims, _ptr(dev, dt, y, ny), _ptr(dev, dt, w_out, nw), _ptr(dev, dt, dout, nx),
        _ptr(dev, dt, dy, ny), _ptr(dev, _F32, dw_out, nw), *_ptrs(dev, ws), _ws(ws, ws_bytes),
        _stream(stream, dev)))
