"""Python binding of the layers around the mixer (``include/swimba_layers.h``).

Argument marshalling only, as in :mod:`.binding`: every step runs in the HIP
kernels of ``libswimba.so``. Tensors are contiguous, but for the inputs and
gradients of the gated scan, which may be column ranges of a wider tensor
(unit stride along the channels, one row stride for all of them). All tensors
of a call must lie on the current device; work goes to that device's current
stream unless ``stream`` is given.
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


def _refuse(t, dev):
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


def _rows(dev, *tensors):
    """Pointers of [M, C] tensors whose rows are equally far apart, and that distance."""
    ld, ptrs, single = None, [], False
    for t in tensors:
        if t is None:
            ptrs.append(None)
            continue
        stride = t.stride()
        if len(stride) != 2:
            t = t.view(-1, t.shape[-1])
            stride = t.stride()
        if ld is None:
            rows, cols = t.shape
            single = rows <= 1  # whatever its stride is, no row follows
            ld = cols if single else stride[0]
        elif stride[0] != ld and not single:
            raise ValueError("the gated scan's tensors must have one row stride")
        if stride[1] != 1 and t.shape[1] > 1:
            raise ValueError("rows of the gated scan must have unit stride along the channels")
        if t.get_device() != dev:
            _refuse(t, dev)
        ptrs.append(t.data_ptr())
    return ptrs, ld


def _stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _ws(ws, ws_bytes):
    return (ws.numel() * ws.element_size() if ws is not None else 0) if ws_bytes is None \
        else ws_bytes


# ----------------------------------------------------------------- raw calls

def swimba_layer_norm(dims, x, residual, weight, bias, eps, sum, y, mean=None, rstd=None,
                      stream=None):
    dev = _device()
    px, pr, pw, pb, ps, py, pm, pq = _ptrs(dev, x, residual, weight, bias, sum, y, mean, rstd)
    _check(lib().swimba_layer_norm(ctypes.byref(dims), px, pr, pw, pb, eps, ps, py, pm, pq,
                                   _stream(stream, dev)))


def swimba_layer_norm_backward(dims, s, weight, mean, rstd, dy, dres, dx, dweight, dbias, ws,
                               ws_bytes=None, stream=None):
    if dy is not None and dy.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"dy of {dy.dtype}: bfloat16 or float32")
    dev = _device()
    dy_dtype = sb.BF16 if dy is not None and dy.dtype == torch.bfloat16 else sb.F32
    p = _ptrs(dev, s, weight, mean, rstd, dy, dres, dx, dweight, dbias, ws)
    _check(lib().swimba_layer_norm_backward(ctypes.byref(dims), *p[:5], dy_dtype, *p[5:],
                                            _ws(ws, ws_bytes), _stream(stream, dev)))


def swimba_gated_scan(dims, x, forget, gate, seq_lens, h_init, y, h_final, carry, ws,
                      ws_bytes=None, stream=None):
    dev = _device()
    rows, ld = _rows(dev, x, forget, gate)
    p = _ptrs(dev, seq_lens, h_init, y, h_final, carry, ws)
    _check(lib().swimba_gated_scan(ctypes.byref(dims), *rows, ld, *p, _ws(ws, ws_bytes),
                                   _stream(stream, dev)))


def swimba_gated_scan_backward(dims, x, forget, gate, seq_lens, carry, dy, dh_final, dx, dforget,
                               dgate, dh_init, ws, ws_bytes=None, stream=None):
    dev = _device()
    rows, ld = _rows(dev, x, forget, gate)
    drows, ldd = _rows(dev, dx, dforget, dgate if gate is not None else None)
    p = _ptrs(dev, seq_lens, carry, dy, dh_final, dh_init, ws)
    _check(lib().swimba_gated_scan_backward(ctypes.byref(dims), *rows, ld, *p[:4], *drows, ldd,
                                            *p[4:], _ws(ws, ws_bytes), _stream(stream, dev)))


def swimba_gated_step(dims, x, forget, gate, h_prev, h, y, stream=None):
    dev = _device()
    rows, ld = _rows(dev, x, forget, gate)
    _check(lib().swimba_gated_step(ctypes.byref(dims), *rows, ld, *_ptrs(dev, h_prev, h, y),
                                   _stream(stream, dev)))


def swimba_gated_project(dims, x, w_in, act, z, h, stream=None):
    dev = _device()
    px, pw, pz, ph = _ptrs(dev, x, w_in, z, h)
    _check(lib().swimba_gated_project(ctypes.byref(dims), px, pw, act, pz, ph, _stream(stream, dev)))


def swimba_gated_project_backward(dims, x, w_in, dh, act, dx, dw_in, ws, ws_bytes=None,
                                  stream=None):
    dev = _device()
    px, pw, pd, pdx, pdw, pws = _ptrs(dev, x, w_in, dh, dx, dw_in, ws)
    _check(lib().swimba_gated_project_backward(ctypes.byref(dims), px, pw, pd, act, pdx, pdw, pws,
                                               _ws(ws, ws_bytes), _stream(stream, dev)))


def swimba_output_project_backward(dims, y, w_out, dout, dy, dw_out, ws, ws_bytes=None,
                                   stream=None):
    dev = _device()
    _check(lib().swimba_output_project_backward(
        ctypes.byref(dims), *_ptrs(dev, y, w_out, dout, dy, dw_out, ws), _ws(ws, ws_bytes),
        _stream(stream, dev)))
