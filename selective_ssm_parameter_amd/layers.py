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
from .binding import SwimbaError, _check, _stream  # noqa: F401  (SwimbaError: what calls raise)

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
             [D, P, P, P, P, I32, P, P, P, SZ, P]),
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


def _ptr(t):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensor on {t.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return sb._ptr(t)


def _rows(*tensors):
    """Pointers of [M, C] tensors whose rows are equally far apart, and that distance."""
    ld, ptrs = None, []
    for t in tensors:
        if t is None:
            ptrs.append(None)
            continue
        t2 = t.reshape(-1, t.shape[-1]) if t.dim() != 2 and t.is_contiguous() else t
        if t2.dim() != 2 or (t2.stride(1) != 1 and t2.shape[1] > 1):
            raise ValueError("rows of the gated scan must be [tokens, channels] with unit stride "
                             "along the channels")
        step = t2.stride(0) if t2.shape[0] > 1 else max(t2.stride(0), t2.shape[1])
        if ld is None or t2.shape[0] <= 1:
            ld = step if ld is None else ld
        elif step != ld:
            raise ValueError("the gated scan's tensors must have one row stride")
        if t2.is_cuda and t2.device.index != torch.cuda.current_device():
            _ptr(t2)  # raises
        ptrs.append(t2.data_ptr())
    return ptrs, ld


def _ws(ws, ws_bytes):
    return (ws.numel() * ws.element_size() if ws is not None else 0) if ws_bytes is None \
        else ws_bytes


# ----------------------------------------------------------------- raw calls

def swimba_layer_norm(dims, x, residual, weight, bias, eps, sum, y, mean=None, rstd=None,
                      stream=None):
    _check(lib().swimba_layer_norm(
        ctypes.byref(dims), _ptr(x), _ptr(residual), _ptr(weight), _ptr(bias), eps, _ptr(sum),
        _ptr(y), _ptr(mean), _ptr(rstd), _stream(stream)))


def swimba_layer_norm_backward(dims, s, weight, mean, rstd, dy, dres, dx, dweight, dbias, ws,
                               ws_bytes=None, stream=None):
    if dy is not None and dy.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"dy of {dy.dtype}: bfloat16 or float32")
    dy_dtype = sb.BF16 if dy is not None and dy.dtype == torch.bfloat16 else sb.F32
    _check(lib().swimba_layer_norm_backward(
        ctypes.byref(dims), _ptr(s), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dy), dy_dtype,
        _ptr(dres), _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(ws), _ws(ws, ws_bytes),
        _stream(stream)))


def swimba_gated_scan(dims, x, forget, gate, seq_lens, h_init, y, h_final, carry, ws,
                      ws_bytes=None, stream=None):
    (px, pf, po), ld = _rows(x, forget, gate)
    _check(lib().swimba_gated_scan(
        ctypes.byref(dims), px, pf, po, ld, _ptr(seq_lens), _ptr(h_init), _ptr(y), _ptr(h_final),
        _ptr(carry), _ptr(ws), _ws(ws, ws_bytes), _stream(stream)))


def swimba_gated_scan_backward(dims, x, forget, gate, seq_lens, carry, dy, dh_final, dx, dforget,
                               dgate, dh_init, ws, ws_bytes=None, stream=None):
    (px, pf, po), ld = _rows(x, forget, gate)
    (pdx, pdf, pdo), ldd = _rows(dx, dforget, dgate if gate is not None else None)
    _check(lib().swimba_gated_scan_backward(
        ctypes.byref(dims), px, pf, po, ld, _ptr(seq_lens), _ptr(carry), _ptr(dy),
        _ptr(dh_final), pdx, pdf, pdo, ldd, _ptr(dh_init), _ptr(ws), _ws(ws, ws_bytes),
        _stream(stream)))


def swimba_gated_step(dims, x, forget, gate, h_prev, h, y, stream=None):
    (px, pf, po), ld = _rows(x, forget, gate)
    _check(lib().swimba_gated_step(ctypes.byref(dims), px, pf, po, ld, _ptr(h_prev), _ptr(h),
                                   _ptr(y), _stream(stream)))


def swimba_gated_project(dims, x, w_in, act, z, h, stream=None):
    _check(lib().swimba_gated_project(ctypes.byref(dims), _ptr(x), _ptr(w_in), act, _ptr(z),
                                      _ptr(h), _stream(stream)))


def swimba_gated_project_backward(dims, x, w_in, z, dh, act, dx, dw_in, ws, ws_bytes=None,
                                  stream=None):
    _check(lib().swimba_gated_project_backward(
        ctypes.byref(dims), _ptr(x), _ptr(w_in), _ptr(z), _ptr(dh), act, _ptr(dx), _ptr(dw_in),
        _ptr(ws), _ws(ws, ws_bytes), _stream(stream)))


def swimba_output_project_backward(dims, y, w_out, dout, dy, dw_out, ws, ws_bytes=None,
                                   stream=None):
    _check(lib().swimba_output_project_backward(
        ctypes.byref(dims), _ptr(y), _ptr(w_out), _ptr(dout), _ptr(dy), _ptr(dw_out), _ptr(ws),
        _ws(ws, ws_bytes), _stream(stream)))
