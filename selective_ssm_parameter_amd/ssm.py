"""Python binding of the selective state space layer and its loss (``include/swimba_ssm.h``).

Argument marshalling only, as in :mod:`.layers`, whose checks these calls share:
tensors are contiguous, but for those that the header gives a row stride, which
may be column ranges of a wider tensor (unit stride along the row). All tensors
of a call must lie on the current device, have the header's element types
(``seq_lens`` and ``targets`` int32) and hold at least the elements that ``dims``
asks for, else ValueError; work goes to that device's current stream unless
``stream`` (one of the same device) is given.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as sb
from .binding import SwimbaError, _check  # noqa: F401  (SwimbaError: what calls raise)
from .layers import _F32, _TYPES, _device, _ptr, _ptrs, _rows, _stream, _ws

CONV_LINEAR, CONV_SILU = 0, 1
(CAUSAL_CONV_BACKWARD, SELECTIVE_SCAN, SELECTIVE_SCAN_BACKWARD, CROSS_ENTROPY,
 CROSS_ENTROPY_BACKWARD) = range(5)

EXPORTS = (
    "swimba_ssm_workspace_size", "swimba_causal_conv", "swimba_causal_conv_backward",
    "swimba_causal_conv_step", "swimba_selective_scan", "swimba_selective_scan_carry_size",
    "swimba_selective_scan_backward", "swimba_selective_step", "swimba_cross_entropy",
    "swimba_cross_entropy_backward",
)

_lib = None


def lib() -> ctypes.CDLL:
    """libswimba.so with these calls' signatures (loaded once)."""
    global _lib
    if _lib is not None:
        return _lib
    L = sb.lib()
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    D = ctypes.POINTER(sb.Dims)
    inputs = [P, I64, P, I64, P, I64, P, P, I64, P, P, P]  # x, dt, z, B, C, A, D, dt_bias
    for name, res, args in (
            ("swimba_ssm_workspace_size", SZ, [D, I32]),
            ("swimba_selective_scan_carry_size", SZ, [D]),
            ("swimba_causal_conv", I32, [D, I32, P, I64, P, P, I32, P, P, P, P, P]),
            ("swimba_causal_conv_backward", I32,
             [D, I32, P, I64, P, P, I32, P, P, P, P, P, I64, P, P, P, P, SZ, P]),
            ("swimba_causal_conv_step", I32, [D, I32, P, I64, P, P, I32, P, P, P, P]),
            ("swimba_selective_scan", I32, [D, *inputs, P, P, P, P, P, P, SZ, P]),
            ("swimba_selective_scan_backward", I32,
             [D, *inputs, P, P, P, P, P, I64, P, I64, P, I64, P, P, I64, P, P, P, P, P, SZ, P]),
            ("swimba_selective_step", I32, [D, *inputs, P, P, P, P]),
            ("swimba_cross_entropy", I32, [D, P, P, P, P, P, P, SZ, P]),
            ("swimba_cross_entropy_backward", I32, [D, P, P, P, P, P, P, P, P, SZ, P])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    _lib = L
    return L


def ssm_dims(batch, seqlen, channels, dstate, ngroups, dtype) -> sb.Dims:
    """Dims of the convolution (dstate and ngroups 1) or of the selective scan."""
    if ngroups < 1 or channels % ngroups:
        raise ValueError(f"{channels} channels in {ngroups} groups")
    return sb.make_dims(batch, seqlen, 1, ngroups, channels // ngroups, dstate, ngroups, 1, 1, 1,
                        dtype)


def loss_dims(tokens, d_model, vocab, dtype) -> sb.Dims:
    """Dims of the cross entropy over a vocabulary."""
    return sb.make_dims(1, tokens, d_model, 1, vocab, 1, 1, 1, 1, 1, dtype)


def ssm_workspace_size(dims, call: int) -> int:
    return lib().swimba_ssm_workspace_size(ctypes.byref(dims), call)


def ssm_workspace(dims, call: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(ssm_workspace_size(dims, call), 16), dtype=torch.uint8, device=device)


def selective_scan_carry(dims, device="cuda") -> torch.Tensor:
    """The tensor that swimba_selective_scan leaves its backward's states in."""
    n = lib().swimba_selective_scan_carry_size(ctypes.byref(dims))
    return torch.empty(max(n // 4, 4), dtype=torch.float32, device=device)


def _row(dev, dt, t, M, C):
    """Pointer and row stride of one [M, C] tensor (None: its stride counts for nothing)."""
    if t is None:
        return None, C
    (ptr,), ld = _rows(dev, t, dt=dt, M=M, C=C)
    return ptr, ld


# ----------------------------------------------------------------- convolution

def swimba_causal_conv(dims, width, x, weight, bias, act, seq_lens, state_in, y, state_out=None,
                       stream=None):
    dev, dt, B, C = _device(), _TYPES.get(dims.dtype), dims.batch, dims.nheads * dims.headdim
    M, n = B * dims.seqlen, B * (width - 1) * C
    _check(lib().swimba_causal_conv(
        dims, width, *_row(dev, dt, x, M, C), _ptr(dev, dt, weight, C * width),
        _ptr(dev, dt, bias, C), act, _ptr(dev, torch.int32, seq_lens, B if M else 0),
        _ptr(dev, dt, state_in, n), _ptr(dev, dt, y, M * C), _ptr(dev, dt, state_out, n),
        _stream(stream, dev)))


def swimba_causal_conv_backward(dims, width, x, weight, bias, act, seq_lens, state_in, dy,
                                dstate_out, dx, dweight, dbias, dstate_in, ws, ws_bytes=None,
                                stream=None):
    dev, dt, B, C = _device(), _TYPES.get(dims.dtype), dims.batch, dims.nheads * dims.headdim
    M, n = B * dims.seqlen, B * (width - 1) * C
    _check(lib().swimba_causal_conv_backward(
        dims, width, *_row(dev, dt, x, M, C), _ptr(dev, dt, weight, C * width),
        _ptr(dev, dt, bias, C), act, _ptr(dev, torch.int32, seq_lens, B if M else 0),
        _ptr(dev, dt, state_in, n), _ptr(dev, dt, dy, M * C), _ptr(dev, _F32, dstate_out, n),
        *_row(dev, dt, dx, M, C), _ptr(dev, _F32, dweight, C * width), _ptr(dev, _F32, dbias, C),
        _ptr(dev, _F32, dstate_in, n), *_ptrs(dev, ws), _ws(ws, ws_bytes), _stream(stream, dev)))


def swimba_causal_conv_step(dims, width, x, weight, bias, act, state_in, state_out, y,
                            stream=None):
    dev, dt, B, C = _device(), _TYPES.get(dims.dtype), dims.batch, dims.nheads * dims.headdim
    n = B * (width - 1) * C
    st = lib().swimba_causal_conv_step(
        dims, width, *_row(dev, dt, x, B, C), _ptr(dev, dt, weight, C * width),
        _ptr(dev, dt, bias, C), act, _ptr(dev, dt, state_in, n), _ptr(dev, dt, state_out, n),
        _ptr(dev, dt, y, B * C), _stream(stream, dev))
    if st:
        _check(st)


# --------------------------------------------------------------- selective scan

def _scan_inputs(dev, dims, x, dt, z, B, C, A, D, dt_bias):
    t, M, Ch = _TYPES.get(dims.dtype), dims.batch * dims.seqlen, dims.nheads * dims.headdim
    GN = dims.ngroups * dims.dstate
    bc, ldbc = _rows(dev, B, C, dt=t, M=M, C=GN)
    return (*_row(dev, t, x, M, Ch), *_row(dev, t, dt, M, Ch), *_row(dev, t, z, M, Ch), *bc,
            GN if ldbc is None else ldbc, _ptr(dev, _F32, A, Ch * dims.dstate if M else 0),
            _ptr(dev, _F32, D, Ch), _ptr(dev, _F32, dt_bias, Ch))


def _scan_carry_ptr(dev, dims, carry):
    return None if carry is None else \
        _ptr(dev, _F32, carry, lib().swimba_selective_scan_carry_size(dims) // 4)


def swimba_selective_scan(dims, x, dt, z, B, C, A, D, dt_bias, seq_lens, h_init, y, h_final,
                          carry, ws, ws_bytes=None, stream=None):
    dev, t, Bt, Ch = _device(), _TYPES.get(dims.dtype), dims.batch, dims.nheads * dims.headdim
    M, n = Bt * dims.seqlen, Bt * Ch * dims.dstate
    _check(lib().swimba_selective_scan(
        dims, *_scan_inputs(dev, dims, x, dt, z, B, C, A, D, dt_bias),
        _ptr(dev, torch.int32, seq_lens, Bt if M else 0), _ptr(dev, _F32, h_init, n),
        _ptr(dev, t, y, M * Ch), _ptr(dev, _F32, h_final, n), _scan_carry_ptr(dev, dims, carry),
        *_ptrs(dev, ws), _ws(ws, ws_bytes), _stream(stream, dev)))


def swimba_selective_scan_backward(dims, x, dt, z, B, C, A, D, dt_bias, seq_lens, carry, dy,
                                   dh_final, dx, ddt, dz, dB, dC, dA, dD, ddt_bias, dh_init, ws,
                                   ws_bytes=None, stream=None):
    dev, t, Bt, Ch = _device(), _TYPES.get(dims.dtype), dims.batch, dims.nheads * dims.headdim
    M, n, GN = Bt * dims.seqlen, Bt * Ch * dims.dstate, dims.ngroups * dims.dstate
    dbc, lddbc = _rows(dev, dB, dC, dt=t, M=M, C=GN)
    _check(lib().swimba_selective_scan_backward(
        dims, *_scan_inputs(dev, dims, x, dt, z, B, C, A, D, dt_bias),
        _ptr(dev, torch.int32, seq_lens, Bt if M else 0), _scan_carry_ptr(dev, dims, carry),
        _ptr(dev, t, dy, M * Ch), _ptr(dev, _F32, dh_final, n), *_row(dev, t, dx, M, Ch),
        *_row(dev, t, ddt, M, Ch), *_row(dev, t, dz if z is not None else None, M, Ch), *dbc,
        GN if lddbc is None else lddbc, _ptr(dev, _F32, dA, Ch * dims.dstate),
        _ptr(dev, _F32, dD, Ch), _ptr(dev, _F32, ddt_bias, Ch), _ptr(dev, _F32, dh_init, n),
        *_ptrs(dev, ws), _ws(ws, ws_bytes), _stream(stream, dev)))


def swimba_selective_step(dims, x, dt, z, B, C, A, D, dt_bias, h_prev, h, y, stream=None):
    dev, t, Bt, Ch = _device(), _TYPES.get(dims.dtype), dims.batch, dims.nheads * dims.headdim
    n = Bt * Ch * dims.dstate
    st = lib().swimba_selective_step(
        dims, *_scan_inputs(dev, dims, x, dt, z, B, C, A, D, dt_bias), _ptr(dev, _F32, h_prev, n),
        _ptr(dev, _F32, h, n), _ptr(dev, t, y, Bt * Ch), _stream(stream, dev))
    if st:
        _check(st)


# ---------------------------------------------------------------- cross entropy

def _loss_sizes(dims):
    return (_TYPES.get(dims.dtype), dims.batch * dims.seqlen, dims.d_model,
            dims.nheads * dims.headdim)


def swimba_cross_entropy(dims, x, w, targets, loss, lse, ws, ws_bytes=None, stream=None):
    dev = _device()
    dt, M, D, V = _loss_sizes(dims)
    _check(lib().swimba_cross_entropy(
        dims, _ptr(dev, dt, x, M * D), _ptr(dev, dt, w, V * D), _ptr(dev, torch.int32, targets, M),
        _ptr(dev, _F32, loss, M), _ptr(dev, _F32, lse, M), *_ptrs(dev, ws), _ws(ws, ws_bytes),
        _stream(stream, dev)))


def swimba_cross_entropy_backward(dims, x, w, targets, lse, dloss, dx, dw, ws, ws_bytes=None,
                                  stream=None):
    dev = _device()
    dt, M, D, V = _loss_sizes(dims)
    _check(lib().swimba_cross_entropy_backward(
        dims, _ptr(dev, dt, x, M * D), _ptr(dev, dt, w, V * D), _ptr(dev, torch.int32, targets, M),
        _ptr(dev, _F32, lse, M), _ptr(dev, _F32, dloss, M), _ptr(dev, _F32, dx, M * D),
        _ptr(dev, _F32, dw, V * D), *_ptrs(dev, ws), _ws(ws, ws_bytes), _stream(stream, dev)))
