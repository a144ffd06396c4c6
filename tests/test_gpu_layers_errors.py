"""What a layer call returns after a HIP call of somebody else has failed."""
from __future__ import annotations

import ctypes

import pytest
import torch

from selective_ssm_parameter_amd import binding as sb
from selective_ssm_parameter_amd import layers as sl

pytestmark = pytest.mark.gpu


def test_an_earlier_error_is_not_the_calls_own():
    """The runtime keeps the last error of the thread until it is asked for. A call
    that launches its kernels succeeds, whatever failed before it, and leaves that
    error to whom it belongs."""
    hip = sl.lib()  # (symbols of the runtime that the library itself uses)
    hip.hipSetDevice.restype = hip.hipGetLastError.restype = ctypes.c_int
    M, T, D, F = 96, 160, 64, 72
    dt = torch.bfloat16
    t = lambda *s, d=dt: torch.randn(*s, device="cuda").to(d)
    f32 = torch.float32
    n = sl.layer_dims(1, M, D, F, "bf16")
    sc = sl.layer_dims(2, T, 8, F, "bf16")
    one = sl.layer_dims(2, 1, 8, F, "bf16")
    # (torch would meet the error as well: nothing is allocated between it and a call)
    ws = [sl.layer_workspace(d, c) for d, c in (
        (n, sl.LAYER_NORM_BACKWARD), (sc, sl.LAYER_GATED_SCAN), (sc, sl.LAYER_GATED_SCAN_BACKWARD),
        (n, sl.LAYER_GATED_PROJECT_BACKWARD), (n, sl.LAYER_OUTPUT_PROJECT_BACKWARD))]
    n0, sc0 = sl.layer_dims(1, 0, D, F, "bf16"), sl.layer_dims(2, 0, 8, F, "bf16")
    few, out = sl.layer_dims(1, 9, D, F, "bf16"), t(M, D)
    x, w, mean, rstd, dx, dw = t(M, D), t(D), t(M, d=f32), t(M, d=f32), t(M, D, d=f32), t(D, d=f32)
    v, h, hh, carry = [t(2 * T, F) for _ in range(7)], t(2, F, d=f32), t(2, F, d=f32), \
        sl.gated_scan_carry(sc)
    win, act, dwin = t(2 * F, D), t(M, F), t(2 * F, D, d=f32)
    y, wout, dwout = t(M, F), t(D, F), t(D, F, d=f32)
    calls = {
        "norm": lambda: sl.swimba_layer_norm(n, x, None, w, None, 1e-5, None, out, mean,
                                             rstd),
        "norm_backward": lambda: sl.swimba_layer_norm_backward(
            n, x, w, mean, rstd, x, None, dx, dw, None, ws[0]),
        "scan": lambda: sl.swimba_gated_scan(sc, v[0], v[1], v[2], None, h, v[3], hh, carry,
                                             ws[1]),
        "scan_backward": lambda: sl.swimba_gated_scan_backward(
            sc, v[0], v[1], v[2], None, carry, v[3], h, v[4], v[5], v[6], hh,
            ws[2]),
        "step": lambda: sl.swimba_gated_step(one, *v[:3], h, hh, v[3]),
        "project": lambda: sl.swimba_gated_project(n, x, win, 0, None, act),
        "project_few": lambda: sl.swimba_gated_project(few, x, win, 0, None, act),
        "project_backward": lambda: sl.swimba_gated_project_backward(
            n, x, win, act, 0, dx, dwin, ws[3]),
        "output_backward": lambda: sl.swimba_output_project_backward(
            n, y, wout, x, act, dwout, ws[4]),
        # without tokens: states copied, gradients cleared
        "norm_backward_none": lambda: sl.swimba_layer_norm_backward(
            n0, x, w, mean, rstd, x, None, dx, dw, None, ws[0]),
        "scan_none": lambda: sl.swimba_gated_scan(sc0, v[0], v[1], v[2], None, h, v[3], hh, None,
                                                  None),
        "project_backward_none": lambda: sl.swimba_gated_project_backward(
            n0, x, win, act, 0, dx, dwin, None),
    }
    for c in calls.values():
        c()
    torch.cuda.synchronize()
    failed = []
    for name, c in calls.items():
        error = hip.hipSetDevice(1 << 20)  # refused by the host: there is no such device
        assert error != 0
        try:
            c()
        except sb.SwimbaError as e:
            failed.append(f"{name}: {e}")
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert not failed, failed


def test_an_earlier_error_is_not_the_mixers_own():
    from gpu_util import upload
    from selective_ssm_parameter_amd import synth
    hip = sl.lib()
    hip.hipSetDevice.restype = hip.hipGetLastError.restype = ctypes.c_int
    wl = synth.small("errors", 51, batch=2, seqlen=200, d_model=128, nheads=2, headdim=64,
                     dstate=64, ngroups=1, n_experts=4, top_k=2, chunk=64, dtype=synth.BF16,
                     a_lo=0.9, a_hi=0.999)
    d = upload(wl, synth.make_inputs(wl))
    dims, one = sb.dims_of(wl), sb.dims_of(wl, seqlen=1)
    buf, grads, sep = sb.alloc_buffers(dims), sb.alloc_grads(dims), sb.alloc_separated(dims)
    a_exp = torch.rand(wl.n_experts, wl.nheads, device="cuda")
    log_decay = torch.empty(wl.batch, wl.nheads, wl.seqlen, device="cuda")
    w_out = torch.randn(wl.d_model, wl.d_inner, device="cuda").bfloat16()
    out = torch.empty(wl.tokens, wl.d_model, device="cuda", dtype=torch.bfloat16)
    ws, _ = sb.workspace(one, sb.CALL_DECODE, "cuda")
    h = torch.zeros(wl.batch, wl.nheads, wl.dstate, 64, device="cuda")
    y1 = torch.empty(wl.batch, wl.nheads, 64, dtype=torch.bfloat16, device="cuda")
    u1 = d["u"][:wl.batch].contiguous()
    dy = torch.randn(wl.tokens, wl.nheads, 64, device="cuda").bfloat16()
    w = (d["u"], d["w_router"], d["w_experts"])
    y = buf.y.view(wl.tokens, wl.d_inner)
    calls = {
        "forward": lambda: sb.forward(dims, *w, d["a"], None, buf),
        "forward_mixed": lambda: sb.forward_mixed(dims, *w, a_exp, None, buf, log_decay),
        "output_project": lambda: sb.swimba_output_project(dims, y, w_out, out),
        "backward": lambda: sb.backward(dims, *w, d["a"], None, dy, None, buf, grads),
        "decode": lambda: sb.swimba_decode_step(one, u1, w[1], w[2], d["a"], h, y1, None, ws),
        "separated": lambda: sb.separated_forward(dims, *w, d["a"], None, sep),
    }
    for c in calls.values():
        c()
    torch.cuda.synchronize()
    failed = []
    stream = torch.cuda.current_stream().cuda_stream  # (asked for without an error before it)
    real = sb._stream
    sb._stream = lambda s: stream
    try:
        for name, c in calls.items():
            assert hip.hipSetDevice(1 << 20) != 0
            try:
                c()
            except sb.SwimbaError as e:
                failed.append(f"{name}: {e}")
            hip.hipGetLastError()
    finally:
        sb._stream = real
    torch.cuda.synchronize()
    assert not failed, failed
