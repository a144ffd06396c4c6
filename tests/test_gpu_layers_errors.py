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
