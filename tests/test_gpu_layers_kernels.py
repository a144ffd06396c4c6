"""Every kernel of the dense layer products against the fp64 oracle
(``layer_kernels.SHAPES``): element by element, and in the 2-norm, whose bound
would show a lost half of dz or a lost token in one tile."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import layer_kernels as lk
from layer_kernels import U
from oracle import layers as ol
from selective_ssm_parameter_amd import layers as sl
from test_gpu_layers import DT, check, dev, empty, gemm_case, half, host, rng

pytestmark = pytest.mark.gpu

IDS = ["x".join(map(str, s[:3])) + "-" + s[3] for s in lk.SHAPES]


def near(name, got, want, tol):
    d = lk.distance(host(got).reshape(want.shape), want)
    assert d <= tol, f"{name}: {d} in the 2-norm, bound {tol}"


@pytest.mark.parametrize("M,D,F,dtype", lk.SHAPES, ids=IDS)
def test_gated_project_and_backward(M, D, F, dtype):
    # (the oracle's erfc is slow: GELU at the smaller sizes)
    act = "gelu" if M * F < 700_000 and (M + D) % 2 else "silu"
    dt, x, w = gemm_case(M, D, F, dtype, seed=M + D + F)
    d = sl.layer_dims(1, M, D, F, dtype)
    code = {"silu": sl.ACT_SILU, "gelu": sl.ACT_GELU}[act]
    z, h = empty(M, 2 * F, dt=dt), empty(M, F, dt=dt)
    sl.swimba_gated_project(d, x, w, code, z, h)
    dh = dev(rng(7).standard_normal((M, F)), dt)
    dx, dw = empty(M, D), empty(2 * F, D)
    sl.swimba_gated_project_backward(d, x, w, dh, code, dx, dw,
                                     sl.layer_workspace(d, sl.LAYER_GATED_PROJECT_BACKWARD))
    xh, wh, dhh, hd = host(x), host(w), host(dh), half(dt)
    wanth, wantz = ol.gated_project(xh, wh, act)
    tz = D * U * (np.abs(xh) @ np.abs(wh).T)
    check("z", z, wantz, hd * np.abs(wantz) + tz)
    ga, ua = np.abs(wantz[:, :F]), np.abs(wantz[:, F:])
    va = np.abs(ol.activation(act, wantz[:, :F])[0])
    arel = (8 + 2 * ga + ga * ga) * U
    check("h", h, wanth, hd * np.abs(wanth) + 1.13 * tz[:, :F] * (ua + tz[:, F:])
          + va * tz[:, F:] + (arel + 2 * U) * va * ua)
    if dtype == "f32":
        near("z", z, wantz, U + lk.accumulation(D))
    wdx, wdw = ol.gated_project_backward(xh, wh, wantz, dhh, act)
    near("dx", dx, wdx, lk.dz_error(D, dtype) + lk.accumulation(2 * F))
    near("dw", dw, wdw, lk.dz_error(D, dtype) + lk.accumulation(M))
    for n, rows in (("dx", (dx, wdx)), ("dw", (dw, wdw))):
        assert torch.isfinite(rows[0]).all(), n


@pytest.mark.parametrize("M,D,F,dtype", lk.SHAPES, ids=IDS)
def test_output_project_backward(M, D, F, dtype):
    dt, r = DT[dtype], rng(M + 3 * D + F)
    y, w = dev(r.standard_normal((M, F)), dt), dev(r.standard_normal((D, F)) / F ** 0.5, dt)
    do = dev(r.standard_normal((M, D)), dt)
    d = sl.layer_dims(1, M, D, F, dtype)
    dy, dw = empty(M, F, dt=dt), empty(D, F)
    sl.swimba_output_project_backward(d, y, w, do, dy, dw,
                                      sl.layer_workspace(d, sl.LAYER_OUTPUT_PROJECT_BACKWARD))
    yh, wh, doh = host(y), host(w), host(do)
    wdy, wdw = ol.output_project_backward(yh, wh, doh)
    check("dy", dy, wdy, half(dt) * np.abs(wdy) + D * U * (np.abs(doh) @ np.abs(wh)))
    if dtype == "f32":
        near("dy", dy, wdy, U + lk.accumulation(D))
    near("dw", dw, wdw, lk.accumulation(M))
