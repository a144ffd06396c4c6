"""The convolution where a thread walks many rows in turn, and single tokens of the scan
where a thread takes two sequences: what large workloads run, against float64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ssm_bounds as sbd
import ssm_runs
from oracle import ssm as osm
from selective_ssm_parameter_amd import ssm
from ssm_bounds import DT, U, check, dev, empty, host

pytestmark = pytest.mark.gpu
F64 = torch.float64


# The convolution and its bounds as ssm_bounds.conv_bounds has them, on the device.

def silu(s):
    g = torch.sigmoid(s)
    return s * g, g + s * g * torch.sigmoid(-s)


def sums(full, w, b, T):
    """s_t of the inputs from token 1 - W on."""
    s = sum(full[:, k:k + T] * w[:, k] for k in range(w.shape[1]))
    return s if b is None else s + b


def transposed(full, w, d, ds, lens):
    """dx, dw, db, ds0 of the gradients d of the sums and ds of the state behind each length."""
    W, T = w.shape[1], d.shape[1]
    g = torch.zeros_like(full)
    for k in range(W):
        g[:, k:k + T] += d * w[:, k]
    if ds is not None:
        for b, n in enumerate(lens):
            g[b, n:n + W - 1] += ds[b]
    dw = torch.stack([(d * full[:, k:k + T]).sum((0, 1)) for k in range(W)], 1)
    dx = g[:, W - 1:].clone()
    for b, n in enumerate(lens):
        dx[b, n:] = 0
    return dx, dw, d.sum((0, 1)), g[:, :W - 1]


def close(name, got, want, tol):
    bad = ~((got.to(F64).reshape(want.shape) - want).abs() <= tol + sbd.TINY)
    assert not bool(bad.any()), (name, int(bad.sum()), torch.nonzero(bad)[0].tolist(),
                                 float(got.to(F64).reshape(want.shape)[bad][0]), float(want[bad][0]),
                                 float(tol.expand_as(want)[bad][0]))


@pytest.mark.parametrize("B,T,C,dtype,W,act,state,ragged,pad", ssm_runs.CONV)
def test_convolution_of_long_runs(B, T, C, dtype, W, act, state, ragged, pad):
    dt, per = DT[dtype], 16 // DT[dtype].itemsize
    gen = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    lens = [T] * B
    if ragged:  # inside a run, at a run's end, shorter than the window, none
        lens = [(T, T - 37, T // 48 * 48, 2, 0, 605)[b % 6] for b in range(B)]
    dims = ssm.ssm_dims(B, T, C, 1, 1, dtype)
    wide = torch.full((B * T, -(-(C + pad) // per) * per), float("nan"), dtype=dt, device="cuda")
    dy = r(B * T, C).to(dt)
    x = wide[:, :C]
    x.copy_(r(B * T, C))
    live = (torch.arange(T, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None])
    off = ~live.reshape(-1)
    x[off], dy[off] = float("nan"), float("nan")
    w, b = (r(C, W) * W ** -0.5).to(dt), r(C).to(dt)
    s0 = r(B, W - 1, C).to(dt) if state else None
    ds = r(B, W - 1, C) if state else None
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda") if ragged else None
    y, s1 = empty(B * T, C, dt=dt), empty(B, W - 1, C, dt=dt)
    ssm.swimba_causal_conv(dims, W, x, w, b, act, ld, s0, y, s1)
    dx = empty(*wide.shape, dt=dt)[:, :C]
    dw, db, ds0 = empty(C, W), empty(C), empty(B, W - 1, C)
    ssm.swimba_causal_conv_backward(dims, W, x, w, b, act, ld, s0, dy, ds, dx, dw, db, ds0,
                                    ssm.ssm_workspace(dims, ssm.CAUSAL_CONV_BACKWARD))
    # the same in float64
    m = live[..., None]
    xd = torch.where(m, x.reshape(B, T, C).to(F64), 0.0)
    full = torch.cat([torch.zeros(B, W - 1, C, dtype=F64, device="cuda") if s0 is None
                      else s0.to(F64), xd], 1)
    wd, bd, h = w.to(F64), b.to(F64), torch.finfo(dt).eps / 2
    s, mag = sums(full, wd, bd, T), sums(full.abs(), wd.abs(), bd.abs(), T)
    es = (W + 1) * U * mag
    v, slope = silu(s) if act else (s, torch.ones_like(s))
    rel = (2 * s.abs() + 8) * U
    ey, ed = (1.1 * es + rel * v.abs(),
              0.5 * es + rel * ((s.abs() + 1) * torch.sigmoid(s) + slope.abs())) if act \
        else (es, 0 * es)
    close("y", y, torch.where(m, v, 0.0), torch.where(m, h * v.abs() + ey * (1 + h), 0.0))
    want = torch.stack([full[i, n:n + W - 1] for i, n in enumerate(lens)])
    assert torch.equal(s1.to(F64), want)
    dyd = torch.where(m, dy.reshape(B, T, C).to(F64), 0.0)
    dsd = None if ds is None else ds.to(F64)
    got = dict(dx=dx, dw=dw, db=db, ds0=ds0)
    want = transposed(full, wd, dyd * slope, dsd, lens)
    mags = transposed(full.abs(), wd.abs(), dyd.abs() * slope.abs(), None if ds is None else dsd.abs(),
                      lens)
    errs = transposed(full.abs(), wd.abs(), dyd.abs() * (ed + 2 * U * slope.abs()), None, lens)
    n = B * T + 8  # (terms that a thread and then the second kernel add one after the other)
    for (name, g), a, e, q in zip(got.items(), want, errs, mags):
        tol = e + (n if name in ("dw", "db") else W + 1) * U * q
        close(name, g, a, h * a.abs() + tol * (1 + h) if name == "dx" else tol)


@pytest.mark.parametrize("Bt,Ch,N,G,gate", ssm_runs.STEP)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_single_tokens_of_two_sequences_a_thread(Bt, Ch, N, G, gate, dtype):
    r, dt = np.random.default_rng(Bt), DT[dtype]
    n = r.standard_normal
    t = {k: dev(n((Bt, Ch)), dt) for k in ("x", "dt", "z")}
    if not gate:
        t["z"] = None
    t.update(B=dev(n((Bt, G * N)), dt), C=dev(n((Bt, G * N)), dt), A=dev(-np.exp(n((Ch, N)))),
             D=dev(n(Ch)), bias=dev(n(Ch) - 1.0), h_init=dev(n((Bt, Ch, N))))
    d = ssm.ssm_dims(Bt, 1, Ch, N, G, dtype)
    inputs = [t[k] for k in ("x", "dt", "z", "B", "C", "A", "D", "bias")]
    h, y, y2 = empty(Bt + 1, Ch, N), empty(Bt + 1, Ch, dt=dt), empty(Bt, Ch, dt=dt)
    ssm.swimba_selective_step(d, *inputs, t["h_init"], h[:Bt], y[:Bt])
    assert bool(torch.isnan(h[Bt]).all()) and bool(torch.isnan(y[Bt]).all())  # no row more
    same = t["h_init"].clone()
    ssm.swimba_selective_step(d, *inputs, same, same, y2)
    assert torch.equal(same, h[:Bt]) and torch.equal(y2, y[:Bt])
    v = {k: None if a is None else host(a) for k, a in t.items()}
    for k in ("x", "dt", "z"):
        v[k] = None if v[k] is None else v[k][:, None]
    for k in ("B", "C"):
        v[k] = v[k].reshape(Bt, 1, G, N)
    tol = sbd.scan_bounds(v, None, dt)
    wy, _, hs = osm.selective_scan(*v.values())
    check("y", y[:Bt], wy, tol["y"])
    check("h", h[:Bt], hs[:, -1], tol["h"])
