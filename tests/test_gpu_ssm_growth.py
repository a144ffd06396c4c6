"""The selective scan with A > 0: states that grow from one token to the next, by more
than float32 holds over the tokens of a segment, while the answer itself stays finite."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ssm as osm
from selective_ssm_parameter_amd import ssm
from ssm_bounds import DT, U, dev, empty, host

pytestmark = pytest.mark.gpu


def case(T, Ch, N, growth, seed):
    """Steps and decays whose product is growth / T per token, all inputs positive (so that
    every sum is one of magnitudes)."""
    r = np.random.default_rng(seed)
    pos = lambda *s: r.uniform(0.5, 2.0, s)
    v = dict(x=pos(1, T, Ch), dt=np.full((1, T, Ch), np.log(np.expm1(0.5))), z=None,
             B=pos(1, T, 1, N), C=pos(1, T, 1, N), A=np.full((Ch, N), 2.0 * growth / T), D=None,
             bias=None, h_init=None)
    return v


def run(v, dtype, dy=None, dh=None):
    _, T, Ch = v["x"].shape
    N, dt = v["A"].shape[1], DT[dtype]
    d = ssm.ssm_dims(1, T, Ch, N, 1, dtype)
    t = {k: None if v[k] is None else dev(v[k].reshape(T, -1), dt) for k in ("x", "dt", "z", "B", "C")}
    A, h0 = dev(v["A"]), None if v["h_init"] is None else dev(v["h_init"])
    for k in ("x", "dt", "B", "C"):  # what the types hold
        v[k] = host(t[k]).reshape(v[k].shape)
    v["A"] = host(A)
    y, h, carry = empty(T, Ch, dt=dt), empty(1, Ch, N), ssm.selective_scan_carry(d)
    inputs = (t["x"], t["dt"], None, t["B"], t["C"], A, None, None, None)
    ssm.swimba_selective_scan(d, *inputs, h0, y, h, carry, ssm.ssm_workspace(d, ssm.SELECTIVE_SCAN))
    if dy is None:
        return y, h
    o = dict(dx=empty(T, Ch, dt=dt), ddt=empty(T, Ch, dt=dt), dz=None, dB=empty(T, N, dt=dt),
             dC=empty(T, N, dt=dt), dA=empty(Ch, N), dD=None, dbias=None, dh_init=empty(1, Ch, N))
    ssm.swimba_selective_scan_backward(
        d, *inputs, carry, dev(dy.reshape(T, Ch), dt), None if dh is None else dev(dh), *o.values(),
        ssm.ssm_workspace(d, ssm.SELECTIVE_SCAN_BACKWARD))
    return o


def tolerance(T, N, growth, dtype):
    """Relative. A step's factor exp(delta A) is off by its exponent's rounding and delta's 20 U
    of the exponent, and 4 U; a segment's by T U of its exponent for the sum of its steps, 4 U
    for its two halves and 4 U for the join; the sums over N states and the roundings of a
    gradient's products add N + 16; all of them along the T steps of the longest way. (All
    terms are positive: nothing cancels.)"""
    return ((24 + T) * growth + 8 * T + N + 16) * U + torch.finfo(DT[dtype]).eps / 2


def close(name, got, want, tol):
    got = host(got).reshape(want.shape)
    bad = ~(np.abs(got - want) <= tol * np.abs(want))
    assert not bad.any(), (name, int(bad.sum()), got[bad][0], want[bad][0], tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 5, 40])
@pytest.mark.parametrize("T,growth,live", [(2000, 12000.0, 10), (700, 3000.0, 15), (100, 1000.0, 5)])
def test_zero_states_stay_zero(T, growth, live, N, dtype):
    """Inputs only at the end (and gradients only at the beginning): the states before them are
    zeros, whatever they would have grown by."""
    v = case(T, 12, N, growth, seed=T + N)
    v["x"][:, :T - live] = 0
    y, h = run(v, dtype)
    wy, _, hs = osm.selective_scan(*v.values())
    tol = tolerance(T, N, growth * live / T, dtype)
    assert (host(y)[:T - live] == 0).all()
    close("y", y, wy, tol)
    close("h", h, hs[:, -1], tol)
    v = case(T, 12, N, growth, seed=T + N)
    v["x"][:] = 0
    dy = np.zeros((1, T, 12))
    dy[:, :live] = np.random.default_rng(1).uniform(0.5, 2.0, (1, live, 12))
    o = run(v, dtype, dy)
    want = osm.selective_scan_backward(*v.values(), host(dev(dy, DT[dtype])), None)
    assert (host(o["dx"])[live:] == 0).all()
    for k in ("dx", "dh_init"):
        close(k, o[k], want[k], tol)


@pytest.mark.parametrize("N", [16, 7])
def test_small_states_grow_into_range(N):
    """A state of 1e-30 that grows by more than float32 holds over one segment, to 1e30."""
    T, growth = 20, 138.0
    v = case(T, 12, N, growth, seed=N)
    v["x"][:] = 0
    v["h_init"] = np.full((1, 12, N), 1e-30)
    y, h = run(v, "f32")
    v["h_init"] = host(dev(v["h_init"]))
    wy, _, hs = osm.selective_scan(*v.values())
    tol = tolerance(T, N, growth, "f32")
    close("y", y, wy, tol)
    close("h", h, hs[:, -1], tol)


def forget(A, value):
    A = A.clone()
    A[::3, ::2] = value
    return A


@pytest.mark.parametrize("T,N,lens", [(37, 16, None), (700, 5, [700, 33, 0]), (130, 40, [130, 1, 64])])
def test_states_that_forget_at_once(T, N, lens):
    """A of -inf (what -exp of a large number is) gives the bits of the largest finite one,
    whose decays are zeros too, wherever a sequence ends."""
    Bt, Ch = 1 if lens is None else len(lens), 12
    gen = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    d, M = ssm.ssm_dims(Bt, T, Ch, N, 1, "f32"), Bt * T
    x, dt, z, B, C, dy = r(M, Ch), r(M, Ch), r(M, Ch), r(M, N), r(M, N), r(M, Ch)
    A, h0, dh = -torch.exp(r(Ch, N)), r(Bt, Ch, N), r(Bt, Ch, N)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    outs = []
    for value in (-torch.finfo(torch.float32).max, float("-inf")):
        Av = forget(A, value)
        y, h, carry = empty(M, Ch), empty(Bt, Ch, N), ssm.selective_scan_carry(d)
        carry.zero_()
        inputs = (x, dt, z, B, C, Av, None, None)
        ssm.swimba_selective_scan(d, *inputs, ln, h0, y, h, carry,
                                  ssm.ssm_workspace(d, ssm.SELECTIVE_SCAN))
        g = [empty(M, Ch) for _ in range(3)] + [empty(M, N), empty(M, N), empty(Ch, N), empty(Ch),
                                                empty(Ch), empty(Bt, Ch, N)]
        ssm.swimba_selective_scan_backward(d, *inputs, ln, carry, dy, dh, *g,
                                           ssm.ssm_workspace(d, ssm.SELECTIVE_SCAN_BACKWARD))
        d1 = ssm.ssm_dims(Bt, 1, Ch, N, 1, "f32")
        y1, h1, dt1 = empty(Bt, Ch), empty(Bt, Ch, N), dt[:Bt].clone()
        dt1[:, ::2] = -200.0  # a step of zero: the state stays
        ssm.swimba_selective_step(d1, x[:Bt], dt1, None, B[:Bt], C[:Bt], Av, None, None, h0, h1, y1)
        assert torch.equal(h1[:, ::2], h0[:, ::2])
        outs.append([y, h, *g, y1, h1])
    for i, (a, b) in enumerate(zip(*outs)):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b), i


def test_nan_decays_stay_nan():
    d, r = ssm.ssm_dims(1, 40, 4, 4, 1, "f32"), lambda *s: torch.randn(*s, device="cuda")
    A = -torch.ones(4, 4, device="cuda")
    A[2, 1] = float("nan")
    y, h = empty(40, 4), empty(1, 4, 4)
    ssm.swimba_selective_scan(d, r(40, 4), r(40, 4), None, r(40, 4), r(40, 4), A, None, None, None,
                              None, y, h, None, ssm.ssm_workspace(d, ssm.SELECTIVE_SCAN))
    bad = torch.isnan(h[0])
    assert bool(bad[2, 1]) and int(bad.sum()) == 1 and torch.isnan(y[:, 2]).all()
