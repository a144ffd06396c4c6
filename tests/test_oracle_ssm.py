"""The oracle of the selective state space layer and its loss against central
differences of its own forward passes, and against plain identities."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import ssm as osm

# Central differences of a function of order 1 in float64: a step h = 1e-5 is off by
# f''' h^2 / 6 and by the rounding 2^-52 / h of values of order 10: below 1e-8 each.
STEP, TOL = 1e-5, 2e-7


def numeric(f, a):
    g = np.zeros(a.shape)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + STEP
        up = f()
        a[i] = keep - STEP
        g[i] = (up - f()) / (2 * STEP)
        a[i] = keep
    return g


def close(name, got, want):
    assert np.abs(got - want).max() <= TOL * (1 + np.abs(want).max()), name


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act,lens", [(1, None), (0, [5, 0, 1]), (1, [7, 2, 9])])
def test_causal_conv(W, act, lens):
    r = np.random.default_rng(W)
    x, w, b = r.standard_normal((3, 7, 2)), r.standard_normal((2, W)), r.standard_normal(2)
    s0, dy, ds = r.standard_normal((3, W - 1, 2)), r.standard_normal((3, 7, 2)), \
        r.standard_normal((3, W - 1, 2))

    def f():
        y, _, s = osm.causal_conv(x, w, b, act, s0, lens)
        return (y * dy).sum() + (s * ds).sum()

    dx, dw, db, ds0 = osm.causal_conv_backward(x, w, b, act, dy, ds, s0, lens)
    for name, got, a in (("dx", dx, x), ("dw", dw, w), ("db", db, b), ("ds0", ds0, s0)):
        close(name, got, numeric(f, a))


def test_causal_conv_in_pieces():
    r = np.random.default_rng(5)
    x, w = r.standard_normal((2, 9, 3)), r.standard_normal((3, 4))
    y, _, s = osm.causal_conv(x, w, None, 1)
    ya, _, sa = osm.causal_conv(x[:, :2], w, None, 1)
    yb, _, sb = osm.causal_conv(x[:, 2:], w, None, 1, sa)
    assert np.array_equal(y, np.concatenate([ya, yb], 1)) and np.array_equal(s, sb)


@pytest.mark.parametrize("G,gate,lens", [(1, True, None), (2, False, [4, 0]), (2, True, [3, 6])])
def test_selective_scan(G, gate, lens):
    r = np.random.default_rng(G)
    n = r.standard_normal
    Bt, T, Ch, N = 2, 5, 4, 3
    v = dict(x=n((Bt, T, Ch)), dt=n((Bt, T, Ch)), z=n((Bt, T, Ch)) if gate else None,
             B=n((Bt, T, G, N)), C=n((Bt, T, G, N)), A=-np.exp(n((Ch, N))), D=n(Ch), bias=n(Ch),
             h_init=n((Bt, Ch, N)))
    dy, dh = n((Bt, T, Ch)), n((Bt, Ch, N))

    def f():
        y, _, hs = osm.selective_scan(*v.values(), lens)
        return (y * dy).sum() + (hs[:, -1] * dh).sum()

    o = osm.selective_scan_backward(*v.values(), dy, dh, lens)
    for name in ("x", "dt", "z", "B", "C", "A", "D", "bias", "h_init"):
        if v[name] is not None:
            close(name, o["d" + name], numeric(f, v[name]))


def test_selective_scan_of_constant_inputs():
    """With A, dt, B, C and x constant the state is the geometric sum."""
    Ch, N, T = 3, 2, 40
    A = -np.array([[0.5, 1.0], [2.0, 0.1], [1.0, 3.0]])
    one = np.ones((1, T, Ch))
    y, _, hs = osm.selective_scan(one, 0 * one, None, np.ones((1, T, 1, N)),
                                  np.ones((1, T, 1, N)), A, None, None, None)
    d = np.log(2.0)
    a = np.exp(d * A)
    assert np.allclose(hs[0, -1], d * (1 - a ** T) / (1 - a), rtol=1e-12)
    assert np.allclose(y[0, -1], hs[0, -1].sum(1), rtol=1e-12)


def test_cross_entropy():
    r = np.random.default_rng(1)
    x, w, t = r.standard_normal((6, 4)), r.standard_normal((5, 4)), np.array([0, 4, -1, 5, 2, 2])
    g = r.standard_normal(6)
    dx, dw, dz = osm.cross_entropy_backward(x, w, t, g)
    f = lambda: (osm.cross_entropy(x, w, t)[0] * g).sum()
    close("dx", dx, numeric(f, x))
    close("dw", dw, numeric(f, w))
    assert np.abs(dz.sum(1)).max() < 1e-14  # a shift of all logits changes nothing
    loss, lse, z = osm.cross_entropy(x, w, t)
    assert loss[2] == loss[3] == 0 and np.allclose(np.exp(z - lse[:, None]).sum(1), 1)
