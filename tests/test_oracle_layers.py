"""Pins of the layer oracle (``oracle/layers.py``) that do not call it back:
closed forms, explicit products, and central differences of the forward for
every gradient."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import layers as ol


def rng(seed):
    return np.random.default_rng(seed)


def directional(fn, args, i, d, h=1e-6):
    up, dn = list(args), list(args)
    up[i], dn[i] = args[i] + h * d, args[i] - h * d
    return (fn(*up) - fn(*dn)) / (2 * h)


def check_grad(fn, args, grads, seed):
    """Every gradient against a central difference along a random direction.
    The values are O(1): the difference's error is about h^2 + 1e-16 / h."""
    r = rng(seed)
    for i, g in enumerate(grads):
        if g is None:
            continue
        d = r.standard_normal(args[i].shape)
        want = directional(fn, args, i, d)
        got = float(np.sum(g * d))
        assert abs(got - want) <= 1e-7 * (1 + abs(want) + np.sum(np.abs(g * d))), (i, got, want)


def test_sigmoid_ends():
    x = np.array([-800.0, -30.0, 0.0, 30.0, 800.0])
    s = ol.sigmoid(x)
    assert s[0] == 0.0 and s[4] == 1.0 and s[2] == 0.5
    assert abs(s[1] - math.exp(-30)) < 1e-25


def test_layer_norm_rows():
    r = rng(1)
    s = r.standard_normal((5, 7)) * 3 + 2
    w, b = r.standard_normal(7), r.standard_normal(7)
    y, mean, rstd = ol.layer_norm(s, w, b, 1e-5)
    for m in range(5):
        mu = sum(s[m]) / 7
        var = sum((v - mu) ** 2 for v in s[m]) / 7
        assert abs(mean[m] - mu) < 1e-14 and abs(rstd[m] - (var + 1e-5) ** -0.5) < 1e-12
        assert np.allclose(y[m], (s[m] - mu) / math.sqrt(var + 1e-5) * w + b, atol=1e-13)
    # one column: the row is its own mean
    y, _, _ = ol.layer_norm(s[:, :1], w[:1], b[:1], 1e-5)
    assert np.array_equal(y, np.broadcast_to(b[:1], (5, 1)))


def test_layer_norm_gradients():
    r = rng(2)
    s, w, b = r.standard_normal((4, 9)), r.standard_normal(9), r.standard_normal(9)
    dy, dres = r.standard_normal((4, 9)), r.standard_normal((4, 9))

    def loss(s, w, b):
        return float(np.sum(dy * ol.layer_norm(s, w, b, 1e-3)[0]) + np.sum(dres * s))

    check_grad(loss, [s, w, b], ol.layer_norm_backward(s, w, 1e-3, dy, dres), 3)


def test_gated_scan_explicit_products():
    r = rng(4)
    x, f = r.standard_normal((1, 6, 3)), r.standard_normal((1, 6, 3)) * 2
    h0 = r.standard_normal((1, 3))
    _, hs, hT = ol.gated_scan(x, f, None, h0)
    p = 1 / (1 + np.exp(-f[0]))
    for t in range(6):
        want = np.prod(p[:t + 1], axis=0) * h0[0]
        for s in range(t + 1):
            want = want + np.prod(p[s + 1:t + 1], axis=0) * (1 - p[s]) * x[0, s]
        assert np.allclose(hs[0, t], want, atol=1e-13)
    assert np.array_equal(hT[0], hs[0, 5])


def test_gated_scan_lengths_and_ends():
    r = rng(5)
    x, f, o = (r.standard_normal((3, 5, 2)) for _ in range(3))
    h0 = r.standard_normal((3, 2))
    x[1, 2:] = np.nan  # behind the length
    y, _, hT = ol.gated_scan(x, f, o, h0, lens=[0, 2, 9])
    assert np.array_equal(hT[0], h0[0]) and not y[0].any() and not y[1, 2:].any()
    assert np.array_equal(hT[1], ol.gated_scan(x[1:2, :2], f[1:2, :2], None, h0[1:2])[2][0])
    assert np.array_equal(y[2], ol.gated_scan(x[2:], f[2:], o[2:], h0[2:])[0][0])
    # f = 0 takes the input, f = 1 keeps the state
    big = np.full((1, 1, 2), 1e3)
    assert np.array_equal(ol.gated_scan(x[2:, :1], -big, None, h0[2:])[2], x[2:, 0])
    assert np.array_equal(ol.gated_scan(x[2:, :1], big, None, h0[2:])[2], h0[2:])


@pytest.mark.parametrize("gated", [True, False])
def test_gated_scan_gradients(gated):
    r = rng(6)
    x, f, o = (r.standard_normal((3, 7, 2)) for _ in range(3))
    h0, dh = r.standard_normal((3, 2)), r.standard_normal((3, 2))
    dy = r.standard_normal((3, 7, 2))
    lens = [7, 0, 4]

    def loss(x, f, o, h0):
        y, _, hT = ol.gated_scan(x, f, o if gated else None, h0, lens)
        return float(np.sum(dy * y) + np.sum(dh * hT))

    dx, df, do, dh0, _ = ol.gated_scan_backward(x, f, o if gated else None, h0, dy, dh, lens)
    assert (do is None) == (not gated)
    check_grad(loss, [x, f, o, h0], [dx, df, do, dh0], 7)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_project_and_gradients(act):
    r = rng(8)
    x, w = r.standard_normal((3, 4)), r.standard_normal((10, 4))
    h, z = ol.gated_project(x, w, act)
    for m in range(3):
        for c in range(5):
            g, u = float(x[m] @ w[c]), float(x[m] @ w[5 + c])
            a = g / (1 + math.exp(-g)) if act == "silu" else \
                g * 0.5 * (1 + math.erf(g / math.sqrt(2)))
            assert abs(h[m, c] - a * u) < 1e-13
    dh = r.standard_normal((3, 5))
    check_grad(lambda x, w: float(np.sum(dh * ol.gated_project(x, w, act)[0])), [x, w],
               ol.gated_project_backward(x, w, z, dh, act), 9)


def test_output_project_gradients():
    r = rng(10)
    y, w, do = r.standard_normal((3, 4)), r.standard_normal((5, 4)), r.standard_normal((3, 5))
    check_grad(lambda y, w: float(np.sum(do * (y @ w.T))), [y, w],
               ol.output_project_backward(y, w, do), 11)
