"""fp64 oracle of the layers around the mixer (numpy, from the formulas).

Layer norm with the residual add, the elementwise gated recurrence token by
token, the gated feed-forward projection, and their backward passes written
out from the chain rule; the output projection's backward.
"""
from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


# ------------------------------------------------------------------ layer norm

def layer_norm(s, weight, bias, eps):
    """s [M, D] -> y, mean [M], rstd [M]."""
    mean = s.sum(1) / s.shape[1]
    var = ((s - mean[:, None]) ** 2).sum(1) / s.shape[1]
    rstd = 1.0 / np.sqrt(var + eps)
    y = (s - mean[:, None]) * rstd[:, None] * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_backward(s, weight, eps, dy, dres=None):
    """-> ds, dweight, dbias."""
    _, mean, rstd = layer_norm(s, weight, None, eps)
    D = s.shape[1]
    xh = (s - mean[:, None]) * rstd[:, None]
    g = dy * weight
    ds = rstd[:, None] * (g - g.sum(1, keepdims=True) / D
                          - xh * (g * xh).sum(1, keepdims=True) / D)
    if dres is not None:
        ds = ds + dres
    return ds, (dy * xh).sum(0), dy.sum(0)


# ------------------------------------------------------------------ gated scan

def gated_scan(x, forget, gate, h_init, lens=None):
    """x, forget, gate [Bt, T, C] (gate may be None), h_init [Bt, C] or None ->
    y [Bt, T, C], h after every token [Bt, T, C], h_final [Bt, C]."""
    Bt, T, C = x.shape
    h = np.zeros((Bt, C)) if h_init is None else np.array(h_init, np.float64)
    y = np.zeros((Bt, T, C))
    hs = np.zeros((Bt, T, C))
    for b in range(Bt):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        for t in range(n):
            f, g = sigmoid(forget[b, t]), sigmoid(-forget[b, t])
            h[b] = f * h[b] + g * x[b, t]
            hs[b, t] = h[b]
            y[b, t] = h[b] if gate is None else h[b] * gate[b, t] * sigmoid(gate[b, t])
    return y, hs, h


def gated_scan_backward(x, forget, gate, h_init, dy, dh_final, lens=None):
    """-> dx, dforget, dgate (None without a gate), dh_init, and e = dl/dh_t."""
    Bt, T, C = x.shape
    _, hs, _ = gated_scan(x, forget, gate, h_init, lens)
    dx, df, es = np.zeros((Bt, T, C)), np.zeros((Bt, T, C)), np.zeros((Bt, T, C))
    dg = None if gate is None else np.zeros((Bt, T, C))
    dh0 = np.zeros((Bt, C))
    for b in range(Bt):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        c = np.zeros(C) if dh_final is None else np.array(dh_final[b], np.float64)
        for t in range(n - 1, -1, -1):
            prev = hs[b, t - 1] if t else (np.zeros(C) if h_init is None else h_init[b])
            f, g = sigmoid(forget[b, t]), sigmoid(-forget[b, t])
            if gate is None:
                e = c + dy[b, t]
            else:
                s = sigmoid(gate[b, t])
                e = c + dy[b, t] * gate[b, t] * s
                dg[b, t] = dy[b, t] * hs[b, t] * (s + gate[b, t] * s * sigmoid(-gate[b, t]))
            es[b, t] = e
            dx[b, t] = g * e
            df[b, t] = f * g * e * (prev - x[b, t])
            c = f * e
        dh0[b] = c
    return dx, df, dg, dh0, es


# ------------------------------------------------------------------ projections

def activation(act, g):
    """-> act(g), act'(g); act "silu" or "gelu"."""
    if act == "silu":
        s = sigmoid(g)
        return g * s, s + g * s * sigmoid(-g)
    phi = 0.5 * _erfc(-g / math.sqrt(2.0))
    return g * phi, phi + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)


def gated_project(x, w_in, act):
    """x [M, D], w_in [2F, D] -> h [M, F], z [M, 2F]."""
    z = x @ w_in.T
    F = w_in.shape[0] // 2
    return activation(act, z[:, :F])[0] * z[:, F:], z


def gated_dz(z, dh, act):
    F = z.shape[1] // 2
    v, d = activation(act, z[:, :F])
    return np.concatenate([dh * z[:, F:] * d, dh * v], axis=1)


def gated_project_backward(x, w_in, z, dh, act):
    """-> dx, dw_in."""
    dz = gated_dz(z, dh, act)
    return dz @ w_in, dz.T @ x


def output_project_backward(y, w_out, dout):
    """-> dy, dw_out."""
    return dout @ w_out, dout.T @ y
