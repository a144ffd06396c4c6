"""fp64 oracle of the selective state space layer and its loss (numpy, from the formulas).

The causal convolution, the selective scan token by token and the softmax cross
entropy, with their backward passes written out from the chain rule.
"""
from __future__ import annotations

import numpy as np

from .layers import sigmoid


def lengths(Bt, T, lens):
    return [T] * Bt if lens is None else [min(max(int(v), 0), T) for v in lens]


def silu(s):
    """-> silu(s), its derivative."""
    g = sigmoid(s)
    return s * g, g + s * g * sigmoid(-s)


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


# ------------------------------------------------------------------ convolution

def _inputs(x, state, b, n, W):
    C = x.shape[2]
    old = np.zeros((W - 1, C)) if state is None else state[b]
    return np.concatenate([old, x[b, :n]])


def causal_conv(x, weight, bias, act, state=None, lens=None):
    """x [Bt, T, C], weight [C, W], state [Bt, W - 1, C] or None -> y, the sums s (both
    [Bt, T, C], zeros past a length), the state behind the last token."""
    Bt, T, C = x.shape
    W = weight.shape[1]
    y, s, out = np.zeros((Bt, T, C)), np.zeros((Bt, T, C)), np.zeros((Bt, W - 1, C))
    for b, n in enumerate(lengths(Bt, T, lens)):
        inp = _inputs(x, state, b, n, W)
        for t in range(n):
            s[b, t] = (inp[t:t + W].T * weight).sum(1) + (0.0 if bias is None else bias)
        y[b, :n] = silu(s[b, :n])[0] if act else s[b, :n]
        out[b] = inp[n:]
    return y, s, out


def causal_conv_backward(x, weight, bias, act, dy, dstate=None, state=None, lens=None):
    """-> dx, dweight, dbias, dstate_in."""
    Bt, T, C = x.shape
    W = weight.shape[1]
    _, s, _ = causal_conv(x, weight, bias, act, state, lens)
    dx, dw, db = np.zeros((Bt, T, C)), np.zeros((C, W)), np.zeros(C)
    ds0 = np.zeros((Bt, W - 1, C))
    for b, n in enumerate(lengths(Bt, T, lens)):
        inp = _inputs(x, state, b, n, W)
        di = np.zeros((n + W - 1, C))
        if dstate is not None:
            di[n:] += dstate[b]
        for t in range(n):
            d = dy[b, t] * (silu(s[b, t])[1] if act else 1.0)
            db += d
            dw += d[:, None] * inp[t:t + W].T
            di[t:t + W] += d[None, :] * weight.T
        ds0[b], dx[b, :n] = di[:W - 1], di[W - 1:]
    return dx, dw, db, ds0


# ------------------------------------------------------------------ selective scan

def selective_scan(x, dt, z, B, C, A, D, bias, h_init, lens=None):
    """x, dt, z [Bt, T, Ch] (z may be None), B, C [Bt, T, G, N], A [Ch, N], D and bias
    [Ch] or None, h_init [Bt, Ch, N] or None -> y, u [Bt, T, Ch], the states before and
    after every token [Bt, T + 1, Ch, N] (the last one in use repeats past a length)."""
    Bt, T, Ch = x.shape
    G, N = B.shape[2:]
    grp = np.arange(Ch) // (Ch // G)
    hs = np.zeros((Bt, T + 1, Ch, N))
    if h_init is not None:
        hs[:, 0] = h_init
    y, u = np.zeros((Bt, T, Ch)), np.zeros((Bt, T, Ch))
    D = np.zeros(Ch) if D is None else D
    for b, n in enumerate(lengths(Bt, T, lens)):
        for t in range(T):
            if t >= n:
                hs[b, t + 1] = hs[b, t]
                continue
            delta = softplus(dt[b, t] + (0.0 if bias is None else bias))
            hs[b, t + 1] = (np.exp(delta[:, None] * A) * hs[b, t]
                            + (delta * x[b, t])[:, None] * B[b, t][grp])
            u[b, t] = (hs[b, t + 1] * C[b, t][grp]).sum(1) + D * x[b, t]
            y[b, t] = u[b, t] if z is None else u[b, t] * silu(z[b, t])[0]
    return y, u, hs


def selective_scan_backward(x, dt, z, B, C, A, D, bias, h_init, dy, dh_final, lens=None):
    """-> a dict of dx, ddt, dz (None without z), dB, dC, dA, dD, dbias, dh_init, and the
    gradients e of the states [Bt, T, Ch, N]."""
    Bt, T, Ch = x.shape
    G, N = B.shape[2:]
    per = Ch // G
    grp = np.arange(Ch) // per
    _, u, hs = selective_scan(x, dt, z, B, C, A, D, bias, h_init, lens)
    o = dict(dx=np.zeros(x.shape), ddt=np.zeros(x.shape), dB=np.zeros(B.shape),
             dC=np.zeros(C.shape), dA=np.zeros(A.shape), dD=np.zeros(Ch), dbias=np.zeros(Ch),
             dh_init=np.zeros((Bt, Ch, N)), e=np.zeros((Bt, T, Ch, N)),
             dz=None if z is None else np.zeros(x.shape))
    Dv = np.zeros(Ch) if D is None else D
    for b, n in enumerate(lengths(Bt, T, lens)):
        c = np.zeros((Ch, N)) if dh_final is None else np.array(dh_final[b], np.float64)
        for t in range(n - 1, -1, -1):
            v = dy[b, t]
            if z is not None:
                g, dg = silu(z[b, t])
                o["dz"][b, t] = v * u[b, t] * dg
                v = v * g
            pre = dt[b, t] + (0.0 if bias is None else bias)
            delta = softplus(pre)
            a = np.exp(delta[:, None] * A)
            e = C[b, t][grp] * v[:, None] + c
            o["e"][b, t] = e
            flow = e * a * hs[b, t]
            eb = (e * B[b, t][grp]).sum(1)
            o["dx"][b, t] = delta * eb + Dv * v
            o["ddt"][b, t] = ((flow * A).sum(1) + x[b, t] * eb) * sigmoid(pre)
            o["dA"] += flow * delta[:, None]
            o["dB"][b, t] = (e * (delta * x[b, t])[:, None]).reshape(G, per, N).sum(1)
            o["dC"][b, t] = (v[:, None] * hs[b, t + 1]).reshape(G, per, N).sum(1)
            o["dD"] += v * x[b, t]
            o["dbias"] += o["ddt"][b, t]
            c = a * e
        o["dh_init"][b] = c
    return o


# ------------------------------------------------------------------ cross entropy

def cross_entropy(x, w, targets):
    """x [M, D], w [V, D] -> loss [M] (0 where there is no target), lse [M], z [M, V]."""
    z = x @ w.T
    top = z.max(1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(z - top).sum(1))
    V = w.shape[0]
    ok = (targets >= 0) & (targets < V)
    return np.where(ok, lse - z[np.arange(len(z)), np.where(ok, targets, 0)], 0.0), lse, z


def cross_entropy_backward(x, w, targets, dloss):
    """-> dx, dw, dz."""
    _, lse, z = cross_entropy(x, w, targets)
    V = w.shape[0]
    ok = (targets >= 0) & (targets < V)
    dz = np.exp(z - lse[:, None])
    dz[np.arange(len(z))[ok], targets[ok]] -= 1.0
    dz *= np.where(ok, dloss, 0.0)[:, None]
    return dz @ w, dz.T @ x, dz
