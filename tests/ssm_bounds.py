"""Error bounds of the selective state space layer's calls, element by element.

U = 2^-24 is the fp32 unit roundoff. A value computed in fp32 by a few operations
is off by the sum of their roundings; hardware exp2, reciprocal and division are
within one unit in the last place (2 U). An argument that is off by d shifts an
exponential by d of itself. A sum of n terms is off by at most n U times the sum
of the magnitudes, whatever its order. Outputs of type t are rounded once, by
half(t) = eps(t) / 2 relative.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import ssm as osm
from oracle.layers import sigmoid

U = 2.0 ** -24
TINY = 2.0 ** -120  # (products of results near the smallest normal fp32 underflow)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def half(t):
    return torch.finfo(t).eps / 2


def dev(a, dt=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dt)


def host(t):
    return t.detach().to(torch.float64).cpu().numpy()


def empty(*shape, dt=torch.float32):
    return torch.full(shape, float("nan"), dtype=dt, device="cuda")


def check(name, got, want, tol):
    got = host(got).reshape(want.shape)
    tol = np.broadcast_to(tol, want.shape)
    bad = ~(np.abs(got - want) <= tol + TINY)
    assert not bad.any(), (
        f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
        f"{got[bad][0]} for {want[bad][0]}, bound {tol[bad][0]}")


# silu(s) for an s that is off by es: the exponential of s (2 U of its argument, 2 U of
# itself), a sum, a reciprocal, a product: sigmoid is off by (2 |s| + 6) U of itself at
# most; the slopes of silu and of its derivative are below 1.1 and 0.5.
def silu_error(s, es):
    v, d = osm.silu(s)
    rel = (2 * np.abs(s) + 8) * U
    return 1.1 * es + rel * np.abs(v), 0.5 * es + rel * (np.abs(s) + 1) * (sigmoid(s) + np.abs(d))


# ------------------------------------------------------------------ convolution

def conv_bounds(x, w, b, act, dy, ds, s0, lens, dt, runs):
    """Bounds of y, dx, dw, db, ds0; runs: terms that a thread and then the second kernel
    add one after the other."""
    W = w.shape[1]
    absb = None if b is None else np.abs(b)
    s0a = None if s0 is None else np.abs(s0)
    _, s, _ = osm.causal_conv(x, w, b, act, s0, lens)
    _, mag, _ = osm.causal_conv(np.abs(x), np.abs(w), absb, 0, s0a, lens)
    es = (W + 1) * U * mag
    y = osm.silu(s)[0] if act else s
    ey, ed = silu_error(s, es) if act else (es, 0 * es)
    out = {"y": half(dt) * np.abs(y) + ey * (1 + half(dt))}
    if dy is None:
        return out
    # ds = dy act'(s), off by |dy| ed and a rounding; dx, dw and db are linear in it
    slope = np.abs(osm.silu(s)[1]) if act else np.ones(s.shape)
    d_err = np.abs(dy) * (ed + 2 * U * slope)
    d_mag = np.abs(dy) * slope
    dsa = None if ds is None else np.abs(ds)
    lin = lambda g, e: osm.causal_conv_backward(np.abs(x), np.abs(w), absb, 0, g, e, s0a, lens)
    edx, edw, edb, es0 = lin(d_err, None)
    mdx, mdw, mdb, ms0 = lin(d_mag, dsa)
    dx = osm.causal_conv_backward(x, w, b, act, dy, ds, s0, lens)[0]
    out["dx"] = half(dt) * np.abs(dx) + (edx + (W + 1) * U * mdx) * (1 + half(dt))
    out["ds0"] = es0 + (W + 1) * U * ms0
    out["dw"] = edw + runs * U * mdw
    out["db"] = edb + runs * U * mdb
    return out


# ------------------------------------------------------------------ selective scan

def delta_error(pre):
    """Relative error of softplus(dt + bias): the sum is rounded (U |pre|, which moves
    softplus by at most that of itself where it is small, less elsewhere); exp(-|pre|) has
    2 U |pre| of its argument and 2 U; s = t / (2 + t) 4 U, the series 10 roundings, the last
    sum 2."""
    return (3 * np.abs(pre) + 20) * U


def scan_bounds(v, lens, dt, dy=None, dh=None):
    """Bounds of every output of the scan (and with dy of its backward). v: x, dt, z, B, C, A,
    D, bias, h_init as the oracle takes them.

    A state is a sum of products; each is off by the roundings on its path: a step's decay by
    r = |delta A| (delta's error + 3 U) + 2 U of itself, and by 2 U for the multiply-add. So a
    bound runs along with the recurrence of the magnitudes:
        M <- a M + |delta B x|,   E <- a (E + (r + 2 U) M) + (delta's error + 4 U) |delta B x|.
    Segments start from products of decays over all their tokens, exp(A sum delta): the sum of
    up to T steps is off by T U of itself (each lane adds T / 4 terms), the factor by the same
    times |A sum delta|, and q exp(-q) < 0.4; by 8 U more for each of the segments' multiply-
    adds: (0.4 (T + 20) + 8) U of the magnitude that enters. The gradients e likewise."""
    x, d, z, B, C, A, D, bias, h0 = v.values()
    Bt, T, Ch = x.shape
    G, N = B.shape[2:]
    per = Ch // G
    grp = np.arange(Ch) // per
    D = np.zeros(Ch) if D is None else D
    pre = d + (0.0 if bias is None else bias)
    delta, rd = osm.softplus(pre), delta_error(pre)
    seg = (0.4 * (T + 20) + 8 + T / 64 * 8) * U
    hM, hE = np.zeros((Bt, T + 1, Ch, N)), np.zeros((Bt, T + 1, Ch, N))
    if h0 is not None:
        hM[:, 0] = np.abs(h0)
    hE[:, 0] = seg * hM[:, 0]
    da = delta[..., None] * np.abs(A)
    a = np.exp(delta[..., None] * A)
    r = da * (rd[..., None] + 3 * U) + 2 * U
    ns = osm.lengths(Bt, T, lens)
    Bx, Cx = np.abs(B)[:, :, grp], np.abs(C)[:, :, grp]
    for b, n in enumerate(ns):
        for t in range(T):
            if t >= n:
                hM[b, t + 1], hE[b, t + 1] = hM[b, t], hE[b, t]
                continue
            src = (delta[b, t] * np.abs(x[b, t]))[:, None] * Bx[b, t]
            hM[b, t + 1] = a[b, t] * hM[b, t] + src
            hE[b, t + 1] = a[b, t] * (hE[b, t] + (r[b, t] + 2 * U) * hM[b, t]) \
                + (rd[b, t][:, None] + 4 * U) * src
    hE = hE + seg * hM
    y, u, _ = osm.selective_scan(*v.values(), lens)
    uM = (Cx * hM[:, 1:]).sum(-1) + np.abs(D * x)
    uE = (Cx * hE[:, 1:]).sum(-1) + (N + 3) * U * uM
    if z is None:
        yE = uE
    else:
        g, dg = osm.silu(z)
        eg, edg = silu_error(z, 0 * z)
        yE = np.abs(g) * uE + uM * (eg + 2 * U * np.abs(g))
    out = {"y": half(dt) * np.abs(y) + yE * (1 + half(dt)), "h": hE[:, T]}
    if dy is None:
        return out
    o = osm.selective_scan_backward(*v.values(), dy, dh, lens)
    if z is None:
        vM, vE = np.abs(dy), 0 * dy
    else:
        vM, vE = np.abs(dy * g), np.abs(dy) * (eg + 2 * U * np.abs(g))
        out["dz"] = np.abs(dy) * (np.abs(dg) * uE + uM * (edg + 4 * U * np.abs(dg)))
    sM, sE = np.zeros((Bt, T, Ch, N)), np.zeros((Bt, T, Ch, N))  # of e_t
    c0M, c0E = np.zeros((Bt, Ch, N)), np.zeros((Bt, Ch, N))
    for b, n in enumerate(ns):
        cM = np.zeros((Ch, N)) if dh is None else np.abs(dh[b])
        cE = seg * cM
        for t in range(n - 1, -1, -1):
            src = vM[b, t][:, None] * Cx[b, t]
            sM[b, t] = src + cM
            sE[b, t] = cE + vE[b, t][:, None] * Cx[b, t] + 2 * U * sM[b, t]
            cM = a[b, t] * sM[b, t]
            cE = a[b, t] * (sE[b, t] + (r[b, t] + 2 * U) * sM[b, t])
        c0M[b], c0E[b] = cM, cE
    sE = sE + seg * sM
    out["dh_init"] = c0E + seg * c0M
    live = np.zeros((Bt, T, 1))
    for b, n in enumerate(ns):
        live[b, :n] = 1
    # flow = e a h_{t-1}
    hp, hpE = hM[:, :-1], hE[:, :-1]
    fM = sM * a * hp
    fE = a * (sE * hp + sM * hpE) + (r + 4 * U) * fM
    ebM, ebE = (sM * Bx).sum(-1), (sE * Bx).sum(-1) + (N + 2) * U * (sM * Bx).sum(-1)
    Aa = np.abs(A)
    ddM = (fM * Aa).sum(-1) + np.abs(x) * ebM
    ddE = (fE * Aa).sum(-1) + np.abs(x) * ebE + (N + 4) * U * ddM
    sg = sigmoid(pre)
    esg = (3 * np.abs(pre) + 8) * U * sg
    out["dx"] = delta * ebE + (rd + 3 * U) * delta * ebM + np.abs(D) * vE + 3 * U * np.abs(D) * vM
    out["ddt"] = sg * ddE + (esg + 2 * U * sg) * ddM
    # sums over tokens: 4 (dD, dbias: T / 4) a lane and block, then sequences and segments
    n = T + Bt * (T // 64 + 2) + 8
    out["dA"] = ((fE + (rd[..., None] + (n + 2) * U) * fM) * delta[..., None]).sum((0, 1))
    out["dD"] = ((vE + n * U * vM) * np.abs(x) * live).sum((0, 1))
    out["dbias"] = ((out["ddt"] + n * U * sg * ddM) * live).sum((0, 1))
    # sums over the group's channels
    ux = (delta * np.abs(x))[..., None]
    bM, bE = sM * ux, sE * ux + (rd[..., None] + (per + 4) * U) * sM * ux
    cE = hE[:, 1:] * vM[..., None] + hM[:, 1:] * (vE + (per + 4) * U * vM)[..., None]
    fold = lambda q: (q * live[..., None]).reshape(Bt, T, G, per, N).sum(3)
    out["dB"], out["dC"] = fold(bE), fold(cE)
    for k in ("dx", "ddt", "dz", "dB", "dC"):
        if k in out:
            out[k] = half(dt) * np.abs(o[k]) + out[k] * (1 + half(dt))
            if k in ("dx", "ddt", "dz"):
                out[k] = out[k] * live
    return out


# ------------------------------------------------------------------ cross entropy

def loss_bounds(x, w, targets, dloss, dtype):
    """Bounds of loss, lse and with dloss of dx and dw.

    z is off by D U sum |x w|. lse: each exponential by (2 |z - m| + 4) U and its z's error; a
    lane adds 64 of them, then 4 lanes and up to 4 waves, then the tiles of 128 words or more
    four ways; |z - m| weighted by the softmax is at most log V + 1 (its entropy). dz = (p - 1)
    dloss with p off by the errors of z and lse, (2 |z - lse| + 4) U and two roundings; bf16
    problems hold it as two bf16 numbers, 2^-16 of itself. The products add V and M terms (and
    a piece of the vocabulary or a run of tokens at a time: no more)."""
    M, D = x.shape
    V = w.shape[0]
    loss, lse, z = osm.cross_entropy(x, w, targets)
    ez = D * U * (np.abs(x) @ np.abs(w).T)
    p = np.exp(z - lse[:, None])
    el = (p * ez).sum(1) + U * (64 + 8 + V / 512 + 8 + 2 * (np.log(V) + 1) + 6
                                + 4 * np.abs(lse) + 2 * np.abs(z).max(1))
    ok = (targets >= 0) & (targets < V)
    at = np.where(ok, targets, 0)
    zt, ezt = z[np.arange(M), at], ez[np.arange(M), at]
    out = {"lse": el, "loss": np.where(ok, el + ezt + U * (np.abs(lse) + np.abs(zt)), 0.0)}
    if dloss is None:
        return out
    ep = p * (ez + el[:, None] + (2 * np.abs(z - lse[:, None]) + 6) * U)
    dl = np.where(ok, np.abs(dloss), 0.0)[:, None]
    _, _, dz = osm.cross_entropy_backward(x, w, targets, dloss)
    a = np.abs(dz)
    ed = dl * ep + (3 * U + (2.0 ** -16 if dtype == "bf16" else 0.0)) * a
    out["dx"] = (ed + (V + 8) * U * a) @ np.abs(w)
    out["dw"] = (ed + (M + 8) * U * a).T @ np.abs(x)
    return out
