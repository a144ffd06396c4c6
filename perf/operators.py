"""Cases, plain forms and calls of the operators around the mixer.

Four operators of ``include/swimba_layers.h``: the layer norm, the gated
linear recurrence, the gated feed-forward projection and the backward of the
output projection. ``listed()`` gives fixed cases, ``draw(rng)`` more of the
same ranges; ``prepare`` makes a case's inputs on the GPU, ``run`` is one pass
(elementary torch operations in 32 bits while ``own`` is false, the library's
calls while it is true), ``exact`` the same outputs from the definition in 64
bits, ``work`` the bytes and operations a pass cannot do without.

Kinds: ``norm`` (forward), ``norm_train`` (forward and backward), ``scan``,
``scan_train``, ``step`` (one token), ``gated`` (forward), ``gated_train``
(forward keeping the pre-activations, and backward), ``outproj_bwd``.
"""
from __future__ import annotations

import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-5


def _tdt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the pre-norm of one decode step: 256 sequences, d_model 2048
        dict(name="norm_decode", kind="norm", batch=256, seqlen=1, d=2048, residual=True,
             bias=True, dtype=BF16),
        # the pre-norm with the residual add of a 4 x 8192-token prefill
        dict(name="norm_prefill", kind="norm", batch=4, seqlen=8192, d=2048, residual=True,
             bias=True, dtype=BF16),
        # a training step's pre-norm, 8 x 2048 tokens; the mixer's input gradient is float32
        dict(name="norm_train", kind="norm_train", batch=8, seqlen=2048, d=768, residual=False,
             bias=True, dy_f32=True, dtype=BF16),
        # one decode step of the recurrence: 256 sequences, 4096 channels
        dict(name="step_decode", kind="step", batch=256, seqlen=1, d=4096, gate=True, dtype=BF16),
        # a long-context prefill: one sequence of 65536 tokens
        dict(name="scan_long", kind="scan", batch=1, seqlen=65536, d=2048, gate=True,
             ragged=False, pad=0, dtype=BF16),
        # training on a padded batch of sequences of different lengths
        dict(name="scan_train", kind="scan_train", batch=8, seqlen=2048, d=1536, gate=True,
             ragged=True, pad=0, dtype=BF16),
        # float32, odd length, odd channel count, rows inside a wider tensor
        dict(name="scan_train_odd", kind="scan_train", batch=3, seqlen=1777, d=1001, gate=True,
             ragged=True, pad=5, dtype=F32),
        # a feed-forward decode step of 16 sequences (bound by streaming the weights)
        dict(name="gated_decode", kind="gated", batch=16, seqlen=1, d=2048, f=4096, act="silu",
             dtype=BF16),
        # a feed-forward prefill of 4 x 8192 tokens
        dict(name="gated_prefill", kind="gated", batch=4, seqlen=8192, d=2048, f=4096,
             act="silu", dtype=BF16),
        # a training step, 8 x 2048 tokens
        dict(name="gated_train", kind="gated_train", batch=8, seqlen=2048, d=768, f=2048,
             act="gelu", dtype=BF16),
        # the output projection's backward of a training step, 8 x 2048 tokens
        dict(name="outproj_bwd", kind="outproj_bwd", batch=8, seqlen=2048, d=768, f=1536,
             dtype=BF16),
        # the same in float32 at ragged sizes
        dict(name="outproj_bwd_odd", kind="outproj_bwd", batch=1, seqlen=999, d=480, f=1016,
             dtype=F32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm_train", "scan", "scan_train", "step", "gated",
                       "gated_train", "outproj_bwd"])
    dtype = rng.choice([BF16, BF16, F32])
    if kind in ("norm", "norm_train"):
        d = _log_int(rng, 16, 8192)
        rows = _log_int(rng, 1, min(32768, (1 << 25) // d))
        batch = 1 if rows < 4 else rng.choice([1, 2, 3])
        case = dict(kind=kind, batch=batch, seqlen=rows // batch, d=d,
                    residual=rng.random() < 0.5, bias=rng.random() < 0.7, dtype=dtype)
        if kind == "norm_train":
            case["dy_f32"] = dtype == F32 or rng.random() < 0.5
        return case
    if kind == "step":
        d = _log_int(rng, 64, 8192)
        return dict(kind=kind, batch=_log_int(rng, 1, 512), seqlen=1, d=d,
                    gate=rng.random() < 0.7, dtype=dtype)
    if kind in ("scan", "scan_train"):
        d = _log_int(rng, 64, 4096)
        if rng.random() < 0.7:
            d = (d + 7) // 8 * 8
        tokens = _log_int(rng, 1, min(65536, (1 << 25) // d))
        batch = 1 if tokens < 16 else rng.choice([1, 2, 5, 8])
        return dict(kind=kind, batch=batch, seqlen=max(1, tokens // batch), d=d,
                    gate=rng.random() < 0.7, ragged=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 8, 3]), dtype=dtype)
    cap = 1 << (35 if dtype == BF16 else 32)  # rows * d * f
    d = 8 * _log_int(rng, 8, 320)
    f = 8 * _log_int(rng, 8, 640)
    rows = _log_int(rng, 1, max(1, min(16384, cap // (d * f))))
    batch = 1 if rows < 4 else rng.choice([1, 3])
    case = dict(kind=kind, batch=batch, seqlen=rows // batch, d=d, f=f, dtype=dtype)
    if kind != "outproj_bwd":
        case["act"] = rng.choice(["silu", "gelu"])
    return case


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _tdt(case)
    B, T, D = case["batch"], case["seqlen"], case["d"]
    M, kind = B * T, case["kind"]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        t = torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)
        return t.mul_(std).add_(mean).to(dtype)

    st = {"case": case}
    if kind in ("norm", "norm_train"):
        # a residual stream: rows of different scales around a common offset
        scale = torch.exp(torch.randn(M, 1, generator=gen, device=dev))
        st["x"] = (normal(M, D, dtype=torch.float32) * scale + 0.5).to(dt)
        st["res"] = normal(M, D) if case["residual"] else None
        st["w"] = normal(D, std=0.1, mean=1.0)
        st["b"] = normal(D, std=0.1) if case["bias"] else None
        if kind == "norm_train":
            st["dy"] = normal(M, D, dtype=torch.float32 if case["dy_f32"] else dt)
            st["dres"] = normal(M, D, dtype=torch.float32)
    elif kind in ("scan", "scan_train", "step"):
        pad = case.get("pad", 0)
        n = 3 if case["gate"] else 2
        # x | f | o as one projection leaves them: column ranges of one tensor
        wide = torch.zeros(M, n * D + pad, dtype=dt, device=dev)
        wide[:, :D] = normal(M, D)
        # forget logits with a different memory per channel, from about 1 to 1000 tokens
        bias = torch.rand(D, generator=gen, device=dev) * 8 - 1
        wide[:, D:2 * D] = (normal(M, D, dtype=torch.float32) + bias).to(dt)
        if case["gate"]:
            wide[:, 2 * D:3 * D] = normal(M, D)
        st["wide"] = wide
        st["x"], st["f"] = wide[:, :D], wide[:, D:2 * D]
        st["o"] = wide[:, 2 * D:3 * D] if case["gate"] else None
        if D * dt.itemsize % 16:
            # column ranges of an odd width are not 16-byte aligned: a program copies them out
            st["x"], st["f"] = [_aligned(t, pad) for t in (st["x"], st["f"])]
            st["o"] = _aligned(st["o"], pad) if case["gate"] else None
        st["h0"] = normal(B, D, dtype=torch.float32)
        st["lens"] = None
        if case.get("ragged"):
            lens = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
            lens[0] = T
            st["lens"] = lens
        if kind == "scan_train":
            st["dy"] = normal(M, D)
            st["dh"] = normal(B, D, dtype=torch.float32)
    elif kind in ("gated", "gated_train"):
        F = case["f"]
        st["x"] = normal(M, D)
        st["w_in"] = normal(2 * F, D, std=D ** -0.5)
        if kind == "gated_train":
            st["dh"] = normal(M, F)
    else:
        F = case["f"]
        st["y"] = normal(M, F)
        st["w_out"] = normal(D, F, std=F ** -0.5)
        st["dout"] = normal(M, D)
    if own:
        _prepare_own(st)
    return st


def _aligned(t, pad):
    """A copy of t's rows in a tensor of its own whose rows are `pad` elements wider."""
    buf = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def _prepare_own(st):
    """What a program that calls the library keeps: dims, outputs, workspaces."""
    from selective_ssm_parameter_amd import layers as sl
    case = st["case"]
    B, T, D = case["batch"], case["seqlen"], case["d"]
    M, kind, dt = B * T, case["kind"], _tdt(case)
    F = case.get("f", D)
    dims = sl.layer_dims(B, T, D, F, case["dtype"])
    st["dims"] = dims
    f32 = torch.float32

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if kind in ("norm", "norm_train"):
        st["sum"] = empty(M, D) if case["residual"] else None
        st["y"] = empty(M, D)
        if kind == "norm_train":
            st["mean"], st["rstd"] = empty(M, dtype=f32), empty(M, dtype=f32)
            st["dx"], st["dw"] = empty(M, D, dtype=f32), empty(D, dtype=f32)
            st["db"] = empty(D, dtype=f32) if case["bias"] else None
            st["ws"] = sl.layer_workspace(dims, sl.LAYER_NORM_BACKWARD)
    elif kind in ("scan", "scan_train", "step"):
        st["y"] = empty(M, D)
        st["h"] = empty(B, D, dtype=f32)
        if kind != "step":
            st["ws"] = sl.layer_workspace(dims, sl.LAYER_GATED_SCAN)
        if kind == "scan_train":
            st["carry"] = sl.gated_scan_carry(dims)
            st["dx"], st["df"] = empty(M, D), empty(M, D)
            st["do"] = empty(M, D) if case["gate"] else None
            st["dh0"] = empty(B, D, dtype=f32)
            st["ws_b"] = sl.layer_workspace(dims, sl.LAYER_GATED_SCAN_BACKWARD)
    elif kind in ("gated", "gated_train"):
        st["h"] = empty(M, F)
        st["act"] = {"silu": sl.ACT_SILU, "gelu": sl.ACT_GELU}[case["act"]]
        if kind == "gated_train":
            st["z"] = empty(M, 2 * F)
            st["dx"], st["dw"] = empty(M, D, dtype=f32), empty(2 * F, D, dtype=f32)
            st["ws"] = sl.layer_workspace(dims, sl.LAYER_GATED_PROJECT_BACKWARD)
    else:
        st["dy"], st["dw"] = empty(M, F), empty(D, F, dtype=f32)
        st["ws"] = sl.layer_workspace(dims, sl.LAYER_OUTPUT_PROJECT_BACKWARD)


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from selective_ssm_parameter_amd import layers as sl
    case, kind, dims = st["case"], st["case"]["kind"], st["dims"]
    if kind == "norm":
        sl.swimba_layer_norm(dims, st["x"], st["res"], st["w"], st["b"], EPS, st["sum"], st["y"])
        return {"y": st["y"], "sum": st["sum"]} if case["residual"] else {"y": st["y"]}
    if kind == "norm_train":
        sl.swimba_layer_norm(dims, st["x"], st["res"], st["w"], st["b"], EPS, st["sum"], st["y"],
                             st["mean"], st["rstd"])
        s = st["sum"] if case["residual"] else st["x"]
        sl.swimba_layer_norm_backward(dims, s, st["w"], st["mean"], st["rstd"], st["dy"],
                                      st["dres"], st["dx"], st["dw"], st["db"], st["ws"])
        out = {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"], "dx": st["dx"],
               "dw": st["dw"]}
        if case["bias"]:
            out["db"] = st["db"]
        return out
    if kind == "step":
        sl.swimba_gated_step(dims, st["x"], st["f"], st["o"], st["h0"], st["h"], st["y"])
        return {"y": st["y"], "h": st["h"]}
    if kind in ("scan", "scan_train"):
        carry = st.get("carry")
        sl.swimba_gated_scan(dims, st["x"], st["f"], st["o"], st["lens"], st["h0"], st["y"],
                             st["h"], carry, st["ws"])
        out = {"y": st["y"], "h": st["h"]}
        if kind == "scan_train":
            sl.swimba_gated_scan_backward(dims, st["x"], st["f"], st["o"], st["lens"], carry,
                                          st["dy"], st["dh"], st["dx"], st["df"], st["do"],
                                          st["dh0"], st["ws_b"])
            out.update(dx=st["dx"], df=st["df"], dh0=st["dh0"])
            if case["gate"]:
                out["do"] = st["do"]
        return out
    if kind == "gated":
        sl.swimba_gated_project(dims, st["x"], st["w_in"], st["act"], None, st["h"])
        return {"h": st["h"]}
    if kind == "gated_train":
        sl.swimba_gated_project(dims, st["x"], st["w_in"], st["act"], st["z"], st["h"])
        sl.swimba_gated_project_backward(dims, st["x"], st["w_in"], st["dh"], st["act"],
                                         st["dx"], st["dw"], st["ws"])
        return {"h": st["h"], "z": st["z"], "dx": st["dx"], "dw": st["dw"]}
    sl.swimba_output_project_backward(dims, st["y"], st["w_out"], st["dout"], st["dy"], st["dw"],
                                      st["ws"])
    return {"dy": st["dy"], "dw": st["dw"]}


# ---- plain forms: elementary operations in 32 bits, rounded once at the end

def _scan_doubling(a, b):
    """All prefixes of h = a h + b along dim 1 (h before the first: zero), by doubling."""
    a, b = a.clone(), b.clone()
    n, step = a.shape[1], 1
    while step < n:
        b[:, step:] = b[:, step:] + a[:, step:] * b[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return b


def _plain_act(name, g):
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    phi = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * phi, phi + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _run_plain(st):
    case = st["case"]
    kind, dt = case["kind"], _tdt(case)
    B, T, D = case["batch"], case["seqlen"], case["d"]
    if kind in ("norm", "norm_train"):
        s = st["x"].float()
        out = {}
        if case["residual"]:
            out["sum"] = (s + st["res"].float()).to(dt)
            s = out["sum"].float()
        mean = s.mean(1, keepdim=True)
        c = s - mean
        rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
        xh = c * rstd
        w = st["w"].float()
        y = xh * w
        if case["bias"]:
            y = y + st["b"].float()
        out["y"] = y.to(dt)
        if kind == "norm":
            return out
        out.pop("sum", None)
        dy = st["dy"].float()
        g = dy * w
        out["mean"], out["rstd"] = mean[:, 0], rstd[:, 0]
        out["dx"] = st["dres"] + rstd * (g - g.mean(1, keepdim=True)
                                         - xh * (g * xh).mean(1, keepdim=True))
        out["dw"] = (dy * xh).sum(0)
        if case["bias"]:
            out["db"] = dy.sum(0)
        return out
    if kind in ("scan", "scan_train", "step"):
        x = st["x"].float().reshape(B, T, D)
        fl = st["f"].float().reshape(B, T, D)
        f, g = 1 / (1 + torch.exp(-fl)), 1 / (1 + torch.exp(fl))
        live = None
        if st["lens"] is not None:
            live = (torch.arange(T, device=x.device)[None, :] < st["lens"][:, None])[:, :, None]
            f = torch.where(live, f, torch.ones((), device=x.device))
            g = torch.where(live, g, torch.zeros((), device=x.device))
        b = g * x
        b[:, 0] += f[:, 0] * st["h0"]
        h = _scan_doubling(f, b)
        if case["gate"]:
            ol = st["o"].float().reshape(B, T, D)
            so = 1 / (1 + torch.exp(-ol))
            o = ol * so
            y = h * o
        else:
            y = h
        if live is not None:
            y = y * live
        out = {"y": y.to(dt).reshape(B * T, D), "h": h[:, -1].contiguous()}
        if kind != "scan_train":
            return out
        dy = st["dy"].float().reshape(B, T, D)
        if live is not None:
            dy = dy * live
        e = dy * o if case["gate"] else dy.clone()
        e[:, -1] += st["dh"]
        fn = torch.cat([f[:, 1:], torch.zeros_like(f[:, :1])], 1)
        e = _scan_doubling(fn.flip(1), e.flip(1)).flip(1)
        hp = torch.cat([st["h0"][:, None], h[:, :-1]], 1)
        out["dx"] = (g * e).to(dt).reshape(B * T, D)
        out["df"] = (f * g * e * (hp - x)).to(dt).reshape(B * T, D)
        out["dh0"] = f[:, 0] * e[:, 0]
        if case["gate"]:
            out["do"] = (dy * h * so * (1 + ol * (1 - so))).to(dt).reshape(B * T, D)
        return out
    if kind in ("gated", "gated_train"):
        F = case["f"]
        x, w = st["x"].float(), st["w_in"].float()
        z = x @ w.t()
        act, dact = _plain_act(case["act"], z[:, :F])
        out = {"h": (act * z[:, F:]).to(dt)}
        if kind == "gated":
            return out
        dh = st["dh"].float()
        dz = torch.cat([dh * z[:, F:] * dact, dh * act], 1)
        out["z"] = z.to(dt)
        out["dx"] = dz @ w
        out["dw"] = dz.t() @ x
        return out
    dout = st["dout"].float()
    return {"dy": (dout @ st["w_out"].float()).to(dt), "dw": dout.t() @ st["y"].float()}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """run's outputs from the definitions in float64 (the recurrence token by token)."""
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    kind = case["kind"]
    B, T, D = case["batch"], case["seqlen"], case["d"]
    f64 = torch.float64
    if kind in ("norm", "norm_train"):
        s = st["x"].to(f64)
        out = {}
        if case["residual"]:
            tot = s + st["res"].to(f64)
            out["sum"] = tot
            s = tot.to(_tdt(case)).to(f64)  # the norm is of the stored sum
        mean = s.sum(1) / D
        var = ((s - mean[:, None]) ** 2).sum(1) / D
        rstd = (var + EPS) ** -0.5
        xh = (s - mean[:, None]) * rstd[:, None]
        out["y"] = xh * st["w"].to(f64) + (st["b"].to(f64) if case["bias"] else 0.0)
        if kind == "norm":
            return out
        out.pop("sum", None)
        dy = st["dy"].to(f64)
        dxh = dy * st["w"].to(f64)
        m1, m2 = dxh.sum(1, keepdim=True) / D, (dxh * xh).sum(1, keepdim=True) / D
        out.update(mean=mean, rstd=rstd,
                   dx=st["dres"].to(f64) + (dxh - m1 - xh * m2) * rstd[:, None],
                   dw=torch.einsum("md,md->d", dy, xh))
        if case["bias"]:
            out["db"] = dy.sum(0)
        return out
    if kind in ("scan", "scan_train", "step"):
        lens = [T] * B if st["lens"] is None else st["lens"].tolist()
        lens_t = torch.tensor(lens, device="cuda")[:, None]
        x = st["x"].to(f64).reshape(B, T, D)
        f = torch.sigmoid(st["f"].to(f64)).reshape(B, T, D)
        gate = case["gate"]
        ol = st["o"].to(f64).reshape(B, T, D) if gate else None
        hs = torch.empty(B, T + 1, D, dtype=f64, device="cuda")
        hs[:, 0] = st["h0"].to(f64)
        gx = (1 - f) * x
        keep_t = lens_t > torch.arange(T, device="cuda")[None, :]
        full = min(lens) == T
        for t in range(T):
            torch.addcmul(gx[:, t], f[:, t], hs[:, t], out=hs[:, t + 1])
            if not full:
                hs[:, t + 1] = torch.where(keep_t[:, t, None], hs[:, t + 1], hs[:, t])
        h, hp = hs[:, 1:], hs[:, :-1]
        y = h * (ol * torch.sigmoid(ol)) if gate else h
        y = torch.where(keep_t[:, :, None], y, torch.zeros((), dtype=f64, device="cuda"))
        out = {"y": y.reshape(B * T, D), "h": h[:, -1]}
        if kind != "scan_train":
            return out
        dy = st["dy"].to(f64).reshape(B, T, D)
        sig = torch.sigmoid(ol) if gate else None
        es = torch.zeros(B, T, D, dtype=f64, device="cuda")
        nxt = st["dh"].to(f64)  # the gradient of the state behind token t
        for t in range(T - 1, -1, -1):
            k = keep_t[:, t, None]
            e = nxt + (dy[:, t] * ol[:, t] * sig[:, t] if gate else dy[:, t])
            es[:, t] = torch.where(k, e, es[:, t])
            nxt = torch.where(k, f[:, t] * e, nxt)
        out["dx"] = ((1 - f) * es).reshape(B * T, D)
        out["df"] = (f * (1 - f) * es * (hp - x)).reshape(B * T, D)
        out["dh0"] = nxt
        if gate:
            do = dy * h * (sig + ol * sig * (1 - sig))
            out["do"] = torch.where(keep_t[:, :, None], do,
                                    torch.zeros((), dtype=f64, device="cuda")).reshape(B * T, D)
        return out
    if kind in ("gated", "gated_train"):
        F = case["f"]
        x, w = st["x"].to(f64), st["w_in"].to(f64)
        a, u = x @ w[:F].t(), x @ w[F:].t()
        if case["act"] == "silu":
            s = torch.sigmoid(a)
            act, dact = a * s, s + a * s * (1 - s)
        else:
            cdf = torch.special.ndtr(a)
            act, dact = a * cdf, cdf + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        out = {"h": act * u}
        if kind == "gated":
            return out
        dh = st["dh"].to(f64)
        da, du = dh * u * dact, dh * act
        out["z"] = torch.cat([a, u], 1)
        out["dx"] = da @ w[:F] + du @ w[F:]
        out["dw"] = torch.cat([da.t() @ x, du.t() @ x], 0)
        return out
    dout = st["dout"].to(f64)
    return {"dy": dout @ st["w_out"].to(f64), "dw": dout.t() @ st["y"].to(f64)}


# ------------------------------------------------------------------ work

def work(case):
    kind = case["kind"]
    es = 2 if case["dtype"] == BF16 else 4
    B, T, D = case["batch"], case["seqlen"], case["d"]
    M = B * T
    n = M * D
    if kind in ("norm", "norm_train"):
        nb = 2 * n * es + (2 * n * es if case["residual"] else 0) + 2 * D * es
        if kind == "norm":
            return {"bytes": nb, "flops": 8 * n}
        dyb = 4 if case["dy_f32"] else es
        # forward and backward: the backward reads x and dy and dres, writes dx
        return {"bytes": nb + 8 * M + n * (es + dyb + 4 + 4) + 8 * D, "flops": 20 * n}
    if kind in ("scan", "scan_train", "step"):
        k = 3 if case["gate"] else 2
        nb = n * es * (k + 1) + 8 * B * D
        if kind != "scan_train":
            return {"bytes": nb, "flops": 12 * n}
        return {"bytes": nb + n * es * (2 * k + 1) + 8 * B * D, "flops": 32 * n}
    F = case["f"]
    if kind == "gated":
        return {"bytes": es * (M * D + 2 * F * D + M * F), "flops": 4 * M * D * F}
    if kind == "gated_train":
        fwd = es * (M * D + 2 * F * D + 3 * M * F)
        bwd = es * (M * D + 2 * F * D + 3 * M * F) + 4 * (M * D + 2 * F * D)
        return {"bytes": fwd + bwd, "flops": 12 * M * D * F}
    return {"bytes": es * (2 * M * F + D * F + M * D) + 4 * D * F, "flops": 4 * M * D * F}
