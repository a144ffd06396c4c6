"""Cases, plain forms and calls of the selective state space layer and its loss.

Three operators of ``include/swimba_ssm.h``: the short causal convolution, the
selective scan that follows it, and the softmax cross entropy over a vocabulary
that trains a stack of such layers. ``listed()`` gives fixed cases, ``draw(rng)``
more of the same ranges; ``prepare`` makes a case's inputs on the GPU, ``run`` is
one pass (elementary torch operations in 32 bits while ``own`` is false, the
library's calls while it is true), ``exact`` the same outputs from the definition
in 64 bits, ``work`` the bytes and operations a pass cannot do without.

Kinds: ``conv``, ``conv_train`` (forward and backward), ``conv_step`` (one
token); ``ssm``, ``ssm_train``, ``ssm_step``; ``loss`` (forward), ``loss_train``.
"""
from __future__ import annotations

import math

import torch

own = False

BF16, F32 = "bf16", "f32"


def _tdt(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the convolution of one decode step: 256 sequences, 4096 channels
        dict(name="conv_decode", kind="conv_step", batch=256, seqlen=1, c=4096, width=4,
             silu=True, bias=True, pad=0, dtype=BF16),
        # a 4 x 8192-token prefill, x as the first half of the input projection's rows
        dict(name="conv_prefill", kind="conv", batch=4, seqlen=8192, c=4096, width=4, silu=True,
             bias=True, ragged=False, pad=4096, dtype=BF16),
        # training on a padded batch of sequences of different lengths, x as the first columns of
        # a projection that also gives the gate and 16 states each of B and C
        dict(name="conv_train", kind="conv_train", batch=8, seqlen=2048, c=1536, width=4,
             silu=True, bias=True, ragged=True, pad=1568, dtype=BF16),
        # float32, odd length and channel count, width 3, no activation
        dict(name="conv_train_odd", kind="conv_train", batch=3, seqlen=1777, c=1001, width=3,
             silu=False, bias=False, ragged=False, pad=0, dtype=F32),
        # one decode step of the recurrence: 256 sequences, 4096 channels, 16 states each
        dict(name="ssm_decode", kind="ssm_step", batch=256, seqlen=1, c=4096, n=16, g=1, gate=True,
             pad=0, dtype=BF16),
        # a long-context prefill: one sequence of 65536 tokens
        dict(name="ssm_long", kind="ssm", batch=1, seqlen=65536, c=2048, n=16, g=1, gate=True,
             ragged=False, pad=0, dtype=BF16),
        # training on a padded batch, the gate as columns of that projection
        dict(name="ssm_train", kind="ssm_train", batch=8, seqlen=2048, c=1536, n=16, g=1,
             gate=True, ragged=True, pad=1568, dtype=BF16),
        # float32, odd length, channels and states, two groups of B and C
        dict(name="ssm_train_odd", kind="ssm_train", batch=2, seqlen=777, c=402, n=11, g=2,
             gate=False, ragged=True, pad=3, dtype=F32),
        # scoring one short text: the largest share is streaming the vocabulary's weights
        dict(name="loss_score", kind="loss", batch=1, seqlen=128, d=2048, v=65536, dtype=BF16),
        # the loss of a long evaluation batch
        dict(name="loss_eval", kind="loss", batch=8, seqlen=2048, d=2048, v=65536, dtype=BF16),
        # the loss of a training step with its gradients, 8 x 2048 tokens
        dict(name="loss_train", kind="loss_train", batch=8, seqlen=2048, d=768, v=32768,
             dtype=BF16),
        # the same in float32, an odd vocabulary
        dict(name="loss_train_odd", kind="loss_train", batch=3, seqlen=333, d=480, v=10007,
             dtype=F32),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["conv", "conv_train", "conv_step", "ssm", "ssm_train", "ssm_train",
                       "ssm_step", "loss", "loss_train"])
    dtype = rng.choice([BF16, BF16, F32])
    if kind in ("loss", "loss_train"):
        d = 8 * _log_int(rng, 8, 256)
        v = _log_int(rng, 500, 131072)
        if rng.random() < 0.5:
            v = (v + 63) // 64 * 64
        cap = 1 << (38 if dtype == BF16 else 35)  # tokens * d * v
        tokens = _log_int(rng, 1, max(1, min(16384, cap // (d * v))))
        batch = 1 if tokens < 4 else rng.choice([1, 2, 3])
        return dict(kind=kind, batch=batch, seqlen=tokens // batch, d=d, v=v, dtype=dtype)
    step = kind.endswith("step")
    c = _log_int(rng, 16, 4096)
    if rng.random() < 0.7:
        c = (c + 7) // 8 * 8
    case = dict(kind=kind, c=c, dtype=dtype, pad=rng.choice([0, 0, 8, 64, c]))
    if step:
        case.update(batch=_log_int(rng, 1, 512), seqlen=1)
    else:
        tokens = _log_int(rng, 1, min(65536, (1 << 27) // c if kind[:4] == "conv"
                                      else (1 << 25) // c))
        batch = 1 if tokens < 16 else rng.choice([1, 1, 2, 5, 8])
        case.update(batch=batch, seqlen=max(1, tokens // batch), ragged=rng.random() < 0.5)
    if kind[:4] == "conv":
        case.update(width=rng.choice([2, 3, 4, 4, 4]), silu=rng.random() < 0.7,
                    bias=rng.random() < 0.7)
    else:
        case.update(n=rng.choice([4, 8, 16, 16, 16, 32, 64]) if rng.random() < 0.8
                    else rng.randint(1, 40),
                    g=2 if c % 2 == 0 and rng.random() < 0.2 else 1, gate=rng.random() < 0.7)
        if not step:  # no more work than the largest listed case
            while case["batch"] * case["seqlen"] * c * case["n"] > 1 << 29:
                case["n"] = (case["n"] + 1) // 2
    return case


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _tdt(case)
    B, T, kind = case["batch"], case["seqlen"], case["kind"]
    M = B * T
    f32 = torch.float32

    def normal(*shape, std=1.0, dtype=dt):
        t = torch.randn(*shape, generator=gen, device=dev, dtype=f32)
        return t.mul_(std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=dev, dtype=f32) * (hi - lo) + lo

    def rows(cols):
        """[M, cols] as the first columns of a tensor whose rows are `pad` elements wider (and
        start on 16 bytes)."""
        per = 16 // dt.itemsize
        wide = torch.zeros(M, -(-(cols + case["pad"]) // per) * per, dtype=dt, device=dev)
        wide[:, :cols] = normal(M, cols)
        return wide[:, :cols]

    st = {"case": case}
    if kind in ("loss", "loss_train"):
        D, V = case["d"], case["v"]
        st["x"] = normal(M, D)
        # logits of a spread of about 2 around each token
        st["w"] = normal(V, D, std=2.0 * D ** -0.5)
        tgt = torch.randint(0, V, (M,), generator=gen, device=dev, dtype=torch.int32)
        # one token in eight is not a target (the prompt's, or padding)
        skip = torch.rand(M, generator=gen, device=dev) < 0.125
        st["targets"] = torch.where(skip, torch.full_like(tgt, -1), tgt)
        if kind == "loss_train":
            # the mean over the tokens that count
            n = (~skip).sum().clamp(min=1)
            st["dloss"] = torch.where(skip, 0.0, 1.0 / n).to(f32)
    else:
        C = case["c"]
        st["lens"] = None
        if case.get("ragged"):
            lens = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
            lens[0] = T
            st["lens"] = lens
        if kind[:4] == "conv":
            W = case["width"]
            st["x"] = rows(C)
            st["w"] = normal(C, W, std=W ** -0.5)
            st["b"] = normal(C, std=0.1) if case["bias"] else None
            st["s0"] = normal(B, W - 1, C)
            if kind == "conv_train":
                st["dy"] = normal(M, C)
                st["ds"] = normal(B, W - 1, C, dtype=f32)
        else:
            N, G = case["n"], case["g"]
            st["x"] = normal(M, C)
            st["dt"] = normal(M, C, std=0.5)
            st["z"] = rows(C) if case["gate"] else None
            st["B"], st["C"] = normal(M, G * N), normal(M, G * N)
            # decay rates 1 .. N with a spread, steps of 0.001 to 0.1 around the bias
            st["A"] = -(torch.arange(1, N + 1, device=dev, dtype=f32)
                        * torch.exp(normal(C, N, std=0.1, dtype=f32)))
            step = torch.exp(uniform(C, lo=math.log(1e-3), hi=math.log(1e-1)))
            st["bias"] = step + torch.log(-torch.expm1(-step))
            st["D"] = normal(C, std=0.5, dtype=f32) + 1.0
            st["h0"] = normal(B, C, N, dtype=f32)
            if kind == "ssm_train":
                st["dy"] = normal(M, C)
                st["dh"] = normal(B, C, N, dtype=f32)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """What a program that calls the library keeps: dims, outputs, workspaces."""
    from selective_ssm_parameter_amd import ssm
    case = st["case"]
    B, T, kind, dt = case["batch"], case["seqlen"], case["kind"], _tdt(case)
    M, f32 = B * T, torch.float32

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if kind in ("loss", "loss_train"):
        D, V = case["d"], case["v"]
        dims = st["dims"] = ssm.loss_dims(M, D, V, case["dtype"])
        st["loss"], st["lse"] = empty(M, dtype=f32), empty(M, dtype=f32)
        st["ws"] = ssm.ssm_workspace(dims, ssm.CROSS_ENTROPY)
        if kind == "loss_train":
            st["dx"], st["dw"] = empty(M, D, dtype=f32), empty(V, D, dtype=f32)
            st["ws_b"] = ssm.ssm_workspace(dims, ssm.CROSS_ENTROPY_BACKWARD)
        return
    C = case["c"]
    if kind[:4] == "conv":
        W = case["width"]
        dims = st["dims"] = ssm.ssm_dims(B, T, C, 1, 1, case["dtype"])
        st["act"] = ssm.CONV_SILU if case["silu"] else ssm.CONV_LINEAR
        st["y"], st["s"] = empty(M, C), empty(B, W - 1, C)
        if kind == "conv_train":
            st["dx"], st["dw"] = empty(M, C), empty(C, W, dtype=f32)
            st["db"] = empty(C, dtype=f32) if case["bias"] else None
            st["ds0"] = empty(B, W - 1, C, dtype=f32)
            st["ws_b"] = ssm.ssm_workspace(dims, ssm.CAUSAL_CONV_BACKWARD)
        return
    N, G = case["n"], case["g"]
    dims = st["dims"] = ssm.ssm_dims(B, T, C, N, G, case["dtype"])
    st["y"], st["h"] = empty(M, C), empty(B, C, N, dtype=f32)
    if kind != "ssm_step":
        st["ws"] = ssm.ssm_workspace(dims, ssm.SELECTIVE_SCAN)
    if kind == "ssm_train":
        st["carry"] = ssm.selective_scan_carry(dims)
        st["dx"], st["ddt"] = empty(M, C), empty(M, C)
        st["dz"] = empty(M, C) if case["gate"] else None
        st["dB"], st["dC"] = empty(M, G * N), empty(M, G * N)
        st["dA"], st["dD"] = empty(C, N, dtype=f32), empty(C, dtype=f32)
        st["dbias"], st["dh0"] = empty(C, dtype=f32), empty(B, C, N, dtype=f32)
        st["ws_b"] = ssm.ssm_workspace(dims, ssm.SELECTIVE_SCAN_BACKWARD)


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from selective_ssm_parameter_amd import ssm
    case, kind, dims = st["case"], st["case"]["kind"], st["dims"]
    if kind in ("loss", "loss_train"):
        ssm.swimba_cross_entropy(dims, st["x"], st["w"], st["targets"], st["loss"], st["lse"],
                                 st["ws"])
        out = {"loss": st["loss"], "lse": st["lse"]}
        if kind == "loss_train":
            ssm.swimba_cross_entropy_backward(dims, st["x"], st["w"], st["targets"], st["lse"],
                                              st["dloss"], st["dx"], st["dw"], st["ws_b"])
            out.update(dx=st["dx"], dw=st["dw"])
        return out
    if kind == "conv_step":
        ssm.swimba_causal_conv_step(dims, case["width"], st["x"], st["w"], st["b"], st["act"],
                                    st["s0"], st["s"], st["y"])
        return {"y": st["y"], "s": st["s"]}
    if kind in ("conv", "conv_train"):
        ssm.swimba_causal_conv(dims, case["width"], st["x"], st["w"], st["b"], st["act"],
                               st["lens"], st["s0"], st["y"], st["s"])
        out = {"y": st["y"], "s": st["s"]}
        if kind == "conv_train":
            ssm.swimba_causal_conv_backward(dims, case["width"], st["x"], st["w"], st["b"],
                                            st["act"], st["lens"], st["s0"], st["dy"], st["ds"],
                                            st["dx"], st["dw"], st["db"], st["ds0"], st["ws_b"])
            out.update(dx=st["dx"], dw=st["dw"], ds0=st["ds0"])
            if case["bias"]:
                out["db"] = st["db"]
        return out
    if kind == "ssm_step":
        ssm.swimba_selective_step(dims, st["x"], st["dt"], st["z"], st["B"], st["C"], st["A"],
                                  st["D"], st["bias"], st["h0"], st["h"], st["y"])
        return {"y": st["y"], "h": st["h"]}
    carry = st.get("carry")
    ssm.swimba_selective_scan(dims, st["x"], st["dt"], st["z"], st["B"], st["C"], st["A"],
                              st["D"], st["bias"], st["lens"], st["h0"], st["y"], st["h"], carry,
                              st["ws"])
    out = {"y": st["y"], "h": st["h"]}
    if kind == "ssm_train":
        ssm.swimba_selective_scan_backward(dims, st["x"], st["dt"], st["z"], st["B"], st["C"],
                                           st["A"], st["D"], st["bias"], st["lens"], carry,
                                           st["dy"], st["dh"], st["dx"], st["ddt"], st["dz"],
                                           st["dB"], st["dC"], st["dA"], st["dD"], st["dbias"],
                                           st["dh0"], st["ws_b"])
        out.update({k: st[k] for k in ("dx", "ddt", "dB", "dC", "dA", "dD", "dbias", "dh0")})
        if case["gate"]:
            out["dz"] = st["dz"]
    return out


# ---- plain forms: elementary operations in 32 bits, rounded once at the end

def _silu(z):
    """silu(z) and its derivative."""
    s = 1 / (1 + torch.exp(-z))
    return z * s, s * (1 + z * (1 - s))


def _live(st, B, T, dev):
    """[B, T, 1]: the tokens in use, or None for all of them."""
    if st["lens"] is None:
        return None
    return (torch.arange(T, device=dev)[None, :] < st["lens"][:, None])[:, :, None]


def _scan_doubling(a, b):
    """All prefixes of h = a h + b along dim 1 (h before the first: zero), by doubling."""
    a, b = a.clone(), b.clone()
    n, step = a.shape[1], 1
    while step < n:
        b[:, step:] = b[:, step:] + a[:, step:] * b[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return b


def _run_plain(st):
    kind = st["case"]["kind"]
    if kind in ("loss", "loss_train"):
        return _plain_loss(st)
    if kind[:4] == "conv":
        return _plain_conv(st)
    return _plain_ssm(st)


def _plain_conv(st):
    case = st["case"]
    dt, B, T, C, W = _tdt(case), case["batch"], case["seqlen"], case["c"], case["width"]
    x = st["x"].float().reshape(B, T, C)
    w = st["w"].float()
    full = torch.cat([st["s0"].float(), x], 1)  # the inputs from token 1 - W on
    live = _live(st, B, T, x.device) if case["kind"] != "conv_step" else None
    pre = full[:, :T] * w[:, 0]
    for k in range(1, W):
        pre = pre + full[:, k:k + T] * w[:, k]
    if case["bias"]:
        pre = pre + st["b"].float()
    y, dy_dpre = _silu(pre) if case["silu"] else (pre, None)
    if live is not None:
        y = torch.where(live, y, torch.zeros((), device=x.device))
        idx = st["lens"].long()[:, None] + torch.arange(W - 1, device=x.device)
        s = torch.gather(full, 1, idx[:, :, None].expand(B, W - 1, C))
    else:
        s = full[:, T:]
    out = {"y": y.to(dt).reshape(B * T, C), "s": s.to(dt)}
    if case["kind"] != "conv_train":
        return out
    dpre = st["dy"].float().reshape(B, T, C)
    if case["silu"]:
        dpre = dpre * dy_dpre
    if live is not None:
        dpre = torch.where(live, dpre, torch.zeros((), device=x.device))
    dfull = torch.zeros_like(full)
    dw = []
    for k in range(W):
        dfull[:, k:k + T] += dpre * w[:, k]
        inp = full[:, k:k + T]
        if live is not None:
            inp = torch.where(live, inp, torch.zeros((), device=x.device))
        dw.append((dpre * inp).sum((0, 1)))
    if live is not None:
        dfull.scatter_add_(1, idx[:, :, None].expand(B, W - 1, C), st["ds"])
    else:
        dfull[:, T:] += st["ds"]
    out.update(dx=dfull[:, W - 1:].to(dt).reshape(B * T, C), dw=torch.stack(dw, 1),
               ds0=dfull[:, :W - 1].contiguous())
    if case["bias"]:
        out["db"] = dpre.sum((0, 1))
    return out


def _plain_ssm(st):
    """Blocks of channels one after the other, so that [tokens, channels, states] stays small."""
    case = st["case"]
    dt, B, T, C = _tdt(case), case["batch"], case["seqlen"], case["c"]
    N, G, kind = case["n"], case["g"], case["kind"]
    dev, per = st["x"].device, C // G
    live = _live(st, B, T, dev) if kind != "ssm_step" else None
    zero = torch.zeros((), device=dev)
    block = max(1, min(per, (1 << 28) // (B * T * N)))
    outs = {}

    def put(name, shape, dtype, where, value):
        if name not in outs:
            outs[name] = torch.zeros(shape, dtype=dtype, device=dev)
        outs[name][where] += value.to(dtype) if dtype != torch.float32 else value

    for g in range(G):
        Bm = st["B"].float().reshape(B, T, G, N)[:, :, g, None]  # [B, T, 1, N]
        Cm = st["C"].float().reshape(B, T, G, N)[:, :, g, None]
        for c0 in range(g * per, (g + 1) * per, block):
            cs = slice(c0, min(c0 + block, (g + 1) * per))
            x = st["x"][:, cs].float().reshape(B, T, -1)
            pre = st["dt"][:, cs].float().reshape(B, T, -1) + st["bias"][cs]
            delta = torch.clamp(pre, min=0) + torch.log1p(torch.exp(-torch.abs(pre)))
            if live is not None:
                x, delta = torch.where(live, x, zero), torch.where(live, delta, zero)
            A, Dv, h0 = st["A"][cs], st["D"][cs], st["h0"][:, cs]
            a = torch.exp(delta[..., None] * A)
            b = (delta * x)[..., None] * Bm
            if live is not None:
                b = torch.where(live[..., None], b, zero)
            b[:, 0] += a[:, 0] * h0
            h = _scan_doubling(a, b) if T > 1 else b
            del b
            hc = h * Cm
            if live is not None:
                hc = torch.where(live[..., None], hc, zero)
            u = hc.sum(-1) + Dv * x
            del hc
            if case["gate"]:
                z = st["z"][:, cs].float().reshape(B, T, -1)
                sz, dsz = _silu(z)
                y = u * sz
            else:
                y = u
            if live is not None:
                y = torch.where(live, y, zero)
            put("y", (B * T, C), dt, (slice(None), cs), y.reshape(B * T, -1))
            put("h", (B, C, N), torch.float32, (slice(None), cs), h[:, -1])
            if kind != "ssm_train":
                continue
            dy = st["dy"][:, cs].float().reshape(B, T, -1)
            if live is not None:
                dy = torch.where(live, dy, zero)
            if case["gate"]:
                dz = dy * u * dsz
                if live is not None:
                    dz = torch.where(live, dz, zero)
                put("dz", (B * T, C), dt, (slice(None), cs), dz.reshape(B * T, -1))
                dy = dy * sz
                if live is not None:
                    dy = torch.where(live, dy, zero)
            e = dy[..., None] * Cm
            if live is not None:
                e = torch.where(live[..., None], e, zero)
            e[:, -1] += st["dh"][:, cs]
            an = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
            e = _scan_doubling(an.flip(1), e.flip(1)).flip(1) if T > 1 else e
            del an
            put("dh0", (B, C, N), torch.float32, (slice(None), cs), a[:, 0] * e[:, 0])
            dCm = (dy[..., None] * h).sum(2)
            dBm = (e * (delta * x)[..., None]).sum(2)
            if live is not None:
                dCm, dBm = torch.where(live, dCm, zero), torch.where(live, dBm, zero)
            gn = (slice(None), slice(None), g)
            put("dC32", (B, T, G, N), torch.float32, gn, dCm)
            put("dB32", (B, T, G, N), torch.float32, gn, dBm)
            ah = a * torch.cat([h0[:, None], h[:, :-1]], 1)
            del h, a
            eB = e * Bm
            if live is not None:
                eB = torch.where(live[..., None], eB, zero)
            eB = eB.sum(-1)
            eah = e * ah
            del e, ah
            put("dA", (C, N), torch.float32, cs, (eah * delta[..., None]).sum((0, 1)))
            ddt = ((eah * A).sum(-1) + eB * x) * (1 / (1 + torch.exp(-pre)))
            if live is not None:
                ddt = torch.where(live, ddt, zero)
            del eah
            put("dx", (B * T, C), dt, (slice(None), cs),
                (delta * eB + Dv * dy).reshape(B * T, -1))
            put("ddt", (B * T, C), dt, (slice(None), cs), ddt.reshape(B * T, -1))
            put("dbias", (C,), torch.float32, cs, ddt.sum((0, 1)))
            put("dD", (C,), torch.float32, cs, (dy * x).sum((0, 1)))
    for name in ("dB", "dC"):
        if name + "32" in outs:
            outs[name] = outs.pop(name + "32").to(dt).reshape(B * T, G * N)
    return outs


def _plain_loss(st):
    """Blocks of tokens one after the other, so that a block's logits stay below 4 GiB."""
    case = st["case"]
    M, V = case["batch"] * case["seqlen"], case["v"]
    x, w, tgt = st["x"].float(), st["w"].float(), st["targets"].long()
    train = case["kind"] == "loss_train"
    loss, lse, dx, dw = [], [], [], None
    block = max(1, (1 << 30) // V)
    for m0 in range(0, M, block):
        ms = slice(m0, m0 + block)
        z = x[ms] @ w.t()
        top = z.max(1, keepdim=True).values
        l = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
        t = tgt[ms]
        counts = (t >= 0) & (t < V)
        at = t.clamp(0, V - 1)[:, None]
        loss.append(torch.where(counts, l - z.gather(1, at)[:, 0], torch.zeros_like(l)))
        lse.append(l)
        if train:
            g = torch.where(counts, st["dloss"][ms], torch.zeros_like(l))[:, None]
            dz = torch.exp(z - l[:, None])
            dz.scatter_add_(1, at, -torch.ones_like(l)[:, None])
            dz *= g
            dx.append(dz @ w)
            dw = dz.t() @ x[ms] if dw is None else dw + dz.t() @ x[ms]
    out = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    if train:
        out.update(dx=torch.cat(dx), dw=dw)
    return out


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
    if kind in ("loss", "loss_train"):
        return _exact_loss(st)
    if kind[:4] == "conv":
        return _exact_conv(st)
    return _exact_ssm(st)


def _lens(st, B, T):
    return [T] * B if st["lens"] is None else st["lens"].tolist()


def _exact_conv(st):
    """Sequence by sequence, each cut to its length; the gradient through the transposed sum."""
    case, f64 = st["case"], torch.float64
    B, T, C, W = case["batch"], case["seqlen"], case["c"], case["width"]
    dev, train = st["x"].device, case["kind"] == "conv_train"
    w = st["w"].to(f64)
    out = {"y": torch.zeros(B, T, C, dtype=f64, device=dev),
           "s": torch.zeros(B, W - 1, C, dtype=f64, device=dev)}
    if train:
        out.update(dx=torch.zeros(B, T, C, dtype=f64, device=dev),
                   dw=torch.zeros(C, W, dtype=f64, device=dev),
                   ds0=torch.zeros(B, W - 1, C, dtype=f64, device=dev))
        if case["bias"]:
            out["db"] = torch.zeros(C, dtype=f64, device=dev)
    for b, n in enumerate(_lens(st, B, T)):
        inp = torch.cat([st["s0"][b].to(f64), st["x"].reshape(B, T, C)[b, :n].to(f64)], 0)
        out["s"][b] = inp[n:n + W - 1]
        win = inp.unfold(0, W, 1)  # [n, C, W]
        pre = torch.einsum("ncw,cw->nc", win, w)
        if case["bias"]:
            pre = pre + st["b"].to(f64)
        sg = torch.sigmoid(pre)
        out["y"][b, :n] = pre * sg if case["silu"] else pre
        if not train:
            continue
        d = st["dy"].reshape(B, T, C)[b, :n].to(f64)
        if case["silu"]:
            d = d * (sg + pre * sg * (1 - sg))
        out["dw"] += torch.einsum("nc,ncw->cw", d, win)
        if case["bias"]:
            out["db"] += d.sum(0)
        di = torch.zeros_like(inp)
        for j in range(n + W - 1):  # input j meets weight k in output j - k
            if j >= 64 and j < n:
                continue
            for k in range(W):
                if 0 <= j - k < n:
                    di[j] += d[j - k] * w[:, k]
        if n > 64:  # the inputs that all weights meet, at once
            di[64:n] = sum(d[64 - k:n - k] * w[:, k] for k in range(W))
        di[n:] += st["ds"][b].to(f64)
        out["ds0"][b] = di[:W - 1]
        out["dx"][b, :n] = di[W - 1:]
        # the gradient of the state behind the last token reaches the first state where n < W - 1
    out["y"] = out["y"].reshape(B * T, C)
    if train:
        out["dx"] = out["dx"].reshape(B * T, C)
    return out


def _exact_ssm(st):
    case, f64 = st["case"], torch.float64
    B, T, C, N, G = (case[k] for k in ("batch", "seqlen", "c", "n", "g"))
    dev, train, gate = st["x"].device, case["kind"] == "ssm_train", case["gate"]
    lens = torch.tensor(_lens(st, B, T), device=dev)
    use = torch.arange(T, device=dev)[None, :] < lens[:, None]  # [B, T]
    x = st["x"].to(f64).reshape(B, T, C)
    delta = torch.nn.functional.softplus(st["dt"].to(f64).reshape(B, T, C) + st["bias"].to(f64),
                                         threshold=60.0)
    sig = torch.sigmoid(st["dt"].to(f64).reshape(B, T, C) + st["bias"].to(f64)) if train else None
    grp = torch.arange(C, device=dev) // (C // G)
    Bm = st["B"].to(f64).reshape(B, T, G, N)
    Cm = st["C"].to(f64).reshape(B, T, G, N)
    A, Dv = st["A"].to(f64), st["D"].to(f64)
    h = st["h0"].to(f64)
    u = torch.zeros(B, T, C, dtype=f64, device=dev)
    hs = torch.empty(T + 1, B, C, N, dtype=f64, device=dev) if train else None
    if train:
        hs[0] = h
    ragged = st["lens"] is not None
    for t in range(T):
        nh = torch.exp(delta[:, t, :, None] * A) * h \
            + (delta[:, t] * x[:, t])[..., None] * Bm[:, t][:, grp]
        h = torch.where(use[:, t, None, None], nh, h) if ragged else nh
        if train:
            hs[t + 1] = h
        u[:, t] = (h * Cm[:, t][:, grp]).sum(-1) + Dv * x[:, t]
    z = st["z"].to(f64).reshape(B, T, C) if gate else None
    sz = torch.sigmoid(z) if gate else None
    mask = use[..., None]
    y = u * z * sz if gate else u
    out = {"y": torch.where(mask, y, 0.0).reshape(B * T, C), "h": h}
    if not train:
        return out
    dy = st["dy"].to(f64).reshape(B, T, C)
    if gate:
        out["dz"] = torch.where(mask, dy * u * (sz + z * sz * (1 - sz)), 0.0).reshape(B * T, C)
        dy = dy * z * sz
    dy = torch.where(mask, dy, 0.0)
    e = st["dh"].to(f64)  # the gradient of the state behind token t
    dx, dd = torch.zeros_like(x), torch.zeros_like(x)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    dA = torch.zeros_like(A)
    for t in range(T - 1, -1, -1):
        on = use[:, t, None, None]
        et = torch.where(on, e + dy[:, t, :, None] * Cm[:, t][:, grp], 0.0)
        a = torch.exp(delta[:, t, :, None] * A)
        flow = et * a * hs[t]
        eb = (et * Bm[:, t][:, grp]).sum(-1)
        dx[:, t] = delta[:, t] * eb + Dv * dy[:, t]
        dd[:, t] = (flow * A).sum(-1) + x[:, t] * eb
        dA += (flow * delta[:, t, :, None]).sum(0)
        dB[:, t] = (et * (delta[:, t] * x[:, t])[..., None]).reshape(B, G, C // G, N).sum(2)
        dC[:, t] = (dy[:, t, :, None] * hs[t + 1]).reshape(B, G, C // G, N).sum(2)
        e = torch.where(on, a * et, e)
    ddt = dd * sig
    out.update(dx=torch.where(mask, dx, 0.0).reshape(B * T, C),
               ddt=torch.where(mask, ddt, 0.0).reshape(B * T, C),
               dB=dB.reshape(B * T, G * N), dC=dC.reshape(B * T, G * N), dA=dA,
               dD=(dy * x).sum((0, 1)), dbias=torch.where(mask, ddt, 0.0).sum((0, 1)), dh0=e)
    return out


def _exact_loss(st):
    case, f64 = st["case"], torch.float64
    M, V = case["batch"] * case["seqlen"], case["v"]
    x, w, tgt = st["x"].to(f64), st["w"].to(f64), st["targets"].long()
    counts = (tgt >= 0) & (tgt < V)
    loss = torch.zeros(M, dtype=f64, device=x.device)
    lse = torch.zeros_like(loss)
    train = case["kind"] == "loss_train"
    dx = torch.zeros_like(x) if train else None
    dw = torch.zeros_like(w) if train else None
    for m0 in range(0, M, 1024):
        ms = slice(m0, min(m0 + 1024, M))
        z = torch.matmul(x[ms], w.t())
        lse[ms] = torch.logsumexp(z, 1)
        own_z = (x[ms] * w[tgt[ms].clamp(0, V - 1)]).sum(1)
        loss[ms] = torch.where(counts[ms], lse[ms] - own_z, 0.0)
        if train:
            p = torch.softmax(z, 1)
            hot = torch.arange(V, device=x.device)[None, :] == tgt[ms][:, None]
            dz = (p - hot.to(f64)) * torch.where(counts[ms], st["dloss"][ms].to(f64), 0.0)[:, None]
            dx[ms] = torch.matmul(dz, w)
            dw += torch.matmul(dz.t(), x[ms])
    out = {"loss": loss, "lse": lse}
    if train:
        out.update(dx=dx, dw=dw)
    return out


# ------------------------------------------------------------------ work

def work(case):
    """(An exponential, a division or a logarithm counts as one operation.)"""
    kind = case["kind"]
    es = 2 if case["dtype"] == BF16 else 4
    B, T = case["batch"], case["seqlen"]
    M = B * T
    if kind in ("loss", "loss_train"):
        D, V = case["d"], case["v"]
        nb = es * (M * D + V * D) + 12 * M
        if kind == "loss":
            return {"bytes": nb, "flops": 2 * M * D * V + 4 * M * V}
        return {"bytes": nb + 4 * (M * D + V * D) + 4 * M, "flops": 6 * M * D * V + 7 * M * V}
    C = case["c"]
    n = M * C
    if kind[:4] == "conv":
        W = case["width"]
        state = B * (W - 1) * C
        nb = 2 * n * es + 2 * state * es + C * W * es
        if kind != "conv_train":
            return {"bytes": nb, "flops": (2 * W + 4) * n}
        # the backward reads x and dy and writes dx
        return {"bytes": nb + 3 * n * es + state * (es + 8) + 4 * C * W,
                "flops": (6 * W + 16) * n}
    N, G, gate = case["n"], case["g"], case["gate"]
    k = 3 if gate else 2
    small = 2 * M * G * N * es
    nb = n * es * (k + 1) + small + 8 * B * C * N + 4 * C * N
    if kind != "ssm_train":
        return {"bytes": nb, "flops": n * (7 * N + 12)}
    # the backward reads x, dt, z and dy and writes their gradients
    return {"bytes": nb + n * es * (2 * k + 1) + 2 * small + 8 * B * C * N + 8 * C * N,
            "flops": n * (27 * N + 40)}
