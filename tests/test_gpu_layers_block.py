"""The layer calls as a program uses them: a whole block forward and backward
with the mixer's output projection between them, captured into graphs,
repeated, on other streams, and on tensors past 32-bit offsets."""
from __future__ import annotations

import pytest
import torch

from selective_ssm_parameter_amd import binding as sb
from selective_ssm_parameter_amd import layers as sl

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def randn(gen, *shape, dt=torch.float32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen) * std + mean).to("cuda", dt)


class Block:
    """x -> x + W_o scan([x|f|o] = W_r norm(x)); then + W_d gated(W_in norm(.)).
    Everything a program would keep: parameters, activations, workspaces."""

    def __init__(self, B, T, D, C, F, dtype, seed=0):
        self.B, self.T, self.D, self.C, self.F, self.dtype = B, T, D, C, F, dtype
        dt = self.dt = DT[dtype]
        M = self.M = B * T
        gen = torch.Generator().manual_seed(seed)
        p = self.p = {
            "n1w": randn(gen, D, dt=dt, std=0.2, mean=1), "n1b": randn(gen, D, dt=dt, std=0.2),
            "wr": randn(gen, 3 * C, D, dt=dt, std=D ** -0.5),
            "wo": randn(gen, D, C, dt=dt, std=C ** -0.5),
            "n2w": randn(gen, D, dt=dt, std=0.2, mean=1), "n2b": randn(gen, D, dt=dt, std=0.2),
            "win": randn(gen, 2 * F, D, dt=dt, std=D ** -0.5),
            "wd": randn(gen, D, F, dt=dt, std=F ** -0.5)}
        self.x = randn(gen, M, D, dt=dt)
        self.h0 = randn(gen, B, C)
        self.lens = torch.tensor([T - 3 * i for i in range(B)], dtype=torch.int32, device="cuda")
        self.dout = randn(gen, M, D)
        self.dh = randn(gen, B, C)
        e = lambda *s, d=dt: torch.empty(*s, dtype=d, device="cuda")
        f32 = torch.float32
        self.d_norm = sl.layer_dims(B, T, D, 8, dtype)
        self.d_rec = sl.layer_dims(B, T, 3 * C, D, dtype)   # output_project: [M, D] -> [M, 3C]
        self.d_scan = sl.layer_dims(B, T, 8, C, dtype)
        self.d_o = sl.layer_dims(B, T, D, C, dtype)
        self.d_ff = sl.layer_dims(B, T, D, F, dtype)
        self.a = {"n1": e(M, D), "xfo": e(M, 3 * C), "y": e(M, C), "hT": e(B, C, d=f32),
                  "mix": e(M, D), "s": e(M, D), "n2": e(M, D), "h": e(M, F), "ff": e(M, D),
                  "mean1": e(M, d=f32), "rstd1": e(M, d=f32), "mean2": e(M, d=f32),
                  "rstd2": e(M, d=f32), "carry": sl.gated_scan_carry(self.d_scan)}
        self.g = {"dff": e(M, D), "dh": e(M, F), "dwd": e(D, F, d=f32), "dn2": e(M, D, d=f32),
                  "dwin": e(2 * F, D, d=f32), "ds": e(M, D, d=f32), "dn2w": e(D, d=f32),
                  "dn2b": e(D, d=f32), "dmix": e(M, D), "dy": e(M, C), "dwo": e(D, C, d=f32),
                  "dxfo": e(M, 3 * C), "dh0": e(B, C, d=f32), "dn1": e(M, D),
                  "dwr": e(3 * C, D, d=f32), "dx": e(M, D, d=f32), "dn1w": e(D, d=f32),
                  "dn1b": e(D, d=f32)}
        w = sl.layer_workspace
        self.ws = {"norm": w(self.d_norm, sl.LAYER_NORM_BACKWARD),
                   "scan": w(self.d_scan, sl.LAYER_GATED_SCAN),
                   "scan_b": w(self.d_scan, sl.LAYER_GATED_SCAN_BACKWARD),
                   "ff": w(self.d_ff, sl.LAYER_GATED_PROJECT_BACKWARD),
                   "down": w(self.d_ff, sl.LAYER_OUTPUT_PROJECT_BACKWARD),
                   "o": w(self.d_o, sl.LAYER_OUTPUT_PROJECT_BACKWARD),
                   "rec": w(self.d_rec, sl.LAYER_OUTPUT_PROJECT_BACKWARD)}

    def xfo(self, t):
        return [t[:, i * self.C:(i + 1) * self.C] for i in range(3)]

    def forward(self, stream=None):
        p, a = self.p, self.a
        kw = {"stream": stream}
        sl.swimba_layer_norm(self.d_norm, self.x, None, p["n1w"], p["n1b"], EPS, None, a["n1"],
                             a["mean1"], a["rstd1"], **kw)
        sb.swimba_output_project(self.d_rec, a["n1"], p["wr"], a["xfo"], **kw)
        sl.swimba_gated_scan(self.d_scan, *self.xfo(a["xfo"]), self.lens, self.h0, a["y"],
                             a["hT"], a["carry"], self.ws["scan"], **kw)
        sb.swimba_output_project(self.d_o, a["y"], p["wo"], a["mix"], **kw)
        sl.swimba_layer_norm(self.d_norm, a["mix"], self.x, p["n2w"], p["n2b"], EPS, a["s"],
                             a["n2"], a["mean2"], a["rstd2"], **kw)
        sl.swimba_gated_project(self.d_ff, a["n2"], p["win"], sl.ACT_SILU, None, a["h"], **kw)
        sb.swimba_output_project(self.d_ff, a["h"], p["wd"], a["ff"], **kw)

    def backward(self, stream=None):
        """From dout = dl/d(s + ff) and dh = dl/d(final state)."""
        p, a, g = self.p, self.a, self.g
        kw = {"stream": stream}
        g["dff"].copy_(self.dout)
        sl.swimba_output_project_backward(self.d_ff, a["h"], p["wd"], g["dff"], g["dh"], g["dwd"],
                                          self.ws["down"], **kw)
        sl.swimba_gated_project_backward(self.d_ff, a["n2"], p["win"], g["dh"], sl.ACT_SILU,
                                         g["dn2"], g["dwin"], self.ws["ff"], **kw)
        sl.swimba_layer_norm_backward(self.d_norm, a["s"], p["n2w"], a["mean2"], a["rstd2"],
                                      g["dn2"], self.dout, g["ds"], g["dn2w"], g["dn2b"],
                                      self.ws["norm"], **kw)
        g["dmix"].copy_(g["ds"])
        sl.swimba_output_project_backward(self.d_o, a["y"], p["wo"], g["dmix"], g["dy"], g["dwo"],
                                          self.ws["o"], **kw)
        sl.swimba_gated_scan_backward(self.d_scan, *self.xfo(a["xfo"]), self.lens, a["carry"],
                                      g["dy"], self.dh, *self.xfo(g["dxfo"]), g["dh0"],
                                      self.ws["scan_b"], **kw)
        sl.swimba_output_project_backward(self.d_rec, a["n1"], p["wr"], g["dxfo"], g["dn1"],
                                          g["dwr"], self.ws["rec"], **kw)
        sl.swimba_layer_norm_backward(self.d_norm, self.x, p["n1w"], a["mean1"], a["rstd1"],
                                      g["dn1"], g["ds"], g["dx"], g["dn1w"], g["dn1b"],
                                      self.ws["norm"], **kw)

    def outputs(self):
        return [self.a[k] for k in ("s", "ff", "hT")] + [
            self.g[k] for k in ("dx", "dwr", "dwo", "dwin", "dwd", "dn1w", "dn1b", "dn2w", "dn2b",
                                "dh0")]

    NAMES = ["s", "ff", "hT", "dx", "dwr", "dwo", "dwin", "dwd", "dn1w", "dn1b", "dn2w", "dn2b",
             "dh0"]

    def reference(self):
        """The same block in float64 on the CPU, gradients by autograd."""
        leaf = lambda t: t.double().cpu().requires_grad_()
        p = {k: leaf(v) for k, v in self.p.items()}
        x, h0 = leaf(self.x), leaf(self.h0)
        B, T, C, F = self.B, self.T, self.C, self.F

        def norm(s, w, b):
            c = s - s.mean(1, keepdim=True)
            return c / torch.sqrt((c * c).mean(1, keepdim=True) + EPS) * w + b

        xfo = norm(x, p["n1w"], p["n1b"]) @ p["wr"].t()
        v, f, o = (xfo[:, i * C:(i + 1) * C].reshape(B, T, C) for i in range(3))
        f = torch.sigmoid(f)
        rows, finals = [], []
        for b in range(B):
            h = h0[b]
            for t in range(T):
                if t < int(self.lens[b]):
                    h = f[b, t] * h + (1 - f[b, t]) * v[b, t]
                    rows.append(h * o[b, t] * torch.sigmoid(o[b, t]))
                else:
                    rows.append(torch.zeros_like(h))
            finals.append(h)
        y, hT = torch.stack(rows), torch.stack(finals)
        s = x + y @ p["wo"].t()
        z = norm(s, p["n2w"], p["n2b"]) @ p["win"].t()
        hid = z[:, :F] * torch.sigmoid(z[:, :F]) * z[:, F:]
        ff = hid @ p["wd"].t()
        loss = ((s + ff) * self.dout.double().cpu()).sum() + (hT * self.dh.double().cpu()).sum()
        loss.backward()
        return [s, ff, hT, x.grad] + [p[k].grad for k in ("wr", "wo", "win", "wd", "n1w", "n1b",
                                                          "n2w", "n2b")] + [h0.grad]


# A result of the chain is behind at most 10 roundings to dtype (n1, xfo, y, mix,
# s, n2, h, and going back dff, dh, dmix, dy, dxfo, dn1: the longest path to a
# gradient crosses all 13), each at most eps / 2 of a value and amplified by a
# factor of about 1 in the norm (unit-variance rows, 1 / sqrt(fan-in) weights; the
# norms and gates have slopes up to about 2): in the 2-norm they add at random,
# sqrt(13) * 2 * eps / 2. The float32 sums add K U with K <= 500 per product.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_against_autograd(dtype):
    blk = Block(3, 150, 96, 64, 136, dtype)
    blk.forward()
    blk.backward()
    eps = torch.finfo(DT[dtype]).eps
    bound = 13 ** 0.5 * 2 * eps / 2 + 8 * 500 * 2.0 ** -24
    for name, got, want in zip(Block.NAMES, blk.outputs(), blk.reference()):
        got, want = got.double().cpu(), want.detach()
        err = ((got - want).norm() / want.norm()).item()
        assert err <= bound, f"{name}: {err} against {bound}"


def test_block_repeats_bitwise_and_on_another_stream():
    blk = Block(2, 700, 256, 192, 320, "bf16", seed=1)
    blk.forward()
    blk.backward()
    torch.cuda.synchronize()
    ref = [t.clone() for t in blk.outputs()]
    side = torch.cuda.Stream()
    for rep in range(3):
        for t in blk.outputs():
            t.zero_()
        for w in blk.ws.values():
            w.fill_(rep)  # whatever a workspace holds
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            blk.forward(stream=side if rep == 1 else None)
            blk.backward(stream=side if rep == 1 else None)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for name, a, b in zip(Block.NAMES, blk.outputs(), ref):
            assert torch.equal(a, b), f"repeat {rep}: {name}"


def test_block_replays_from_graphs_that_share_workspaces():
    """Two graphs of the same block (one the forward, one both passes) with the
    same workspaces, replayed in turn with eager work between."""
    blk = Block(2, 600, 128, 128, 192, "bf16", seed=2)
    blk.forward()
    blk.backward()
    torch.cuda.synchronize()
    ref = [t.clone() for t in blk.outputs()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        blk.forward()
        blk.backward()
        torch.cuda.synchronize()
        with torch.cuda.graph(g1, stream=s):
            blk.forward()
        with torch.cuda.graph(g2, stream=s):
            blk.forward()
            blk.backward()
    torch.cuda.synchronize()
    for rep in range(4):
        for t in blk.outputs():
            t.zero_()
        torch.cuda.synchronize()
        g1.replay()
        torch.cuda.synchronize()
        for name, a, b in list(zip(Block.NAMES, blk.outputs(), ref))[:3]:
            assert torch.equal(a, b), f"replay {rep}: {name} of the forward"
        blk.backward()  # eager, on the replayed forward
        torch.cuda.synchronize()
        for name, a, b in zip(Block.NAMES, blk.outputs(), ref):
            assert torch.equal(a, b), f"replay {rep}: {name} eager"
            a.zero_()
        g2.replay()
        torch.cuda.synchronize()
        for name, a, b in zip(Block.NAMES, blk.outputs(), ref):
            assert torch.equal(a, b), f"replay {rep}: {name}"


@pytest.mark.parametrize("Bt,T,C", [(1, 40000, 320), (7, 3000, 1000), (300, 200, 72)])
def test_gated_scan_repeats_bitwise(Bt, T, C):
    """Many chunks in flight: the order of the sums does not depend on which
    workgroup is first."""
    gen = torch.Generator().manual_seed(3)
    d = sl.layer_dims(Bt, T, 8, C, "bf16")
    dt = torch.bfloat16
    x, f, o, dy = (randn(gen, Bt * T, C, dt=dt) for _ in range(4))
    f += 3
    ws = sl.layer_workspace(d, sl.LAYER_GATED_SCAN)
    carry = sl.gated_scan_carry(d)
    outs = []
    for _ in range(3):
        y, dx, df, do = (torch.empty_like(x) for _ in range(4))
        h, dh0 = torch.empty(Bt, C, device="cuda"), torch.empty(Bt, C, device="cuda")
        sl.swimba_gated_scan(d, x, f, o, None, None, y, h, carry, ws)
        sl.swimba_gated_scan_backward(d, x, f, o, None, carry, dy, None, dx, df, do, dh0, ws)
        outs.append([y, h, dx, df, do, dh0, carry.clone()])
    torch.cuda.synchronize()
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)


def test_gated_scan_past_32_bit_offsets():
    """2.4e9 elements per tensor. A sequence cut at a multiple of 2048 tokens
    and resumed from its state takes the same steps, so its outputs are equal
    bit for bit."""
    T, C, cut = 600_000, 4096, 2048 * 280
    dt = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty(T, C, dtype=dt, device="cuda").normal_(generator=gen)
    f = torch.empty(T, C, dtype=dt, device="cuda").normal_(3.0, 1.0, generator=gen)
    y, h = torch.empty_like(x), torch.empty(1, C, device="cuda")
    d = sl.layer_dims(1, T, 8, C, "bf16")
    carry = sl.gated_scan_carry(d)
    sl.swimba_gated_scan(d, x, f, None, None, None, y, h, carry,
                         sl.layer_workspace(d, sl.LAYER_GATED_SCAN))
    d1, d2 = sl.layer_dims(1, cut, 8, C, "bf16"), sl.layer_dims(1, T - cut, 8, C, "bf16")
    y2, h1, h2 = torch.empty(T - cut, C, dtype=dt, device="cuda"), torch.empty_like(h), \
        torch.empty_like(h)
    y1 = torch.empty(cut, C, dtype=dt, device="cuda")
    sl.swimba_gated_scan(d1, x[:cut], f[:cut], None, None, None, y1, h1, None,
                         sl.layer_workspace(d1, sl.LAYER_GATED_SCAN))
    sl.swimba_gated_scan(d2, x[cut:], f[cut:], None, None, h1, y2, h2, None,
                         sl.layer_workspace(d2, sl.LAYER_GATED_SCAN))
    torch.cuda.synchronize()
    assert torch.equal(y[cut:], y2) and torch.equal(y[:cut], y1) and torch.equal(h, h2)
    del y1, y2
    # the backward's last chunks against a call on the last tokens alone
    tail = 2048 * 8 + (T - cut) % 2048
    dy, dx, df = y, torch.empty_like(x), torch.empty_like(x)
    dh0 = torch.empty(1, C, device="cuda")
    sl.swimba_gated_scan_backward(d, x, f, None, None, carry, dy, None, dx, df, None, dh0,
                                  sl.layer_workspace(d, sl.LAYER_GATED_SCAN_BACKWARD))
    t0 = (T - tail) // 128 * 128
    d3 = sl.layer_dims(1, T - t0, 8, C, "bf16")
    dx3, df3 = (torch.empty(T - t0, C, dtype=dt, device="cuda") for _ in range(2))
    sl.swimba_gated_scan_backward(d3, x[t0:], f[t0:], None, None,
                                  carry.view(-1, C)[t0 // 128:].contiguous(), dy[t0:], None, dx3,
                                  df3, None, dh0.clone(),
                                  sl.layer_workspace(d3, sl.LAYER_GATED_SCAN_BACKWARD))
    torch.cuda.synchronize()
    assert torch.equal(dx[t0:], dx3) and torch.equal(df[t0:], df3)


def test_layer_norm_past_32_bit_offsets():
    M, D = 1_200_000, 2048
    dt = torch.bfloat16
    x = torch.empty(M, D, dtype=dt, device="cuda").normal_()
    w = torch.ones(D, dtype=dt, device="cuda")
    y = torch.empty_like(x)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    d = sl.layer_dims(1, M, D, 8, "bf16")
    sl.swimba_layer_norm(d, x, None, w, None, EPS, None, y, mean, rstd)
    n = 5000
    dn = sl.layer_dims(1, n, D, 8, "bf16")
    yn, mn, rn = torch.empty(n, D, dtype=dt, device="cuda"), torch.empty(n, device="cuda"), \
        torch.empty(n, device="cuda")
    sl.swimba_layer_norm(dn, x[-n:], None, w, None, EPS, None, yn, mn, rn)
    dx, dw = torch.empty(M, D, device="cuda"), torch.empty(D, device="cuda")
    sl.swimba_layer_norm_backward(d, x, w, mean, rstd, y, None, dx, dw, None,
                                  sl.layer_workspace(d, sl.LAYER_NORM_BACKWARD))
    dxn, dwn = torch.empty(n, D, device="cuda"), torch.empty(D, device="cuda")
    sl.swimba_layer_norm_backward(dn, x[-n:], w, mn, rn, yn, None, dxn, dwn, None,
                                  sl.layer_workspace(dn, sl.LAYER_NORM_BACKWARD))
    torch.cuda.synchronize()
    assert torch.equal(y[-n:], yn) and torch.equal(mean[-n:], mn) and torch.equal(dx[-n:], dxn)
    # sum of y xh with y = xh rounded: about M per column
    assert torch.isfinite(dw).all() and (dw / M - 1).abs().max() < 0.02


def test_projections_past_32_bit_offsets():
    """x of 2.6 GB: rows against the same rows alone, and dw against the sum
    of two halves."""
    M, D, F = 640_000, 2048, 64
    dt = torch.bfloat16
    x = torch.empty(M, D, dtype=dt, device="cuda").normal_()
    w = torch.empty(2 * F, D, dtype=dt, device="cuda").normal_(0.0, D ** -0.5)
    h, dh = torch.empty(M, F, dtype=dt, device="cuda"), \
        torch.empty(M, F, dtype=dt, device="cuda").normal_()
    dx, dw = torch.empty(M, D, device="cuda"), torch.empty(2 * F, D, device="cuda")

    def run(x, h, dh, dx, dw):
        d = sl.layer_dims(1, x.shape[0], D, F, "bf16")
        sl.swimba_gated_project(d, x, w, sl.ACT_SILU, None, h)
        sl.swimba_gated_project_backward(d, x, w, dh, sl.ACT_SILU, dx, dw,
                                         sl.layer_workspace(d, sl.LAYER_GATED_PROJECT_BACKWARD))

    run(x, h, dh, dx, dw)
    halves = []
    for sl_ in (slice(0, M // 2), slice(M // 2, M)):
        n = M // 2
        hn, dxn = torch.empty(n, F, dtype=dt, device="cuda"), torch.empty(n, D, device="cuda")
        dwn = torch.empty(2 * F, D, device="cuda")
        run(x[sl_], hn, dh[sl_], dxn, dwn)
        torch.cuda.synchronize()
        assert torch.equal(hn, h[sl_]) and torch.equal(dxn, dx[sl_])
        halves.append(dwn.double())
        del hn, dxn
    want = halves[0] + halves[1]
    # fp32 sums of 640000 terms in random order: sqrt(M) U of the terms' norm
    bound = 8 * M ** 0.5 * 2.0 ** -24
    assert ((dw.double() - want).norm() / want.norm()).item() <= bound
