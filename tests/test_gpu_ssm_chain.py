"""A whole layer as a program runs it - input projection, causal convolution,
projection to dt, B and C, selective scan, output projection, cross entropy, and
back - against float64 autograd; the same from graphs, on another stream, with new
inputs each time and in buffers that were filled with NaN."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from layer_kernels import accumulation
from selective_ssm_parameter_amd import binding as sb
from selective_ssm_parameter_amd import layers as sl
from selective_ssm_parameter_amd import ssm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32 = torch.float32


def bits(name, a, b):
    """Equal as bits (NaN included)."""
    ints = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    assert torch.equal(a.contiguous().view(ints), b.contiguous().view(ints)), name


class Layer:
    """Weights, inputs and every tensor between the calls of one training step."""

    WEIGHTS = ("w_in", "w_conv", "b_conv", "w_x", "A", "D", "bias", "w_out", "w_voc")
    INPUTS = ("h", "targets", "lens", "s0", "h0", "dloss")

    def __init__(self, dtype, B=3, T=150, D=64, C=96, N=16, V=333, W=4, seed=0):
        self.dtype, self.dt = dtype, torch.bfloat16 if dtype == "bf16" else F32
        self.B, self.T, self.D, self.C, self.N, self.V, self.W, self.M = B, T, D, C, N, V, W, B * T
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s, std=1.0, dt=None: (torch.randn(*s, generator=gen) * std).to(
            "cuda", self.dt if dt is None else dt)
        X = self.X = C + 2 * N
        self.w_in, self.w_conv, self.b_conv = r(2 * C, D, std=D ** -0.5), r(C, W, std=0.5), r(C)
        self.w_x, self.w_out = r(X, C, std=C ** -0.5), r(D, C, std=C ** -0.5)
        self.A, self.Dv, self.bias = -torch.exp(r(C, N, dt=F32)), r(C, dt=F32), r(C, dt=F32) - 2
        self.w_voc = r(V, D, std=D ** -0.5)
        d = lambda k, o: sl.layer_dims(1, self.M, o, k, dtype)  # (a product k -> o)
        self.d_in, self.d_x, self.d_out = d(D, 2 * C), d(C, X), d(C, D)
        self.d_conv = ssm.ssm_dims(B, T, C, 1, 1, dtype)
        self.d_scan, self.d_loss = ssm.ssm_dims(B, T, C, N, 1, dtype), \
            ssm.loss_dims(self.M, D, V, dtype)
        ws = ssm.ssm_workspace
        self.ws = {"conv": ws(self.d_conv, ssm.CAUSAL_CONV_BACKWARD),
                   "scan": ws(self.d_scan, ssm.SELECTIVE_SCAN),
                   "scan_b": ws(self.d_scan, ssm.SELECTIVE_SCAN_BACKWARD),
                   "loss": ws(self.d_loss, ssm.CROSS_ENTROPY),
                   "loss_b": ws(self.d_loss, ssm.CROSS_ENTROPY_BACKWARD)}
        for k, dd in (("in", self.d_in), ("x", self.d_x), ("out", self.d_out)):
            self.ws[k] = sl.layer_workspace(dd, sl.LAYER_OUTPUT_PROJECT_BACKWARD)
        e = lambda *s, dt=None: torch.empty(*s, dtype=self.dt if dt is None else dt, device="cuda")
        M = self.M
        self.t = dict(
            xz=e(M, 2 * C), xc=e(M, C), s1=e(B, W - 1, C), xdb=e(M, X), y=e(M, C),
            h1=e(B, C, N, dt=F32), o=e(M, D), loss=e(M, dt=F32), lse=e(M, dt=F32),
            carry=ssm.selective_scan_carry(self.d_scan), do=e(M, D, dt=F32), dot=e(M, D),
            dw_voc=e(V, D, dt=F32), dy=e(M, C), dw_out=e(D, C, dt=F32), dxs=e(M, C), dxdb=e(M, X),
            dA=e(C, N, dt=F32), dD=e(C, dt=F32), dbias=e(C, dt=F32), dh0=e(B, C, N, dt=F32),
            dxp=e(M, C), dw_x=e(X, C, dt=F32), dxc=e(M, C), dxz=e(M, 2 * C),
            dw_conv=e(C, W, dt=F32), db_conv=e(C, dt=F32), ds0=e(B, W - 1, C, dt=F32),
            dh=e(M, D), dw_in=e(2 * C, D, dt=F32))
        self.i = {k: torch.empty_like(v) for k, v in self.inputs(0).items()}
        self.load(0)

    def inputs(self, k):
        gen = torch.Generator().manual_seed(1000 + k)
        r = lambda *s, dt=None: torch.randn(*s, generator=gen).to(
            "cuda", self.dt if dt is None else dt)
        t = torch.randint(-1, self.V, (self.M,), generator=gen, dtype=torch.int32)
        lens = torch.randint(0, self.T + 1, (self.B,), generator=gen, dtype=torch.int32)
        lens[0] = self.T
        t.view(self.B, self.T)[torch.arange(self.T)[None, :] >= lens[:, None]] = -1
        return dict(h=r(self.M, self.D), targets=t.cuda(), lens=lens.cuda(),
                    s0=r(self.B, self.W - 1, self.C), h0=r(self.B, self.C, self.N, dt=F32),
                    dloss=torch.where(t >= 0, 1.0, 0.0).cuda() / max(1, int((t >= 0).sum())))

    def load(self, k):
        for name, v in self.inputs(k).items():
            self.i[name].copy_(v)

    def step(self, sync=lambda: None):
        t, i, C, N, W = self.t, self.i, self.C, self.N, self.W
        x, z = t["xz"][:, :C], t["xz"][:, C:]
        dt, Bm, Cm = t["xdb"][:, :C], t["xdb"][:, C:C + N], t["xdb"][:, C + N:]
        ddt, dB, dC = t["dxdb"][:, :C], t["dxdb"][:, C:C + N], t["dxdb"][:, C + N:]
        scan = (t["xc"], dt, z, Bm, Cm, self.A, self.Dv, self.bias, i["lens"])
        conv = (self.d_conv, W, x, self.w_conv, self.b_conv, ssm.CONV_SILU, i["lens"], i["s0"])
        for call in (
            lambda: sb.swimba_output_project(self.d_in, i["h"], self.w_in, t["xz"]),
            lambda: ssm.swimba_causal_conv(*conv, t["xc"], t["s1"]),
            lambda: sb.swimba_output_project(self.d_x, t["xc"], self.w_x, t["xdb"]),
            lambda: ssm.swimba_selective_scan(self.d_scan, *scan, i["h0"], t["y"], t["h1"],
                                              t["carry"], self.ws["scan"]),
            lambda: sb.swimba_output_project(self.d_out, t["y"], self.w_out, t["o"]),
            lambda: ssm.swimba_cross_entropy(self.d_loss, t["o"], self.w_voc, i["targets"],
                                             t["loss"], t["lse"], self.ws["loss"]),
            lambda: ssm.swimba_cross_entropy_backward(
                self.d_loss, t["o"], self.w_voc, i["targets"], t["lse"], i["dloss"], t["do"],
                t["dw_voc"], self.ws["loss_b"]),
            lambda: t["dot"].copy_(t["do"]),
            lambda: sl.swimba_output_project_backward(self.d_out, t["y"], self.w_out, t["dot"],
                                                      t["dy"], t["dw_out"], self.ws["out"]),
            lambda: ssm.swimba_selective_scan_backward(
                self.d_scan, *scan, t["carry"], t["dy"], None, t["dxs"], ddt, t["dxz"][:, C:], dB,
                dC, t["dA"], t["dD"], t["dbias"], t["dh0"], self.ws["scan_b"]),
            lambda: sl.swimba_output_project_backward(self.d_x, t["xc"], self.w_x, t["dxdb"],
                                                      t["dxp"], t["dw_x"], self.ws["x"]),
            lambda: torch.add(t["dxs"], t["dxp"], out=t["dxc"]),
            lambda: ssm.swimba_causal_conv_backward(
                *conv, t["dxc"], None, t["dxz"][:, :C], t["dw_conv"], t["db_conv"], t["ds0"],
                self.ws["conv"]),
            lambda: sl.swimba_output_project_backward(self.d_in, i["h"], self.w_in, t["dxz"],
                                                      t["dh"], t["dw_in"], self.ws["in"]),
        ):
            call()
            sync()

    def poison(self):
        for v in (*self.t.values(), *self.ws.values()):
            v.view(torch.uint8).fill_(255)

    def snapshot(self):
        return {k: v.clone() for k, v in self.t.items()}


def autograd(q):
    """The step in float64: the loss's gradients by torch's own differentiation."""
    f64 = torch.float64
    leaf = lambda t: t.detach().to(f64).requires_grad_()
    w = {k: leaf(getattr(q, "Dv" if k == "D" else k)) for k in Layer.WEIGHTS}
    h, s0, h0 = leaf(q.i["h"]), leaf(q.i["s0"]), leaf(q.i["h0"])
    B, T, C, N, W = q.B, q.T, q.C, q.N, q.W
    live = torch.arange(T, device="cuda")[None, :] < q.i["lens"][:, None]
    xz = (h @ w["w_in"].t()).view(B, T, 2 * C)
    full = torch.cat([s0, xz[..., :C]], 1)
    s = sum(full[:, k:k + T] * w["w_conv"][:, k] for k in range(W)) + w["b_conv"]
    xc = s * torch.sigmoid(s)
    xc = torch.where(live[..., None], xc, 0.0)
    xdb = xc @ w["w_x"].t()
    delta = torch.nn.functional.softplus(xdb[..., :C] + w["bias"], threshold=60.0)
    st, ys = h0, []
    for t in range(T):
        a = torch.exp(delta[:, t, :, None] * w["A"])
        new = a * st + (delta[:, t] * xc[:, t])[..., None] * xdb[:, t, None, C:C + N]
        st = torch.where(live[:, t, None, None], new, st)
        ys.append((st * xdb[:, t, None, C + N:]).sum(-1) + w["D"] * xc[:, t])
    z = xz[..., C:]
    y = torch.stack(ys, 1) * z * torch.sigmoid(z)
    y = torch.where(live[..., None], y, 0.0)
    o = (y @ w["w_out"].t()).view(B * T, q.D)
    logits = o @ w["w_voc"].t()
    lse = torch.logsumexp(logits, 1)
    tgt = q.i["targets"].long()
    ok = tgt >= 0
    loss = torch.where(ok, lse - logits[torch.arange(B * T, device="cuda"), tgt.clamp(min=0)], 0.0)
    (loss * q.i["dloss"].to(f64)).sum().backward()
    g = {k: v.grad for k, v in w.items()}
    return dict(y=y.reshape(B * T, C), h1=st, loss=loss, lse=lse, dh=h.grad, ds0=s0.grad,
                dh0=h0.grad, dw_in=g["w_in"], dw_conv=g["w_conv"], db_conv=g["b_conv"],
                dw_x=g["w_x"], dA=g["A"], dD=g["D"], dbias=g["bias"], dw_out=g["w_out"],
                dw_voc=g["w_voc"])


def distance(got, want):
    got, want = got.double().reshape(want.shape), want.detach()
    return float((got - want).norm() / want.norm())


def test_layer_against_autograd():
    """In float32. Every tensor on the way is off by what its own call adds and what it was
    given: a product of n terms by accumulation(n) in the 2-norm; the scan by up to T steps of
    30 U of the state, the convolution and the loss by less. A gradient has passed all of them
    twice."""
    q = Layer("f32")
    q.step()
    want = autograd(q)
    bound = 2 * (sum(accumulation(n) for n in (q.D, q.C, q.C, q.D, q.V, q.M)) + 30 * q.T * U)
    assert bound < 1.2e-3
    got = {k: distance(q.t[k], v) for k, v in want.items()}
    assert all(v <= bound for v in got.values()), got


def test_layer_in_bfloat16():
    """Tensors between the calls are rounded to bf16: 2^-9 of an element on average less than
    that in the 2-norm, 14 of them on the longest way, each carried on with a gain of order 1."""
    q = Layer("bf16")
    q.step()
    want = autograd(q)
    got = {k: distance(q.t[k], v) for k, v in want.items()}
    assert all(v <= 14 * 2.0 ** -8 for v in got.values()), got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_passes_with_new_inputs(dtype):
    """Pass after pass without waiting, on two streams, against waited-for passes in buffers
    that hold NaN; and each pass again: the same bits."""
    q, ref = Layer(dtype, T=230, seed=3), Layer(dtype, T=230, seed=3)
    side = torch.cuda.Stream()
    for k in range(4):
        q.load(k)
        if k % 2:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                q.step()
            torch.cuda.current_stream().wait_stream(side)
        else:
            q.step()
        got = q.snapshot()
        ref.load(k)
        ref.poison()
        ref.step(torch.cuda.synchronize)
        for name, v in got.items():
            if name != "carry":
                bits(f"pass {k}: {name}", v, ref.t[name])
        q.step()
        for name, v in got.items():
            if name != "carry":
                bits(f"pass {k} again: {name}", q.t[name], v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_replays_from_graphs_that_share_workspaces(dtype):
    a, b = Layer(dtype, seed=4), Layer(dtype, B=2, T=210, seed=5)
    # the larger workspaces serve both
    for k in a.ws:
        if a.ws[k].numel() < b.ws[k].numel():
            a.ws[k] = b.ws[k]
        else:
            b.ws[k] = a.ws[k]
    a.step(), b.step()
    torch.cuda.synchronize()
    graphs = []
    for q in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.step()
        graphs.append(g)
    for k in range(3):
        for q, g in zip((a, b), graphs):
            q.load(10 + k)
            q.poison()
            torch.cuda.synchronize()
            g.replay()
        torch.cuda.synchronize()
        for q in (a, b):
            got = q.snapshot()
            q.step(torch.cuda.synchronize)
            for name, v in got.items():
                if name != "carry":
                    bits(f"replay {k}: {name}", v, q.t[name])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decoding_continues_a_prompt(dtype):
    """A prompt at once and tokens one by one in place, from one captured step, against all
    tokens at once."""
    B, T0, T1, C, N, W = 2, 37, 6, 48, 16, 4
    dt = torch.bfloat16 if dtype == "bf16" else F32
    T = T0 + T1
    r = lambda *s: torch.randn(*s, device="cuda")
    x, z, d = [r(B, T, C).to(dt) for _ in range(3)]
    Bm, Cm = r(B, T, N).to(dt), r(B, T, N).to(dt)
    w, b, A, D, bias = r(C, W).to(dt), r(C).to(dt), -torch.exp(r(C, N)), r(C), r(C) - 2

    def run(t0, t1, s, h):
        n = t1 - t0
        cut = lambda a: a[:, t0:t1].reshape(B * n, -1).contiguous()
        dims = ssm.ssm_dims(B, n, C, N, 1, dtype)
        xc, y = torch.empty(B * n, C, dtype=dt, device="cuda"), \
            torch.empty(B * n, C, dtype=dt, device="cuda")
        s1, h1 = torch.empty(B, W - 1, C, dtype=dt, device="cuda"), torch.empty(B, C, N,
                                                                              device="cuda")
        ssm.swimba_causal_conv(dims, W, cut(x), w, b, 1, None, s, xc, s1)
        ssm.swimba_selective_scan(dims, xc, cut(d), cut(z), cut(Bm), cut(Cm), A, D, bias, None, h,
                                  y, h1, None, ssm.ssm_workspace(dims, ssm.SELECTIVE_SCAN))
        return y.view(B, n, C), s1, h1

    want, s_end, h_end = run(0, T, None, None)
    got, s, h = run(0, T0, None, None)
    d1 = ssm.ssm_dims(B, 1, C, N, 1, dtype)
    tok = {k: torch.empty(B, n, dtype=dt, device="cuda") for k, n in
           (("x", C), ("z", C), ("d", C), ("B", N), ("C", N), ("xc", C), ("y", C))}

    def step():
        ssm.swimba_causal_conv_step(d1, W, tok["x"], w, b, 1, s, s, tok["xc"])
        ssm.swimba_selective_step(d1, tok["xc"], tok["d"], tok["z"], tok["B"], tok["C"], A, D,
                                  bias, h, h, tok["y"])

    keep = s.clone(), h.clone()
    step()
    torch.cuda.synchronize()
    s.copy_(keep[0]), h.copy_(keep[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in range(T0, T):
        for k, a in (("x", x), ("z", z), ("d", d), ("B", Bm), ("C", Cm)):
            tok[k].copy_(a[:, t])
        g.replay()
        got = torch.cat([got, tok["y"][:, None]], 1)
    bits("convolution state", s, s_end)
    # the same operations but for the segments' joins: 30 U a step of the states' magnitude
    tol = 30 * T * U
    assert distance(h, h_end.double()) <= tol
    assert distance(got, want.double()) <= tol + torch.finfo(dt).eps / 2


def test_an_earlier_error_is_not_the_calls_own():
    """A call that launches its kernels succeeds, whatever failed before it in the thread."""
    hip = ssm.lib()
    hip.hipSetDevice.restype = hip.hipGetLastError.restype = ctypes.c_int
    q = Layer("bf16")
    q.step()
    torch.cuda.synchronize()
    i, t, C = q.i, q.t, q.C
    d0 = ssm.ssm_dims(2, 0, C, 16, 1, "bf16")
    one = ssm.ssm_dims(2, 1, C, 16, 1, "bf16")
    h, ho, s = torch.zeros(2, C, 16, device="cuda"), torch.zeros(2, C, 16, device="cuda"), \
        torch.zeros(2, 3, C, device="cuda").bfloat16()
    so, y1 = torch.empty_like(s), torch.empty(2, C, device="cuda").bfloat16()
    x1, b1 = torch.zeros(2, C, device="cuda").bfloat16(), torch.zeros(2, 16, device="cuda").bfloat16()
    calls = {
        "conv": lambda: ssm.swimba_causal_conv(q.d_conv, 4, t["xz"][:, :C], q.w_conv, None, 1,
                                               None, None, t["xc"]),
        "conv_backward": lambda: ssm.swimba_causal_conv_backward(
            q.d_conv, 4, t["xz"][:, :C], q.w_conv, None, 1, None, None, t["dxc"], None, t["dxp"],
            t["dw_conv"], None, None, q.ws["conv"]),
        "conv_step": lambda: ssm.swimba_causal_conv_step(one, 4, x1, q.w_conv, None, 1, s, so, y1),
        "conv_none": lambda: ssm.swimba_causal_conv(d0, 4, x1, q.w_conv, None, 1, None, None, y1,
                                                    so),
        "scan": lambda: ssm.swimba_selective_scan(
            q.d_scan, t["xc"], t["xdb"][:, :C], None, t["xdb"][:, C:C + 16],
            t["xdb"][:, C + 16:], q.A, None, None, None, None, t["y"], None, t["carry"],
            q.ws["scan"]),
        "scan_backward": lambda: ssm.swimba_selective_scan_backward(
            q.d_scan, t["xc"], t["xdb"][:, :C], None, t["xdb"][:, C:C + 16],
            t["xdb"][:, C + 16:], q.A, None, None, None, t["carry"], t["dy"], None, t["dxs"],
            t["dxdb"][:, :C], None, t["dxdb"][:, C:C + 16], t["dxdb"][:, C + 16:], t["dA"], None,
            None, None, q.ws["scan_b"]),
        "scan_none": lambda: ssm.swimba_selective_scan(d0, x1, x1, None, b1, b1, q.A, None, None,
                                                       None, h, y1, ho, None, None),
        "step": lambda: ssm.swimba_selective_step(one, x1, x1, None, b1, b1, q.A, None, None, h,
                                                  ho, y1),
        "loss": lambda: ssm.swimba_cross_entropy(q.d_loss, t["o"], q.w_voc, i["targets"],
                                                 t["loss"], t["lse"], q.ws["loss"]),
        "loss_backward": lambda: ssm.swimba_cross_entropy_backward(
            q.d_loss, t["o"], q.w_voc, i["targets"], t["lse"], i["dloss"], t["do"], t["dw_voc"],
            q.ws["loss_b"]),
    }
    for c in calls.values():
        c()
    torch.cuda.synchronize()
    failed = []
    for name, c in calls.items():
        assert hip.hipSetDevice(1 << 20) != 0  # refused by the host: there is no such device
        try:
            c()
        except sb.SwimbaError as e:
            failed.append(f"{name}: {e}")
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert not failed, failed


def test_refusals_on_the_device():
    """A stride, a type, a size and a workspace that the binding lets nobody pass."""
    d = ssm.ssm_dims(2, 40, 32, 16, 1, "bf16")
    x = torch.zeros(80, 32, device="cuda").bfloat16()
    w, y = torch.zeros(32, 4, device="cuda").bfloat16(), torch.zeros_like(x)
    conv = lambda **k: ssm.swimba_causal_conv(**{**dict(
        dims=d, width=4, x=x, weight=w, bias=None, act=1, seq_lens=None, state_in=None, y=y), **k})
    conv()
    for bad in (dict(x=x[:79]), dict(x=x.float()), dict(x=x.t()), dict(weight=w[:, :3]),
                dict(y=y.cpu()), dict(seq_lens=torch.zeros(2, device="cuda", dtype=torch.int64)),
                dict(seq_lens=torch.zeros(1, device="cuda", dtype=torch.int32))):
        with pytest.raises(ValueError):
            conv(**bad)
    five = torch.zeros(32, 5, device="cuda").bfloat16()
    odd = torch.zeros(80, 33, device="cuda").bfloat16()[:, 1:]
    for bad in (dict(width=5, weight=five), dict(act=7), dict(x=odd)):
        with pytest.raises(sb.SwimbaError):
            conv(**bad)
    ld = ssm.loss_dims(80, 32, 100, "bf16")
    wv, t = torch.zeros(100, 32, device="cuda").bfloat16(), \
        torch.zeros(80, device="cuda", dtype=torch.int32)
    l = torch.zeros(80, device="cuda")
    with pytest.raises(sb.SwimbaError, match="workspace"):
        ssm.swimba_cross_entropy(ld, x, wv, t, l, l.clone(), torch.empty(16, device="cuda",
                                                                         dtype=torch.uint8))
    with pytest.raises(ValueError):
        ssm.swimba_cross_entropy(ld, x, wv[:99], t, l, l.clone(),
                                 ssm.ssm_workspace(ld, ssm.CROSS_ENTROPY))
