"""Runs of layer calls whose inputs change from pass to pass, and the mixer's
training step with the layer norm before it and the output projection behind it.

A pass reads what the pass before left nowhere: every tensor between the calls
is compared bit for bit with a pass in buffers of its own that were filled with
NaN and in which every call was waited for. A kernel that read an earlier pass's
value (of a tensor that the call before it stored past the L2's reuse order, for
instance) would differ."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import TOL, check_routing, dev, host, tdt
from oracle import backward as ob
from oracle import layers as ol
from oracle import swimba as osw
from selective_ssm_parameter_amd import binding as sb
from selective_ssm_parameter_amd import layers as sl
from selective_ssm_parameter_amd import synth
from test_gpu_layers_block import Block

pytestmark = pytest.mark.gpu

EPS = 1e-5


def same_bits(name, a, b):
    """Equal as bits, so that equal NaN count as equal and -0 does not equal 0."""
    ints = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[a.element_size()]
    assert torch.equal(a.view(ints), b.view(ints)), name


def poison(tensors):
    for t in tensors:
        t.view(torch.uint8).fill_(255)


class LayerPasses:
    """The block of recurrence and feed-forward layer, a new x, dout, h0, dh and
    lengths in every pass."""

    def __init__(self, B, T, D, C, F, dtype):
        self.args, self.shape = (B, T, D, C, F, dtype), (B * T, D)
        self.blk = Block(*self.args, seed=5)

    def inputs(self, i):
        gen = torch.Generator().manual_seed(100 + i)
        b = self.blk
        f = lambda t: torch.randn(t.shape, generator=gen).to("cuda", t.dtype)
        lens = torch.randint(0, b.T + 1, (b.B,), generator=gen).to("cuda", torch.int32)
        return {"x": f(b.x), "dout": f(b.dout), "h0": f(b.h0), "dh": f(b.dh), "lens": lens}

    def load(self, blk, inp):
        for k, v in inp.items():
            getattr(blk, k).copy_(v)

    def run(self, blk):
        blk.forward()
        blk.backward()

    def between(self, blk):
        # the carry's rows behind a length are not written
        return {k: v for k, v in {**blk.a, **blk.g}.items() if k != "carry"}

    def fresh(self):
        blk = Block(*self.args, seed=5)
        poison(list(blk.a.values()) + list(blk.g.values()) + list(blk.ws.values()))
        return blk


class MixerStep:
    """n = norm(x), y = mixer(n), out = y W_out^T, and back to dx."""

    def __init__(self, wl, seed=0):
        self.wl = wl
        dt, M, D, HP = tdt(wl), wl.tokens, wl.d_model, wl.d_inner
        inp = synth.make_inputs(wl)
        r = np.random.default_rng(wl.seed + 17)
        self.wr, self.we = dev(inp["w_router"], dt), dev(inp["w_experts"], dt)
        self.av = dev(inp["a"], torch.float32)
        self.w_out = dev(synth.output_projection_inputs(wl, rows=1)["w_out"], dt)
        self.w, self.b = dev(1 + 0.2 * r.standard_normal(D), dt), \
            dev(0.2 * r.standard_normal(D), dt)
        self.x = dev(inp["u"].reshape(M, D), dt)
        self.dout = dev(r.standard_normal((M, D)), dt)
        self.dims, self.d_norm = sb.dims_of(wl), sl.layer_dims(wl.batch, wl.seqlen, D, 8, wl.dtype)
        e = lambda *s, d=dt: torch.empty(*s, dtype=d, device="cuda")
        f32 = torch.float32
        self.buf, self.grads = sb.alloc_buffers(self.dims, "cuda"), sb.alloc_grads(self.dims)
        self.t = {"n": e(M, D), "mean": e(M, d=f32), "rstd": e(M, d=f32), "out": e(M, D),
                  "dy": e(M, HP), "dwo": e(D, HP, d=f32), "dx": e(M, D, d=f32),
                  "dw": e(D, d=f32), "db": e(D, d=f32)}
        self.ws = [sl.layer_workspace(self.d_norm, sl.LAYER_NORM_BACKWARD),
                   sl.layer_workspace(self.dims, sl.LAYER_OUTPUT_PROJECT_BACKWARD)]

    def run(self, between=lambda: None):
        t, wl, b, g = self.t, self.wl, self.buf, self.grads
        M, HP = wl.tokens, wl.d_inner
        sl.swimba_layer_norm(self.d_norm, self.x, None, self.w, self.b, EPS, None, t["n"],
                             t["mean"], t["rstd"])
        between()
        sb.forward(self.dims, t["n"], self.wr, self.we, self.av, None, b)
        between()
        sb.swimba_output_project(self.dims, b.y.view(M, HP), self.w_out, t["out"])
        between()
        sl.swimba_output_project_backward(self.dims, b.y.view(M, HP), self.w_out, self.dout,
                                          t["dy"], t["dwo"], self.ws[1])
        between()
        sb.backward(self.dims, t["n"], self.wr, self.we, self.av, None,
                    t["dy"].view(M, wl.nheads, wl.headdim), None, b, g)
        between()
        sl.swimba_layer_norm_backward(self.d_norm, self.x, self.w, t["mean"], t["rstd"], g.du,
                                      None, t["dx"], t["dw"], t["db"], self.ws[0])
        between()

    def tensors(self):
        b, g = self.buf, self.grads
        return {**self.t, "idx": b.topk_idx, "B_hat": b.B_hat, "X_hat": b.X_hat, "C_mix": b.C_mix,
                "y": b.y, "du": g.du, "dW_router": g.dW_router, "dW_experts": g.dW_experts,
                "da": g.da}


class MixerPasses:
    def __init__(self, wl):
        self.wl = wl
        self.blk = MixerStep(wl)

    def inputs(self, i):
        gen = torch.Generator().manual_seed(200 + i)
        f = lambda t: torch.randn(t.shape, generator=gen).to("cuda", t.dtype)
        return {"x": f(self.blk.x), "dout": f(self.blk.dout)}

    load = LayerPasses.load

    def run(self, blk):
        blk.run()

    def between(self, blk):
        return blk.tensors()

    def fresh(self):
        blk = MixerStep(self.wl)
        poison(list(blk.tensors().values()) + blk.ws)
        return blk


MIXER = synth.small("layers_chain", 31, batch=3, seqlen=700, d_model=512, nheads=6, headdim=64,
                    dstate=128, ngroups=1, n_experts=4, top_k=2, chunk=64, dtype=synth.BF16,
                    a_lo=0.9, a_hi=0.999)
PASSES = {
    # every output row starts on a 128-byte line
    "layers": lambda: LayerPasses(4, 2048, 512, 384, 640, "bf16"),
    "layers_f32": lambda: LayerPasses(3, 700, 256, 192, 320, "f32"),
    "mixer": lambda: MixerPasses(MIXER),
}


@pytest.mark.parametrize("kind", PASSES)
def test_passes_with_new_inputs(kind):
    p, n = PASSES[kind](), 5
    inputs = [p.inputs(i) for i in range(n)]
    torch.cuda.synchronize()
    got = []
    for inp in inputs:  # one after the other in the same buffers, nothing waited for
        p.load(p.blk, inp)
        p.run(p.blk)
        got.append({k: v.clone() for k, v in p.between(p.blk).items()})
    torch.cuda.synchronize()
    for i, inp in enumerate(inputs):
        blk = p.fresh()
        torch.cuda.synchronize()
        p.load(blk, inp)
        torch.cuda.synchronize()
        p.run(blk)
        torch.cuda.synchronize()
        for k, v in p.between(blk).items():
            same_bits(f"pass {i}: {k}", got[i][k], v)


@pytest.mark.parametrize("kind", ["layers", "mixer"])
def test_replays_with_new_inputs(kind):
    """The same from a captured graph, with eager passes between the replays."""
    p, n = PASSES[kind](), 5
    inputs = [p.inputs(10 + i) for i in range(n)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        p.run(p.blk)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            p.run(p.blk)
    torch.cuda.synchronize()
    got = []
    for i, inp in enumerate(inputs):
        p.load(p.blk, inp)
        if i == 2:
            p.run(p.blk)
        else:
            g.replay()
        got.append({k: v.clone() for k, v in p.between(p.blk).items()})
    torch.cuda.synchronize()
    for i, inp in enumerate(inputs):
        blk = p.fresh()
        p.load(blk, inp)
        torch.cuda.synchronize()
        p.run(blk)
        torch.cuda.synchronize()
        for k, v in p.between(blk).items():
            same_bits(f"replay {i}: {k}", got[i][k], v)


# In the 2-norm. The mixer's own results are within TOL of the exact ones for
# the inputs they get (each row against its largest or root mean square element,
# which bounds the 2-norm's ratio by the square root of 2 times that). Around it
# the chain rounds y, out and dy to dtype, each by at most eps / 2 of a value. No
# result is behind more than two of them, and a rounding passes the linear maps
# behind it as the value does: a factor of 2 is left for the difference.
def chain_bound(wl):
    return 2 ** 0.5 * TOL[wl.dtype] + 4 * torch.finfo(tdt(wl)).eps / 2


@pytest.mark.parametrize("dtype", [synth.BF16, synth.F32])
def test_mixer_training_step(dtype):
    """layer norm -> mixer -> output projection and all of it back, against the
    float64 oracle's chain (which takes the norm's output as it is stored, so
    that both route the same tokens alike)."""
    wl = synth.small("mixer_step", 41, batch=2, seqlen=300, d_model=128, nheads=3, headdim=64,
                     dstate=64, ngroups=1, n_experts=4, top_k=2, chunk=64, dtype=dtype, a_lo=0.9,
                     a_hi=0.999)
    st = MixerStep(wl)
    st.run()
    torch.cuda.synchronize()
    M, D, H, P = wl.tokens, wl.d_model, wl.nheads, wl.headdim
    x, w, b = host(st.x), host(st.w), host(st.b)
    n, _, _ = ol.layer_norm(x, w, b, EPS)
    stored = host(st.t["n"])
    half = torch.finfo(tdt(wl)).eps / 2
    assert np.linalg.norm(stored - n) <= (half + 2.0 ** -18) * np.linalg.norm(n)
    u = stored.reshape(wl.batch, wl.seqlen, D)
    wr, we, a, wo, dout = (host(t) for t in (st.wr, st.we, st.av, st.w_out, st.dout))
    kw = dict(nheads=H, headdim=P, ngroups=wl.ngroups, dstate=wl.dstate, top_k=wl.top_k)
    r = check_routing(host(st.buf.topk_idx).astype(np.int64), None,
                      osw.route(u.reshape(M, D), wr, wl.top_k), wl)
    y = osw.forward(u, wr, we, a, None, routing=r, **kw)["y"].reshape(M, H * P)
    dy, dwo = ol.output_project_backward(y, wo, dout)
    ref = ob.forward_backward(u, wr, we, a, None, dy.reshape(wl.batch, wl.seqlen, H, P),
                              np.zeros((wl.batch, H, wl.dstate, P)), routing=r, **kw)
    dx, dw, db = ol.layer_norm_backward(x, w, EPS, ref["du"].reshape(M, D))
    want = {"out": y @ wo.T, "dy": dy, "dwo": dwo, "dW_router": ref["dW_router"],
            "dW_experts": ref["dW_experts"], "da": ref["da"], "dx": dx, "dw": dw, "db": db}
    got = st.tensors()
    for k, v in want.items():
        g = host(got[k]).reshape(v.shape)
        err = np.linalg.norm(g - v) / np.linalg.norm(v)
        assert err <= chain_bound(wl), f"{k}: {err} against {chain_bound(wl)}"


def test_block_in_float32_closely():
    """The block of recurrence and feed-forward layer in float32 against autograd
    in float64. A product of n <= 450 terms is off by U sqrt(n / 2) and by U n / 24
    if blocks of 32 terms truncate: 34 U. A result is behind at most 8 of them, with
    slopes of up to 2, which add at random, and 13 roundings of U: below 200 U; a
    quarter of that again for gates and statistics."""
    blk = Block(3, 150, 96, 64, 136, "f32", seed=3)
    blk.forward()
    blk.backward()
    for name, got, want in zip(Block.NAMES, blk.outputs(), blk.reference()):
        want = want.detach()
        err = ((got.double().cpu() - want).norm() / want.norm()).item()
        assert err <= 256 * 2.0 ** -24, f"{name}: {err}"
