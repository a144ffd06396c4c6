"""The cross entropy's gradients from all bits of dz, whatever the number of tokens."""
from __future__ import annotations

import pytest
import torch

import loss_precision as lp
from selective_ssm_parameter_amd import ssm
from ssm_bounds import DT, dev, empty

pytestmark = pytest.mark.gpu


def run(d, x, w, t, g):
    (M, D), V = x.shape, w.shape[0]
    loss, lse, dx, dw = empty(M), empty(M), empty(M, D), empty(V, D)
    ssm.swimba_cross_entropy(d, x, w, t, loss, lse, ssm.ssm_workspace(d, ssm.CROSS_ENTROPY))
    ssm.swimba_cross_entropy_backward(d, x, w, t, lse, g, dx, dw,
                                      ssm.ssm_workspace(d, ssm.CROSS_ENTROPY_BACKWARD))
    return dx, dw


@pytest.mark.parametrize("M,D,V", lp.STEPS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_take_all_of_dz(M, D, V, dtype):
    x, w, t, g = lp.step(M, D, V, seed=V)
    x, w, t, g = dev(x, DT[dtype]), dev(w, DT[dtype]), dev(t, torch.int32), dev(g)
    dx, dw = run(ssm.loss_dims(M, D, V, dtype), x, w, t, g)
    f64 = torch.float64
    xd, wd, ok = x.to(f64), w.to(f64), t >= 0
    dz = torch.softmax(xd @ wd.t(), 1)
    at = torch.arange(M, device="cuda")[ok], t[ok].long()
    dz[at] -= 1
    dz *= torch.where(ok, g.to(f64), 0.0)[:, None]
    for name, got, want, n in (("dx", dx, dz @ wd, V), ("dw", dw, dz.t().contiguous() @ xd, M)):
        err = float((got.to(f64) - want).norm() / want.norm())
        assert err <= lp.bound(n), (name, err, lp.bound(n))
