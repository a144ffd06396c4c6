"""The loss of the cross entropy to what float32 holds: small losses next to large
logits, and infinite ones."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from selective_ssm_parameter_amd import ssm
from ssm_bounds import DT, U, dev, empty, host

pytestmark = pytest.mark.gpu


def run(d, x, w, t):
    loss, lse = empty(x.shape[0]), empty(x.shape[0])
    ssm.swimba_cross_entropy(d, x, w, t, loss, lse, ssm.ssm_workspace(d, ssm.CROSS_ENTROPY))
    return loss, lse


# (words, distance of the others below the target's logit)
CONFIDENT = [(4, 8), (37, 8), (300, 14), (777, 16), (5003, 17), (4, 40)]


@pytest.mark.parametrize("V,gap", CONFIDENT)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_losses_next_to_large_logits(V, gap, dtype):
    """Tokens whose target's logit is the largest, at up to 2^20 (logits are exact: the largest
    as two features of 8 bits, the gap as a third).

    The logarithm's argument is 1 and little more. Each sum that makes it - a tile's up to 256
    words, lane groups, waves and tiles - rounds by U; the exponential of -gap is off by
    (2 gap + 4) U of itself, the logarithm and the last sum by 2 U of theirs; the difference to
    the largest logit is exact."""
    tops, D, target = [0.0, 20.0, 200.0, 5000.0, 2.0 ** 20, -5000.0], 8, V * 2 // 3
    x, w = np.zeros((len(tops), D)), np.zeros((V, D))
    for m, top in enumerate(tops):
        hi = float(torch.tensor(top).bfloat16())
        x[m, :3] = hi, top - hi, gap
    w[:, :2], w[:, 2], w[target, 2] = 1.0, -1.0, 0.0
    got = run(ssm.loss_dims(len(tops), D, V, dtype), dev(x, DT[dtype]), dev(w, DT[dtype]),
              dev(np.full(len(tops), target), torch.int32))[0]
    want = np.log1p((V - 1) * np.exp(-float(gap)))
    tol = (256 + 8 + V / 128 + (2 * gap + 8) * want) * U
    assert (np.abs(host(got) - want) <= tol).all(), (got, want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_losses_of_infinite_logits(dtype):
    """A target at -inf costs infinitely much; a row of -inf alone, or with +inf or NaN, has no
    loss; a word of -inf that is not the target counts for nothing."""
    V, D = 130, 8
    x, w = np.zeros((5, D)), np.zeros((V, D))
    w[:, 0], w[:, 1], w[3, 1], w[:, 2] = 1.0, 2.0 ** -100, -4.0, -1.0
    x[:2, 0], x[:2, 1] = 2.0, 2.0 ** 127  # word 3 overflows to -inf, the others are at 2^27
    x[2, 2] = np.inf                      # every word at -inf
    x[3, 1] = -2.0 ** 127                 # word 3 at +inf
    x[4, 0] = np.nan
    t = np.array([3, 5, 5, 3, 5], np.int32)
    loss, lse = run(ssm.loss_dims(5, D, V, dtype), dev(x, DT[dtype]), dev(w, DT[dtype]),
                    dev(t, torch.int32))
    loss, lse = host(loss), host(lse)
    assert loss[0] == np.inf and np.isnan(loss[2:]).all()
    assert np.isfinite(lse[:2]).all() and lse[2] == -np.inf and not np.isfinite(lse[3:]).any()
    assert abs(loss[1] - np.log(V - 1)) <= (256 + 8 + 8) * U * np.log(V - 1)
