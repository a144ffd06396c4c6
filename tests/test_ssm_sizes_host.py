"""Sizes that the selective layer's calls ask for and the limits that the header
states (host only)."""
from __future__ import annotations

import os

import pytest

from selective_ssm_parameter_amd import binding as sb
from selective_ssm_parameter_amd import ssm


@pytest.fixture(autouse=True)
def library():
    if not os.path.exists(sb.LIB_PATH):
        pytest.skip("libswimba.so not built")


def dims(d_model=1, batch=2, seqlen=3000, c=64, n=16, dtype="bf16"):
    return sb.make_dims(batch, seqlen, d_model, 1, c, n, 1, 1, 1, 1, dtype)


@pytest.mark.parametrize("call", [ssm.CAUSAL_CONV_BACKWARD, ssm.SELECTIVE_SCAN,
                                  ssm.SELECTIVE_SCAN_BACKWARD])
@pytest.mark.parametrize("d_model", [2, (1 << 20) + 8, 1 << 23])
def test_d_model_means_nothing_to_the_scan_and_the_convolution(call, d_model):
    """(The calls take any d_model that swimba.h takes, so their workspaces must exist.)"""
    want = ssm.ssm_workspace_size(dims(), call)
    assert want > 0 and ssm.ssm_workspace_size(dims(d_model), call) == want


def refused(call, M, D, V, dtype="bf16"):
    """The status of a loss call that has no workspace: -4 where the sizes are taken."""
    fake, d = 0x1000, ssm.loss_dims(M, D, V, dtype)
    if call == ssm.CROSS_ENTROPY:
        return ssm.lib().swimba_cross_entropy(d, fake, fake, fake, fake, fake, None, 0, None)
    return ssm.lib().swimba_cross_entropy_backward(d, fake, fake, fake, fake, fake, fake, fake, None,
                                                   0, None)


@pytest.mark.parametrize("call", [ssm.CROSS_ENTROPY, ssm.CROSS_ENTROPY_BACKWARD])
def test_limits_of_the_vocabulary(call):
    """What the header says of V, D and M, on both sides of each limit."""
    take, dims_, unsupported = -4, -2, -3
    assert refused(call, 8, 8, 1 << 20) == take and refused(call, 8, 8, (1 << 20) + 1) == dims_
    assert refused(call, 8, 8192, (1 << 18) - 3) == take
    assert refused(call, 8, 8192, (1 << 18) - 2) == dims_
    assert refused(call, 8, 1 << 20, 2045) == take and refused(call, 8, 1 << 20, 2046) == dims_
    assert refused(call, 8, (1 << 20) + 8, 8) == dims_
    assert refused(call, 8, 12, 100) == unsupported
    assert refused(call, (1 << 28) - 17, 8, 8) == take and refused(call, 1 << 28, 8, 8) == dims_
    # 2^16 tokens of 2^20 words, and four times as many
    assert refused(call, 1 << 16, 8, 1 << 20) == take
    assert refused(call, 1 << 18, 8, 1 << 20) == dims_


def test_workspace_of_the_loss_backward():
    """dz of a piece as the header states it, besides a copy of x and the partial sums."""
    size = lambda M, D, V, t: ssm.ssm_workspace_size(ssm.loss_dims(M, D, V, t),
                                                     ssm.CROSS_ENTROPY_BACKWARD)
    for t, es, per in (("bf16", 2, 6), ("f32", 4, 4)):
        for M, D, V in ((1000, 64, 500), (8192, 64, 131072), (16384, 64, 32768), (1 << 17, 64, 9000),
                        (1 << 20, 64, 9000)):
            rest = M * D * es + 64 * 4 * (M + 16384) * D + 4096
            dz = per * (max(1 << 27, 1024 * M) if M * V > 1 << 27 else M * (V + 7))
            assert M * D * es < size(M, D, V, t) <= dz + rest, (t, M, D, V)
