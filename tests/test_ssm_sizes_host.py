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
