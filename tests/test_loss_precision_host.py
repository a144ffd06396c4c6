"""What the precision tests of the cross entropy's gradients tell apart: dz as three
bf16 numbers passes their bounds, as two it does not (numpy, on the CPU)."""
from __future__ import annotations

import numpy as np
import pytest

import loss_precision as lp
from oracle import ssm as osm


def test_three_numbers_hold_a_float32():
    r = np.random.default_rng(0)
    a = (r.standard_normal(100000) * np.exp(r.uniform(-20, 20, 100000))).astype(np.float32)
    assert np.array_equal(lp.numbers(a, 3), a.astype(np.float64))


@pytest.mark.parametrize("M,D,V", lp.STEPS)
def test_bounds_tell_two_numbers_from_three(M, D, V):
    if M * V > 1 << 21:
        M = (1 << 21) // V  # (what dz alone is off by does not depend on the tokens' number)
    x, w, t, g = lp.step(M, D, V, seed=V)
    _, _, dz = osm.cross_entropy_backward(x.astype(np.float64), w.astype(np.float64), t, g)
    f = dz.astype(np.float32)
    for n, ok in ((3, True), (2, False), (1, False)):
        d = lp.numbers(f, n)
        for got, want, terms in ((d @ w, dz @ w, V), (d.T @ x, dz.T @ x, max(M, 16400))):
            err = np.linalg.norm(got - want) / np.linalg.norm(want)
            assert (err <= lp.bound(terms)) == ok, (n, terms, err, lp.bound(terms))
