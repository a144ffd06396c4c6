"""Shapes (tokens, d_model, inner width, type) that between them reach every
kernel of the dense layer products: each tile of each product, with k in one run
and in several, and every form that streams the weights. The names are those
that test_layers_plan_host.py asks the library's own choice for."""
from __future__ import annotations

import numpy as np

SHAPES = [
    # at most 64 tokens: the weights streamed
    (9, 1000, 136, "bf16"), (13, 264, 3080, "bf16"), (29, 264, 520, "bf16"),
    (61, 1032, 200, "bf16"),
    (9, 1000, 136, "f32"), (13, 264, 3080, "f32"), (29, 264, 520, "f32"), (61, 1032, 200, "f32"),
    # tiles
    (100, 72, 40, "f32"), (109, 72, 40, "bf16"), (1360, 72, 344, "f32"), (1021, 40, 376, "bf16"),
    (12452, 72, 72, "f32"), (11235, 72, 72, "bf16"), (132, 1272, 816, "bf16"),
    (16742, 72, 168, "bf16"), (100, 736, 40, "f32"), (100, 1648, 904, "f32"),
    (129, 1376, 1544, "bf16"), (104, 136, 4104, "f32"), (3163, 72, 776, "f32"),
    (14357, 136, 40, "f32"), (16425, 72, 336, "bf16"), (1293, 72, 1560, "f32"),
    (101, 1096, 3624, "bf16"), (3359, 2720, 72, "bf16"), (234, 2064, 1560, "f32"),
    (1822, 72, 2112, "f32"), (1417, 3096, 72, "f32"), (13156, 776, 40, "bf16"),
    (2220, 2104, 200, "f32"), (3221, 136, 3328, "bf16"), (100, 2144, 2768, "bf16"),
    (17296, 72, 584, "bf16"), (103, 2536, 3208, "bf16"), (103, 3096, 3832, "bf16"),
    (4332, 392, 2152, "bf16"), (9069, 3008, 136, "bf16"), (8366, 2800, 392, "bf16"),
]

U = 2.0 ** -24


def accumulation(n):
    """Bound of the error in the 2-norm, relative to the result, of fp32 sums of n
    terms of random sign. The k-th partial sum is about sqrt(k) terms large and
    rounds by U of itself: together U n / sqrt(2) terms, against a result of
    sqrt(n). A factor of 11 over that U sqrt(n / 2) covers blocks that add up with
    one sign (32 terms at a time, an error of U n / 24 if every block truncates)."""
    return 8 * np.sqrt(n) * U


def dz_error(D, dtype):
    """The same of dz = [dh u act'(g) | dh act(g)], g and u sums of D terms: their
    own errors reach it with slopes of up to about 1 in each of u, act' and act;
    the activation's exp of a rounded argument is off by (8 + 2 |g| + g^2) U, 32 U
    for values of order 1; bf16 problems hold dz as two bf16 numbers, the second off
    by 2^-8 of what the first left, 2^-8 of dz."""
    return 3 * accumulation(D) + 32 * U + (2.0 ** -16 if dtype == "bf16" else U)


def distance(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))
