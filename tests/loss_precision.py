"""A training step of the cross entropy whose error is that of dz: logits close to
each other, so that a token's dz is -(1 - 1 / V) of its dloss at the target and next
to nothing elsewhere, and a dloss whose product with that is as far as can be from a
sum of two bf16 numbers.

U = 2^-24. An element of dz is off by the roundings of exp - 1 and of the product,
2 U, and by its logit's and lse's errors, which the probability 1 / V makes
negligible (1 U allowed); held as three bf16 numbers it loses nothing more. A sum of
n terms is off, in the 2-norm, by n roundings of partial sums, each at most U of one:
with independent signs U sqrt(sum_k k / n) = U sqrt(n / 2) of the result. Two bf16
numbers of a dz chosen as here are off by 2^-17.3 = 6.2e-6, 104 U."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24

# (tokens, d_model, vocabulary): both sides of 8192 tokens, few and many words, words
# in several pieces; and every tile of both types' products, with the sum in one run and
# in several (test_loss_plan_host.py asks the library's own choice for them).
STEPS = [(1, 64, 40), (246, 480, 832), (1000, 1032, 2051), (8192, 64, 500), (8193, 64, 500),
         (9000, 256, 300), (16400, 64, 9001),
         (134, 2472, 7491), (8637, 232, 2546), (8364, 1384, 24), (2448, 1360, 24),
         (3144, 1360, 24), (4655, 1720, 24), (1358, 224, 18734), (913, 176, 16508),
         (1, 872, 13203), (1, 296, 24227), (1, 1744, 1815), (2680, 1800, 72), (296, 8, 20676),
         (2073, 112, 4106), (1352, 24, 6274), (3076, 72, 1510), (765, 696, 2645),
         (6744, 200, 24), (3838, 520, 24), (1, 144, 10910), (1, 1704, 938)]


def bf16(a):
    """Rounded to bf16 (to nearest, ties to even), as float32."""
    b = np.asarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return (((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def numbers(a, n):
    """The sum of n bf16 numbers nearest to a, one after the other."""
    left, total = np.asarray(a, np.float32), np.zeros(np.shape(a))
    for _ in range(n):
        h = bf16(left)
        total += h.astype(np.float64)
        left = left - h
    return total


def dloss_of(V):
    """The dloss in [1, 2) whose dz at a target, (1 / V - 1) dloss in float32, is farthest
    from two bf16 numbers, relative to itself."""
    g = (1 + np.arange(1 << 16) / (1 << 16) + np.arange(1 << 16) % 128 * U * 2).astype(np.float32)
    d = (np.float32(1.0 / V - 1) * g).astype(np.float32)
    err = np.abs(numbers(d, 2) - d.astype(np.float64)) / np.abs(d)
    return float(g[np.argmax(err)])


def bound(n):
    return U * (3 + np.sqrt(n / 2))


def step(M, D, V, seed):
    """x [M, D], w [V, D] (values of bf16), targets and dloss [M]; every fifth token without
    a target where there are more than a few."""
    r = np.random.default_rng(seed)
    x = bf16(r.standard_normal((M, D)))
    w = bf16(r.standard_normal((V, D)) * 1e-5 * D ** -0.5)
    t = r.integers(0, V, M).astype(np.int32)
    if M > 4:
        t[::5] = -1
    g = np.full(M, dloss_of(V), np.float32) * np.where(np.arange(M) % 3 == 0, -2.0, 1.0)
    return x, w, t, g.astype(np.float32)
