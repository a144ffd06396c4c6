"""Shapes at which a thread of the convolution walks many rows in turn, in both
directions, and at which one of the single-token scan takes two sequences
(test_ssm_plan_host.py asks the library's own choice for them)."""

# batch, tokens, channels, type, width, act, state, ragged, pad: full vectors and single
# elements of both types
CONV = [(3, 16411, 1024, "bf16", 4, 1, True, True, 64), (3, 2100, 1001, "bf16", 4, 1, True, True, 0),
        (2, 12301, 1024, "f32", 3, 0, False, True, 0), (5, 1300, 1001, "f32", 4, 1, True, True, 3),
        (1, 65605, 2048, "bf16", 2, 1, True, False, 0), (70, 733, 1000, "bf16", 4, 1, False, True, 8)]

# batch (odd: the last thread's second sequence does not exist), channels, states, groups, gate
STEP = [(257, 1024, 16, 1, True), (257, 1024, 18, 2, False), (4097, 64, 3, 1, True),
        (131, 2048, 40, 1, True)]
