"""Bounds for comparing the INT8 and grouped products with their 64-bit definition.

An FP32 sum of K products of exactly represented operands, in any order, is off
by at most K * 2^-24 / (1 - K * 2^-24) times the sum of the products'
magnitudes ("mass"); every FP32 operation after it adds at most 2^-24 of its
result. The rounding of the output is off by at most half a step: 2^-24
relative for FP32, 2^-8 for BF16 (half the distance 2^-7 between neighbours of
1), and 2^-134 absolute among BF16's subnormals.
"""
import numpy as np

from tests import tolerance

U = 2.0 ** -24


def bound(y, z, mass, sum_terms, act, bf16, addends=0.0):
    """Largest |out - y|. sum_terms: rounded additions in the sum (0: an exact sum).
    addends: |beta * C| + |bias| of each element."""
    n = sum_terms + 4  # the sum, its cast or scale factors (alpha * sb, sa * that), the multiply-add
    e = n * U / (1 - n * U) * mass + 3 * U * (np.abs(z) + addends + mass)
    e = e * tolerance.slope_bound(z, e, act)
    e = e + (tolerance.ACT_REL[act] + U) * np.abs(y)
    if bf16:
        # GELU for BF16 output is evaluated to 2^-16 relative at the far negative end.
        rel = 2.0 ** -8 + (2.0 ** -16 if act in tolerance.ACT_GELU else 0.0)
        e = e * (1 + 2.0 ** -7) + rel * np.abs(y) + 2.0 ** -134
    return e + 2.0 ** -149


def check(out, y, e, what=""):
    out = np.asarray(out, np.float64)
    assert out.shape == y.shape
    bad = ~(np.abs(out - y) <= e)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first {i}: out={out[i]!r} "
                             f"want={y[i]!r} bound={e[i]!r}")
