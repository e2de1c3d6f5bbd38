"""Products grouped by rows, and their weight gradient. TEST INFRASTRUCTURE ONLY.

Written from the definition, one group and one matrix product at a time, in
float64 on decoded values. Pinned by tests/test_oracle_int8.py (integer
operands against a sum written out per element, and the weight gradient
against central differences of the forward product).
"""
from __future__ import annotations

import numpy as np

from .gemm import activation


def grouped(a, offsets, b, c, alpha=1.0, beta=0.0, scale_a=None, scale_b=None, bias=None, act=0):
    """a: T x K; b: G x K x N (logical); c: T x N, rows outside every group kept.

    Returns (y, z, |products summed| of each element, rows written as a mask).
    """
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    y = np.array(c, np.float64)
    z, mass = np.zeros_like(y), np.zeros_like(y)
    written = np.zeros(y.shape[0], bool)
    for g in range(len(offsets) - 1):
        r = slice(int(offsets[g]), int(offsets[g + 1]))
        s, m = a[r] @ b[g], np.abs(a[r]) @ np.abs(b[g])
        f = alpha * np.ones_like(s)
        if scale_a is not None:
            f = f * np.asarray(scale_a, np.float64)[r, None] * np.asarray(scale_b, np.float64)[g]
        t = f * s
        if beta != 0.0:
            t = t + beta * y[r]
        if bias is not None:
            t = t + np.asarray(bias, np.float64)[g]
        z[r], mass[r], y[r], written[r] = t, np.abs(f) * m, activation(t, act), True
    return y, z, mass, written


def wgrad(d, x, offsets, c, alpha=1.0, beta=0.0):
    """d: T x N, x: T x K, c: G x N x K -> (gradients, |products summed| of each element)."""
    d, x = np.asarray(d, np.float64), np.asarray(x, np.float64)
    out = beta * np.asarray(c, np.float64) if beta != 0.0 else np.zeros(np.shape(c))
    mass = np.zeros_like(out)
    for g in range(len(offsets) - 1):
        r = slice(int(offsets[g]), int(offsets[g + 1]))
        out[g] += alpha * (d[r].T @ x[r])
        mass[g] = abs(alpha) * (np.abs(d[r]).T @ np.abs(x[r]))
    return out, mass
