"""A shared projection with a low-rank adapter per row. TEST INFRASTRUCTURE ONLY.

Written from the definition in float64, a row at a time. Pinned by tests/test_oracle_routing.py.
"""
from __future__ import annotations

import numpy as np

from .gemm import activation


def lora(a, b, adapter, down, up, scale=None, c=None, alpha=1.0, beta=0.0, bias=None, act=0):
    """a: M x K, b: K x N (logical), down: G x R x K, up: G x N x R, bias: N.

    Returns (y, z, magnitudes): the result, it before the activation, and per element the sum of the
    magnitudes of the main product's terms, of the adapter's (both factors' terms) and of the addends.
    """
    a, b, down, up = (np.asarray(v, np.float64) for v in (a, b, down, up))
    z = alpha * (a @ b)
    main = abs(alpha) * (np.abs(a) @ np.abs(b))
    low = np.zeros_like(z)
    for m, g in enumerate(np.asarray(adapter)):
        if 0 <= g < len(down):
            s = 1.0 if scale is None else float(scale[g])
            z[m] += alpha * (up[g] @ (s * (down[g] @ a[m])))
            low[m] = abs(alpha * s) * (np.abs(up[g]) @ (np.abs(down[g]) @ np.abs(a[m])))
    add = np.zeros_like(z)
    if beta != 0.0:
        add += np.abs(beta * np.asarray(c, np.float64))
        z += beta * np.asarray(c, np.float64)
    if bias is not None:
        add += np.abs(np.asarray(bias, np.float64))
        z += np.asarray(bias, np.float64)
    return activation(z, act), z, (main, low, add)
