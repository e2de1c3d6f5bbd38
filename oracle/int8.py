"""INT8 quantisation of rows and the INT8 product. TEST INFRASTRUCTURE ONLY.

    quantise:  scale[m] = float32(max_k |x| / 127) (1 for an all-zero row)
               q = round_half_even(float32(x / scale)) in [-127, 127]
    product:   z = alpha * sa[m] sb[n] * (sum_k (a - za[m]) b) + beta * C + bias[n]

The quantiser's divisions are IEEE float32 divisions (they decide the codes);
the product's sum is an int64 sum and its epilogue is float64. Pinned by
tests/test_oracle_int8.py.
"""
from __future__ import annotations

import numpy as np

from .codecs import decode_bf16
from .gemm import activation


def quantize_rows_int8(x_bits, K: int | None = None):
    """BF16 codes (M x >=K, uint16) -> (int8 codes M x K, scales float32[M])."""
    xb = np.asarray(x_bits)
    K = xb.shape[1] if K is None else K
    x = decode_bf16(xb[:, :K]).astype(np.float32)
    amax = np.abs(x).max(axis=1) if K > 0 else np.zeros(x.shape[0], np.float32)
    scale = np.where(amax > 0, amax / np.float32(127), np.float32(1)).astype(np.float32)
    q = np.rint((x / scale[:, None]).astype(np.float32))
    return np.clip(q, -127, 127).astype(np.int8), scale


def gemm_int8_scaled(a, b, scale_a, zero_a, scale_b, alpha=1.0, beta=0.0, c=None, bias=None, act=0):
    """a: M x K, b: N x K integer codes (K-major); c, bias: values. -> (y, z, |product part|)."""
    a = np.asarray(a, np.int64)
    if zero_a is not None:
        a = a - np.asarray(zero_a, np.int64)[:, None]
    s = a @ np.asarray(b, np.int64).T
    prod = alpha * np.asarray(scale_a, np.float64)[:, None] * np.asarray(scale_b, np.float64) * s
    z = prod.copy()
    if beta != 0.0:
        z = z + beta * np.asarray(c, np.float64)
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    return activation(z, act), z, np.abs(prod)
