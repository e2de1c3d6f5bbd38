"""Pins of the oracle's INT8 quantiser and product, of the grouped product and of its weight gradient."""
import numpy as np
import pytest

import oracle
import synth
from oracle import grouped as og
from oracle import int8 as oi


def test_quantiser_closed_forms_and_ties():
    # amax 127: scale exactly 1, codes are RNE of the values themselves (ties to even).
    x = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 3.25, -126.5, 0.0]])
    q, s = oi.quantize_rows_int8(synth.to_bf16_bits(x))
    assert s[0] == 1.0
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, 3, -126, 0]
    q, s = oi.quantize_rows_int8(synth.to_bf16_bits(np.zeros((2, 5))))
    assert np.all(s == 1.0) and np.all(q == 0)
    x = synth.normal((20, 333), 3.0, 0xD10000)
    bits = synth.to_bf16_bits(x)
    q, s = oi.quantize_rows_int8(bits)
    v = oracle.decode_bf16(bits)
    # Half a step, and the quotient's own rounding (2^-24 of at most 127).
    assert np.all(np.abs(q * s[:, None].astype(np.float64) - v) <= s[:, None] * (0.5 + 2e-5))
    assert np.all(np.abs(q).max(axis=1) == 127)


def test_int8_product_against_the_written_out_sum():
    rng = np.random.default_rng(1)
    a, b = rng.integers(-128, 128, (3, 7)), rng.integers(-128, 128, (4, 7))
    sa, sb, za = rng.random(3), rng.random(4), np.array([0, -128, 100])
    y, _, _ = oi.gemm_int8_scaled(a, b, sa, za, sb, alpha=2.0, beta=3.0, c=np.ones((3, 4)),
                                  bias=np.arange(4.0))
    for m in range(3):
        for n in range(4):
            s = sum((int(a[m, k]) - int(za[m])) * int(b[n, k]) for k in range(7))
            assert y[m, n] == pytest.approx(2.0 * sa[m] * sb[n] * s + 3.0 + n, rel=1e-14)


def test_grouped_product_and_gradient():
    rng = np.random.default_rng(2)
    off = [1, 3, 3, 6]  # row 0 and row 6 in no group, group 1 empty
    a, b = rng.integers(-4, 5, (7, 3)), rng.integers(-4, 5, (3, 3, 5))
    c = rng.integers(-4, 5, (7, 5)).astype(float)
    y, _, _, written = og.grouped(a, off, b, c, alpha=2.0, beta=-1.0)
    assert written.tolist() == [False, True, True, True, True, True, False]
    owner = [None, 0, 0, 2, 2, 2, None]
    for r, g in enumerate(owner):
        for n in range(5):
            want = c[r, n] if g is None else 2 * sum(a[r, k] * b[g, k, n] for k in range(3)) - c[r, n]
            assert y[r, n] == want
    # The gradient of sum(D * Y) with respect to a weight W[n, k] = b[k, n], by differences
    # (exact: the product is linear in the weight).
    d = rng.integers(-4, 5, (7, 5)).astype(float)
    dw, _ = og.wgrad(d, a, off, np.zeros((3, 5, 3)))

    def loss(b):
        out, _, _, w = og.grouped(a, off, b, np.zeros((7, 5)))
        return float((d * out)[w].sum())

    for g in range(3):
        for n in range(5):
            for k in range(3):
                up, down = b.astype(float), b.astype(float)
                up[g, k, n] += 0.5
                down[g, k, n] -= 0.5
                assert dw[g, n, k] == loss(up) - loss(down)
    acc, _ = og.wgrad(d, a, off, np.ones((3, 5, 3)), alpha=2.0, beta=3.0)
    assert np.array_equal(acc, 2 * dw + 3)
