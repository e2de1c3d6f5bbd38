"""Infinite second factors and first products at the end of FP32's range, against the definition.

An infinite factor times a finite h is an infinity with the sign of both; infinities of both signs in one sum, and zero
times an infinity, are NaN. Which elements are infinite, of which sign, or NaN has to be as the definition says; the
others are within the bounds of tests/test_lora_gpu.py.
"""
import numpy as np
import pytest
import torch

import dense_gemm_09_amd as g
from oracle import lora as oracle
from tests.test_lora_gpu import bound

pytestmark = pytest.mark.gpu

INF = float("inf")
# Rows: on the streaming kernel, on the other one for few rows (K above 4096 or more than 32 ranks), on 64-row tiles
# with and without a split K, on 128x128 tiles.
SHAPES = [(3, 96, 64, 8), (16, 80, 64, 40), (5, 64, 8192, 16), (40, 96, 64, 20), (64, 128, 2048, 16),
          (200, 160, 72, 16), (130, 100, 37, 5), (700, 700, 2048, 33)]


def run(a, b, ids, down, up, out):
    (M, K), N, (G, R, _) = a.shape, b.shape[0], down.shape
    c = torch.empty(M, N, device="cuda", dtype=torch.float32 if out == "f32" else torch.bfloat16)
    dev = lambda t: t.cuda()  # noqa: E731
    g.gemm_lora_bf16(M, N, K, G, R, 1.0, dev(a), K, dev(b), K, torch.from_numpy(ids).cuda(), dev(down), K, R * K, dev(up),
                     R, N * R, None, 0.0, c, N, g.OUT_F32 if out == "f32" else g.OUT_BF16)
    return c.cpu().double().numpy()


def check(a, b, ids, down, up, out):
    got = run(a, b, ids, down, up, out)
    with np.errstate(invalid="ignore", over="ignore"):
        y, z, mags = oracle.lora(*(t.double().numpy() for t in (a, b.t())), ids, down.double().numpy(), up.double().numpy())
        e = bound(y, z, mags, a.shape[1], down.shape[1], 0, out == "bf16")
    assert (np.isnan(got) == np.isnan(y)).all()
    assert ((got == INF) == (y == INF)).all() and ((got == -INF) == (y == -INF)).all()
    finite = np.isfinite(y)
    assert (np.abs(got[finite] - y[finite]) <= e[finite]).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("exact", [False, True])
@pytest.mark.parametrize("M,N,K,R", SHAPES)
def test_infinite_second_factors(M, N, K, R, exact, out):
    """exact: every h is a small integer, so that the rest of it past BF16's bits is zero."""
    G = 3
    gen = torch.Generator().manual_seed(M + R)
    small = lambda *s: torch.randint(1, 4, s, generator=gen).bfloat16()  # noqa: E731
    rand = lambda *s: torch.randn(*s, generator=gen).bfloat16()  # noqa: E731
    if exact:
        a, down = torch.zeros(M, K).bfloat16(), torch.zeros(G, R, K).bfloat16()
        a[:, 0], down[:, :, 0] = small(M), small(G, R)
        down[:, ::2] *= -1
        down[1, R // 2] = 0
    else:
        a, down = rand(M, K), rand(G, R, K)
    b, up = rand(N, K), rand(G, N, R)
    up[0, ::5, R - 1] = INF
    up[0, 1::5, 0] = -INF
    up[0, 2::10, :2] = INF        # with factors of both signs: NaN where the two h differ in sign
    up[1, 3::7, R // 2] = INF     # exact: zero times an infinity
    up[1, 4::7, 1] = float("nan")
    check(a, b, (np.arange(M) % (G + 1)).astype(np.int32), down, up, out)


@pytest.mark.parametrize("M,N,K,R", SHAPES)
def test_first_products_that_are_infinite(M, N, K, R):
    gen = torch.Generator().manual_seed(M)
    rand = lambda *s: torch.randn(*s, generator=gen).bfloat16()  # noqa: E731
    a, b, down, up = rand(M, K), rand(N, K), rand(2, R, K), rand(2, N, R)
    a[:, 0] = 1.0
    down[0, 1, 0] = -INF
    up[0, 5] = INF
    up[0, 6] = -INF
    check(a, b, (np.arange(M) % 3).astype(np.int32), down, up, "f32")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,R", [s for s in SHAPES])
def test_first_products_at_the_end_of_the_range(M, N, K, R, out):
    """h = 3.3996e38 is finite in FP32, and would be infinite if it were rounded to BF16."""
    a, b = torch.zeros(M, K).bfloat16(), torch.zeros(N, K).bfloat16()
    down, up = torch.zeros(1, R, K).bfloat16(), torch.zeros(1, N, R).bfloat16()
    a[:, :2] = 1.0
    down[0, R - 1, 0], down[0, R - 1, 1] = torch.finfo(torch.bfloat16).max, 1e36
    up[0, :, R - 1] = torch.randn(N, generator=torch.Generator().manual_seed(0)).bfloat16() * 2.0 ** -6
    check(a, b, np.zeros(M, np.int32), down, up, out)
