"""The INT8 product on 256x256 tiles: FP32 and BF16 output, codes, and sums split along K.

Every test names the tile that its shape is planned on. Sums of INT8 products are exact, and with unit
scales so is every result below 2^24; the 64-bit products are torch's, in float64 on the GPU.
"""
import numpy as np
import pytest
import torch

import dense_gemm_09_amd as g
import oracle
from dense_gemm_09_amd import (ACT_GELU_ERF, ACT_NONE, ACT_RELU, COL, OUT_BF16, OUT_F32, QOUT_E4M3,
                               QOUT_INT8, ROW)
from tests.test_int8_gpu import dev, product

pytestmark = pytest.mark.gpu


def planned(M, N, K, split=1):
    p = g.plan(M, N, K, True)
    assert (p.kernel, p.tile_m, p.tile_n, p.split_k) == (0, 256, 256, split)


def ints(shape, top, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda", dtype=torch.int8)


def exact(a, b, za=None):
    s = a.double() @ b.double().t()
    return s if za is None else s - za.double()[:, None] * b.double().sum(1)


@pytest.mark.parametrize("M,N,K", [(3840, 4096, 201), (4090, 4090, 77), (3841, 4095, 128), (4096, 4096, 1),
                                   (3900, 3900, 640)])
@pytest.mark.parametrize("zero", [False, True])
def test_exact_sums(M, N, K, zero):
    """Whole and partial tiles, K inside and at the end of a slice and of a chunk; padded rows and odd starts."""
    planned(M, N, K)
    print(f"[gpu] int8 wide {M} {N} {K} zero={zero}", flush=True)
    for pad, shift in ((0, 0), (3, 1)):
        a, b = ints((M, K + pad), 9, 1), ints((N, K + pad), 9, 2)
        za = torch.randint(-128, 128, (M,), device="cuda", dtype=torch.int32) if zero else None
        sums = torch.empty(N, dtype=torch.int32, device="cuda") if zero else None
        ad, bd = (torch.zeros(t.numel() + shift, dtype=torch.int8, device="cuda")[shift:] for t in (a, b))
        ad.copy_(a.reshape(-1))
        bd.copy_(b.reshape(-1))
        if zero:
            g.int8_col_sums(K, N, bd, K + pad, sums)
        one = torch.ones(max(M, N), device="cuda")
        want = exact(a[:, :K], b[:, :K], za)
        c = torch.full((M, N + pad), 2.0, device="cuda")
        g.gemm_int8_scaled(M, N, K, 2.0, ad, K + pad, ROW, bd, K + pad, COL, one, za, one, sums, -1.0, c, N + pad,
                           OUT_F32)
        assert torch.equal(c[:, :N].double(), 2 * want - 2)
        assert torch.all(c[:, N:] == 2).item()
        h = torch.full((M, N + pad), 2.0, device="cuda", dtype=torch.bfloat16)
        g.gemm_int8_scaled(M, N, K, 1.0, ad, K + pad, ROW, bd, K + pad, COL, one, za, one, sums, 0.0, h, N + pad,
                           OUT_BF16, None, ACT_RELU)
        assert torch.equal(h[:, :N], want.clamp(min=0).float().to(torch.bfloat16))
        assert torch.all(h[:, N:] == 2).item()


@pytest.mark.parametrize("out", [OUT_F32, OUT_BF16])
@pytest.mark.parametrize("act", [ACT_NONE, ACT_GELU_ERF])
def test_scales_bias_and_activation(out, act):
    planned(3840, 4096, 64)
    product(3840, 4096, 64, out, True, True, act, alpha=0.5, beta=0.0 if act else 0.75, seed=act)


@pytest.mark.parametrize("M,N,K", [(3840, 4096, 201), (4090, 4091, 64)])
@pytest.mark.parametrize("q", [QOUT_INT8, QOUT_E4M3])
def test_codes(M, N, K, q):
    """The quantising epilogue: exact values, so that every code is the definition's."""
    planned(M, N, K)
    print(f"[gpu] int8 wide codes {M} {N} {K} q={q}", flush=True)
    rng = np.random.default_rng(K + q)
    a, b = ints((M, K), 2, 1), ints((N, K), 2, 2)
    one = torch.ones(max(M, N), device="cuda")
    os_ = (2.0 ** rng.integers(-4, 1, M)).astype(np.float32)
    oz = rng.integers(-20, 20, M).astype(np.int32) if q == QOUT_INT8 else None
    za = ints((M,), 3, 3).int()
    sums = b.int().sum(1, dtype=torch.int32)
    out = torch.zeros(M, N, dtype=torch.uint8, device="cuda")
    g.gemm_int8_scaled_quant(M, N, K, 1.0, a, K, ROW, b, K, COL, one, za, one, sums, None, ACT_RELU, dev(os_),
                             None if oz is None else dev(oz), out, N, q)
    y = exact(a, b, za).clamp(min=0).cpu().numpy()
    want = oracle.quantize_output(y, os_, oz, q)
    got = out.cpu().numpy()
    assert np.array_equal(got.view(np.int8).astype(np.int64) if q == QOUT_INT8 else got, want)


def test_split_along_k():
    """A K long enough for two partial sums of 256x256 tiles, whose INT32 partials add exactly."""
    M, N, K = 2048, 4096, 120000
    planned(M, N, K, 2)
    print("[gpu] int8 wide split", flush=True)
    a, b = ints((M, K), 9, 1), ints((N, K), 9, 2)
    za = ints((M,), 9, 3).int()
    one = torch.ones(max(M, N), device="cuda")
    want = exact(a, b, za)
    sums = torch.empty(N, dtype=torch.int32, device="cuda")
    g.int8_col_sums(K, N, b, K, sums)
    c = torch.empty(M, N, device="cuda")
    g.gemm_int8_scaled(M, N, K, 1.0, a, K, ROW, b, K, COL, one, za, one, sums, 0.0, c, N, OUT_F32)
    assert torch.equal(c.double(), want)  # below 2^24
    q = torch.zeros(M, N, dtype=torch.int8, device="cuda")
    scale = torch.full((M,), 2.0 ** -8, device="cuda")
    g.gemm_int8_scaled_quant(M, N, K, 1.0, a, K, ROW, b, K, COL, one, za, one, sums, None, ACT_NONE, scale, None, q, N,
                             QOUT_INT8)
    assert torch.equal(q.double(), (want / 256).round().clamp(-128, 127))
