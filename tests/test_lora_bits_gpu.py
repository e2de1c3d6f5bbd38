"""FP32 output keeps all bits of the adapters' first products; on every kernel.

`exact`: the first product h of a row is one FP32 number of 24 bits (its BF16 pieces added up, without rounding), the
second factors are powers of two, one rank to a column, and the projection is zero: the output is h times the power
of two, which FP32 holds.
`bound`: every step is FP32: a sum of K terms and a scale, a sum of three terms for each rank, the main product's sum,
alpha, and the output: (K + 3 R + 30) U of the magnitudes of both factors' products, and no term of 2^-16. With K = 8
that is below 2^-16 up to 70 ranks.
"""
import numpy as np
import pytest
import torch

import dense_gemm_09_amd as g
from oracle import lora as oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# Rows: streaming, few rows otherwise (ranks; K), 64-row tiles whole and split, 128x128 tiles, both forms, 256x256.
SHAPES = [(1, 64, 64, 16), (16, 80, 64, 32), (16, 96, 128, 100), (9, 64, 8192, 16), (40, 96, 64, 20),
          (64, 128, 2048, 16), (200, 160, 72, 16), (130, 100, 37, 5), (700, 700, 2048, 33), (4000, 4000, 72, 16)]


def call(a, b, ids, down, up, c, scale=None):
    (M, K), N, (G, R, _) = a.shape, b.shape[0], down.shape
    g.gemm_lora_bf16(M, N, K, G, R, 1.0, a.cuda(), K, b.cuda(), K, ids.cuda(), down.cuda(), K, R * K, up.cuda(), R, N * R,
                     scale, 0.0, c, N, g.OUT_F32)
    return c.cpu()


@pytest.mark.parametrize("M,N,K,R", SHAPES)
def test_exact(M, N, K, R):
    G = 3
    gen = torch.Generator().manual_seed(R)
    h = torch.randn(G, R, generator=gen)
    h = (h.view(torch.int32) | 1).view(torch.float32)  # the last bit is set
    down, rest = torch.zeros(G, R, K), h.clone()
    for k in range(3):
        piece = (rest.view(torch.int32) & -65536).view(torch.float32)
        down[..., k] = piece
        rest = rest - piece
    assert (rest == 0).all()
    a = torch.zeros(M, K)
    a[:, :3] = 1.0
    up = torch.zeros(G, N, R)
    power = 2.0 ** torch.randint(-5, 5, (G, N), generator=gen).float()
    for n in range(N):
        up[:, n, n % R] = power[:, n]
    ids = (torch.arange(M) % (G + 1)).int()
    c = call(a.bfloat16(), torch.zeros(N, K).bfloat16(), ids, down.bfloat16(), up.bfloat16(), torch.empty(M, N, device="cuda"))
    for i in range(G):
        assert torch.equal(c[ids == i], (h[i, torch.arange(N) % R] * power[i]).expand(int((ids == i).sum()), N))
    assert (c[ids == G] == 0).all()


@pytest.mark.parametrize("M,N,R", [(1, 256, 1), (16, 128, 8), (16, 96, 60), (40, 96, 8), (200, 160, 4), (129, 260, 1)])
def test_bound(M, N, R):
    K, G = 8, 4
    gen = torch.Generator().manual_seed(N)
    rand = lambda *s: torch.randn(*s, generator=gen).bfloat16()  # noqa: E731
    a, b, down, up = rand(M, K), (rand(N, K) * 2.0 ** -8), rand(G, R, K), rand(G, N, R)
    scale = torch.rand(G, generator=gen) + 0.5
    ids = (torch.arange(M) % G).int()
    c = call(a, b, ids, down, up, torch.empty(M, N, device="cuda"), scale.cuda()).double().numpy()
    y, z, (main, low, _) = oracle.lora(a.double().numpy(), b.double().numpy().T, ids.numpy(), down.double().numpy(),
                                       up.double().numpy(), scale.numpy())
    e = (K + 3 * R + 30) * U * (main + low)
    assert (np.abs(c - y) <= e).all(), (np.abs(c - y) / e).max()
