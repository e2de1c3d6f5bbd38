"""The projection with adapters on every tile that its plans have, each with its plan asserted, and more ranks than the
streaming kernel holds. Bounds: tests/test_lora_gpu.py; the 64-bit products of the larger problems run on the GPU."""
import numpy as np
import pytest
import torch

import dense_gemm_09_amd as g
from tests.test_lora_gpu import bound, problem, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,R", [(8, 300, 1024, 64), (16, 256, 512, 128), (1, 96, 4096, 40), (13, 200, 72, 33),
                                     (16, 4200, 256, 100), (5, 8208, 512, 32), (16, 4100, 64, 17)])
def test_few_rows(M, N, K, R):
    assert g.plan(M, N, K, False).kernel == 1
    for kind in ("mixed", "one"):
        problem(M, N, K, 9, R, rows_of(M, 9, kind, N), act=2, beta=0.5)


def big(M, N, K, G, R, out, tile, split):
    p = g.plan(M, N, K, False)
    assert (p.tile_m, p.tile_n, p.split_k) == (*tile, split)
    gen = torch.Generator("cuda").manual_seed(M + K)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    a, b = rand(M, K).bfloat16(), (rand(N, K) * 0.05).bfloat16()
    down, up = (rand(G, R, K) * 0.05).bfloat16(), (rand(G, N, R) * 0.3).bfloat16()
    ids = torch.randint(-1, G, (M,), device="cuda", generator=gen, dtype=torch.int32)
    ids[: M // 2] = ids[: M // 2].sort().values
    c = torch.full((M, N), float("nan"), device="cuda", dtype=torch.float32 if out == "f32" else torch.bfloat16)
    g.gemm_lora_bf16(M, N, K, G, R, 1.0, a, K, b, K, ids, down, K, R * K, up, R, N * R, None, 0.0, c, N,
                     g.OUT_F32 if out == "f32" else g.OUT_BF16)
    A, B = a.double(), b.double().t().contiguous()
    z, main = A @ B, A.abs() @ B.abs()
    low = torch.zeros_like(z)
    for i in range(G):
        r = (ids == i).nonzero()[:, 0]
        d, u = down[i].double().t().contiguous(), up[i].double().t().contiguous()
        z[r] += (A[r] @ d) @ u
        low[r] = (A[r].abs() @ d.abs()) @ u.abs()
    z, main, low = (t.cpu().numpy() for t in (z, main, low))
    e = bound(z, z, (main, low, np.zeros_like(z)), K, R, 0, out == "bf16")
    assert (np.abs(c.double().cpu().numpy() - z) <= e).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,R,tile,split", [
    (4000, 4000, 72, 16, (256, 256), 1), (4000, 4000, 70, 40, (256, 256), 1), (2100, 2300, 72, 16, (128, 128), 1),
    (2100, 2300, 69, 100, (128, 128), 1), (777, 1000, 4099, 20, (128, 128), 8), (1024, 4096, 4096, 16, (128, 128), 2),
    (777, 4093, 2047, 24, (128, 128), 1), (2048, 4096, 14336, 16, (256, 256), 2), (100, 512, 2048, 64, (256, 128), 16),
    (100, 512, 2046, 3, (256, 128), 16), (64, 4096, 4096, 64, (64, 128), 8), (50, 18432, 4096, 16, (64, 256), 3)])
def test_tiles(M, N, K, R, tile, split, out):
    big(M, N, K, 11, R, out, tile, split)
