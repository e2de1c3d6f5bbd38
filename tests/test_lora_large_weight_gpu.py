"""Few rows with adapters on a weight of 2 GiB and more. Bounds as in tests/test_lora_gpu.py."""
import pytest
import torch

import dense_gemm_09_amd as g

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("M,N,K,R", [(3, (1 << 18) + 5, 4096, 16), (16, (1 << 17) + 3, 8200, 40)])
def test_parity(M, N, K, R):
    G = 3
    gen = torch.Generator("cuda").manual_seed(N)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen, dtype=torch.float32).bfloat16()  # noqa: E731
    a, b, down, up = rand(M, K), rand(N, K), rand(G, R, K), rand(G, N, R)
    assert b.nbytes >= 1 << 31
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % (G + 1)
    c = torch.full((M, N), float("nan"), device="cuda")
    g.gemm_lora_bf16(M, N, K, G, R, 1.0, a, K, b, K, ids, down, K, R * K, up, R, N * R, None, 0.0, c, N, g.OUT_F32)
    A = a.double()
    for n0 in range(0, N, 1 << 15):
        s = slice(n0, min(N, n0 + (1 << 15)))
        bt = b[s].double().t().contiguous()
        z, main, low = A @ bt, A.abs() @ bt.abs(), torch.zeros(M, bt.shape[1], device="cuda", dtype=torch.float64)
        for i in range(G):
            r = ids == i
            d, u = down[i].double().t().contiguous(), up[i, s].double().t().contiguous()
            z[r] += (A[r] @ d) @ u
            low[r] = (A[r].abs() @ d.abs()) @ u.abs()
        n, m = (K + 20) * U, (K + 2 * R + 24) * U
        e = n / (1 - n) * main + (m / (1 - m) + 2.0 ** -16 * (1 + 2.0 ** -7)) * low + 4 * U * (z.abs() + main + low)
        assert ((c[:, s].double() - z).abs() <= e).all(), n0


def test_more_rows_are_refused():
    """17 rows take tiles, whose copies have 32-bit offsets; nothing is enqueued."""
    N, K = 1 << 18, 4096
    b = torch.empty(N, K, device="cuda", dtype=torch.bfloat16)
    a, c = torch.zeros(17, K, device="cuda", dtype=torch.bfloat16), torch.full((17, N), 5.0, device="cuda")
    ids = torch.zeros(17, device="cuda", dtype=torch.int32)
    with pytest.raises(g.GemmError, match="UNSUPPORTED"):
        g.gemm_lora_bf16(17, N, K, 1, 0, 1.0, a, K, b, K, ids, None, K, 0, None, 1, 0, None, 0.0, c, N, g.OUT_F32)
    assert (c == 5).all()
