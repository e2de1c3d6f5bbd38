"""The projection with adapters at so many columns that a workgroup for every 16 of them is more than a launch may have."""
import pytest
import torch

import dense_gemm_09_amd as g

pytestmark = pytest.mark.gpu


def test_more_columns_than_workgroups_of_a_launch():
    """2^26 columns and more, more ranks than the streaming kernel holds: K + 2 R + 24 roundings of 2^-24 and h's 2^-16
    of the adapter's magnitudes, as in tests/test_lora_gpu.py."""
    M, N, K, R = 2, (1 << 26) + 21, 8, 33
    gen = torch.Generator("cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen, dtype=torch.float32).bfloat16()  # noqa: E731
    a, b, down, up = rand(M, K), rand(N, K), rand(1, R, K), rand(1, N, R)
    ids = torch.tensor([0, -1], device="cuda", dtype=torch.int32)
    c = torch.full((M, N), float("nan"), device="cuda")
    g.gemm_lora_bf16(M, N, K, 1, R, 1.0, a, K, b, K, ids, down, K, R * K, up, R, N * R, None, 0.0, c, N, g.OUT_F32)
    h = a[:1].double() @ down[0].double().t()
    low = a[:1].double().abs() @ down[0].double().abs().t()
    U = 2.0 ** -24
    for n0 in range(0, N, 1 << 23):
        s = slice(n0, min(N, n0 + (1 << 23)))
        bt, ut = b[s].double().t().contiguous(), up[0, s].double().t().contiguous()
        z, main = a.double() @ bt, a.double().abs() @ bt.abs()
        z[:1] += h @ ut
        small = torch.zeros_like(z)
        small[:1] = low @ ut.abs()
        e = (K + 24) * U * (main + small) + ((K + 2 * R + 24) * U + 2.0 ** -16 * (1 + 2.0 ** -7)) * small + 2.0 ** -140
        assert ((c[:, s].double() - z).abs() <= e).all(), n0
