"""Sorting tokens by expert, and the layer on it, without a synchronisation."""
import pytest
import torch

from examples import expert_layer as layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 5), (1000, 7), (513, 130)])
def test_nothing_comes_back_to_the_host(T, G, dtype):
    gen = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, 64, device="cuda", generator=gen).bfloat16()
    w = torch.randn(G, 32, 64, device="cuda", generator=gen).bfloat16()
    bias = torch.zeros(G, 32, device="cuda").bfloat16()
    expert = torch.randint(0, max(1, G - 1), (T,), device="cuda", generator=gen).to(dtype)
    torch.cuda.synchronize()
    torch.cuda.set_sync_debug_mode("error")
    try:
        xs, order, offsets = layer.sort_by_expert(x, expert, G)
        layer.forward(xs, w, bias, offsets)
    finally:
        torch.cuda.set_sync_debug_mode("default")
    assert offsets.dtype == torch.int32
    assert offsets.tolist() == [0, *torch.bincount(expert, minlength=G).cumsum(0).tolist()]
    assert torch.equal(xs, x[order])
    e = expert[order].tolist()
    assert e == sorted(e)
    assert all(order[i] < order[i + 1] for i in range(T - 1) if e[i] == e[i + 1])
