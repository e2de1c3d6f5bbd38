"""The expert layer of examples/expert_layer.py against 64 bits, expert by expert."""
import pytest
import torch

import dense_gemm_09_amd as g
from examples import expert_layer as layer
from tests import wide

pytestmark = pytest.mark.gpu

T, G, K, N = 700, 5, 256, 384


def problem():
    gen = torch.Generator("cuda").manual_seed(1)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    w, bias = (randn(G, N, K) * 0.1).bfloat16(), (randn(G, N) * 0.1).bfloat16()
    expert = torch.randint(0, G - 1, (T,), device="cuda", generator=gen)  # the last expert stays idle
    x, order, offsets = layer.sort_by_expert(randn(T, K).bfloat16(), expert, G)
    return x, w, bias, expert[order], offsets, randn(T, N).bfloat16()


def bf16_bound(want, terms, mass, extra=0.0):
    """A BF16 rounding, and the FP32 sum of `terms` products of total magnitude `mass`."""
    u = terms * wide.U
    return 2.0 ** -8 * want.abs() + (1 + 2.0 ** -7) * (u / (1 - u) * mass + 3 * wide.U * (mass + extra))


def test_training_step():
    x, w, bias, expert, offsets, dy = problem()
    assert offsets[-1].item() == offsets[-2].item() == T
    dw = torch.ones(G, N, K, device="cuda")
    y, dx = layer.train_step(x, w, bias, offsets, dy, dw)
    X, W, B, D = (t.double().cpu() for t in (x, w, bias, dy))
    e = expert.cpu()
    for i in range(G):
        r = e == i
        want = X[r] @ W[i].T + B[i]
        mass = X[r].abs() @ W[i].abs().T
        assert torch.all((y.double().cpu()[r] - want).abs() <= bf16_bound(want, K + 2, mass, B[i].abs()))
        want, mass = D[r] @ W[i], D[r].abs() @ W[i].abs()
        assert torch.all((dx.double().cpu()[r] - want).abs() <= bf16_bound(want, N + 2, mass))
        want, mass = 1 + D[r].T @ X[r], D[r].T.abs() @ X[r].abs()
        u = (int(r.sum()) + 4) * wide.U
        assert torch.all((dw[i].double().cpu() - want).abs() <= u / (1 - u) * mass + 2 * wide.U * (1 + mass))


def test_serving():
    x, w, bias, expert, offsets, _ = problem()
    wq, ws = layer.quantise_weight(w)
    y = layer.serve(x, wq, ws, bias, offsets, g.ACT_NONE).double().cpu()
    # The codes and scales are checked bit for bit elsewhere: the product of what they stand for.
    xq = torch.empty(T, K, device="cuda", dtype=torch.int8)
    xs = torch.empty(T, device="cuda")
    g.quantize_int8_rows(T, K, x, K, xq, K, xs)
    X, W = (xq.double() * xs[:, None].double()).cpu(), (wq.double() * ws[..., None].double()).cpu()
    for i in range(G):
        r = expert.cpu() == i
        want = X[r] @ W[i].T + bias[i].double().cpu()
        mass = X[r].abs() @ W[i].abs().T
        assert torch.all((y[r] - want).abs() <= bf16_bound(want, 6, mass, bias[i].double().cpu().abs()))
    # and INT8 stays near BF16: each operand's rounding is at most half a step of its row's 127
    full = layer.forward(x, w, bias, offsets).double().cpu()
    assert ((full - y).norm() / full.norm()).item() < 0.02
