"""An expert layer on the grouped calls: tokens sorted by expert, one weight per expert.

    python examples/expert_layer.py [--tokens T] [--experts G] [--width K] [--hidden N]

`train_step` is the layer's forward and backward pass in BF16 (the weight
gradient in FP32), `quantise_weight` and `serve` the same layer with INT8 weights
and tokens, scaled per channel and per token. Nothing comes back to the host:
the experts' row ranges stay where the router made them.
"""
import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_09_amd as g  # noqa: E402


def sort_by_expert(x, expert, experts):
    """Rows of x in the order of their expert, that order, and INT32[experts + 1] row offsets."""
    in_order, order = torch.sort(expert, stable=True)
    # (Not bincount, which waits for the GPU to size its result.)
    bounds = torch.arange(experts + 1, device=x.device, dtype=expert.dtype)
    return x[order].contiguous(), order, torch.searchsorted(in_order, bounds, out_int32=True)


def forward(x, w, bias, offsets, act=g.ACT_NONE):
    """y[r] = act(x[r] w[e]^T + bias[e]) for the rows r of each expert e. x: T x K, w: G x N x K."""
    (T, K), (G, N, _) = x.shape, w.shape
    y = torch.empty(T, N, device=x.device, dtype=torch.bfloat16)
    g.gemm_grouped_bf16(G, T, N, K, 1.0, x, K, offsets, w, K, g.COL, N * K, 0.0, y, N, g.OUT_BF16, bias, act)
    return y


def train_step(x, w, bias, offsets, dy, dw):
    """The layer without activation and its gradients: returns y and dx; dw (FP32) is added to.

    dx reads the weights as they are stored, along their other axis.
    """
    (T, K), (G, N, _) = x.shape, w.shape
    y = forward(x, w, bias, offsets)
    dx = torch.empty_like(x)
    g.gemm_grouped_bf16(G, T, K, N, 1.0, dy, N, offsets, w, K, g.ROW, N * K, 0.0, dx, K, g.OUT_BF16)
    g.gemm_grouped_bf16_wgrad(G, T, N, K, 1.0, dy, N, x, K, offsets, 1.0, dw, K, N * K, g.OUT_F32)
    return y, dx


def quantise_weight(w):
    """INT8 codes and one scale per output channel of each expert (once per weight)."""
    G, N, K = w.shape
    q = torch.empty(G, N, K, device=w.device, dtype=torch.int8)
    scale = torch.empty(G, N, device=w.device)
    g.quantize_int8_rows(G * N, K, w, K, q, K, scale)
    return q, scale


def serve(x, wq, w_scale, bias, offsets, act=g.ACT_GELU_ERF):
    """The layer on INT8 weights: tokens are quantised one scale each, products are exact sums."""
    (T, K), (G, N, _) = x.shape, wq.shape
    xq = torch.empty(T, K, device=x.device, dtype=torch.int8)
    x_scale = torch.empty(T, device=x.device)
    g.quantize_int8_rows(T, K, x, K, xq, K, x_scale)
    y = torch.empty(T, N, device=x.device, dtype=torch.bfloat16)
    g.gemm_grouped_int8_scaled(G, T, N, K, 1.0, xq, K, offsets, wq, K, g.COL, N * K, x_scale, None, w_scale, None,
                               0.0, y, N, g.OUT_BF16, bias, act)
    return y


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=4096)
    a = ap.parse_args()
    T, G, K, N = a.tokens, a.experts, a.width, a.hidden
    gen = torch.Generator("cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    w = (randn(G, N, K) * 0.02).to(torch.bfloat16)
    bias = (randn(G, N) * 0.1).to(torch.bfloat16)
    expert = torch.randint(0, G, (T,), device="cuda", generator=gen)
    x, _, offsets = sort_by_expert(randn(T, K).to(torch.bfloat16), expert, G)
    dy = randn(T, N).to(torch.bfloat16)
    dw = torch.zeros(G, N, K, device="cuda")
    wq, w_scale = quantise_weight(w)

    def timed(what, flops, call):
        for _ in range(3):
            call()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(10):
            call()
        end.record()
        torch.cuda.synchronize()
        ms = start.elapsed_time(end) / 10
        print(f"{what}: {ms * 1e3:.1f} us, {flops / ms / 1e9:.0f} TFLOP/s")

    timed("training step (forward, dx, dw), BF16", 6 * T * N * K, lambda: train_step(x, w, bias, offsets, dy, dw))
    timed("serving, INT8 with GELU", 2 * T * N * K, lambda: serve(x, wq, w_scale, bias, offsets))
    a, b = forward(x, w, bias, offsets, g.ACT_GELU_ERF).float(), serve(x, wq, w_scale, bias, offsets).float()
    print(f"INT8 against BF16: relative difference {((a - b).norm() / a.norm()).item():.4f}")


if __name__ == "__main__":
    main()
