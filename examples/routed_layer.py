"""An expert layer from its router on: choice, sort, copies, products, weighted sum, and the way back.

    python examples/routed_layer.py [--tokens T] [--experts G] [--top-k K] [--width N] [--hidden H]

A token's output is the weighted sum of its experts' (y_e = x w_e^T). `forward` keeps what `backward` needs;
nothing comes back to the host, and both can be captured into a graph.
"""
import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_09_amd as g  # noqa: E402


def forward(x, logits, w, top_k, bias=None, score=g.SCORE_SOFTMAX, renormalise=True):
    """x: T x K (BF16), logits: T x G (FP32), w: G x N x K (BF16) -> T x N (BF16) and what backward needs."""
    (T, K), (G, N, _) = x.shape, w.shape
    R = T * top_k
    new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, device=x.device, dtype=dtype)  # noqa: E731
    expert, position = new(T, top_k, dtype=torch.int32), new(T, top_k, dtype=torch.int32)
    weight, offsets = new(T, top_k, dtype=torch.float32), new(G + 1, dtype=torch.int32)
    g.route(T, G, top_k, logits, G, g.OUT_F32, score, bias, 1, 1, 1, renormalise, 1.0, expert, weight)
    g.route_order(R, G, expert, offsets, position)
    rows, y, out = new(R, K), new(R, N), new(T, N)
    g.dispatch_rows(T, top_k, R, K, x, K, 2, position, rows, K)
    g.gemm_grouped_bf16(G, R, N, K, 1.0, rows, K, offsets, w, K, g.COL, N * K, 0.0, y, N, g.OUT_BF16)
    g.combine_rows(T, top_k, R, N, y, N, g.OUT_BF16, position, weight, 0.0, out, N, g.OUT_BF16)
    return out, (rows, y, logits, expert, weight, position, offsets, w, top_k, score, renormalise)


def backward(dout, saved):
    """Gradients of x (BF16), logits (FP32) and w (FP32) for the output's gradient (T x N, BF16)."""
    rows, y, logits, expert, weight, position, offsets, w, top_k, score, renormalise = saved
    (R, K), (G, N, _), T = rows.shape, w.shape, logits.shape[0]
    new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, device=rows.device, dtype=dtype)  # noqa: E731
    dy, dweight, dlogits = new(R, N), new(T, top_k, dtype=torch.float32), torch.empty_like(logits)
    g.combine_rows_grad(T, top_k, R, N, dout, N, g.OUT_BF16, y, N, g.OUT_BF16, position, weight, dy, N, dweight)
    g.route_grad(T, G, top_k, logits, G, g.OUT_F32, score, renormalise, 1.0, expert, dweight, dlogits, G)
    drows, dx, dw = new(R, K), new(T, K), new(G, N, K, dtype=torch.float32)
    g.gemm_grouped_bf16(G, R, K, N, 1.0, dy, N, offsets, w, K, g.ROW, N * K, 0.0, drows, K, g.OUT_BF16)
    g.gemm_grouped_bf16_wgrad(G, R, N, K, 1.0, dy, N, rows, K, offsets, 0.0, dw, K, N * K, g.OUT_F32)
    g.combine_rows(T, top_k, R, K, drows, K, g.OUT_BF16, position, None, 0.0, dx, K, g.OUT_BF16)
    return dx, dlogits, dw


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=2)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=4096)
    a = ap.parse_args()
    gen = torch.Generator("cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, w = randn(a.tokens, a.width).bfloat16(), (randn(a.experts, a.hidden, a.width) * 0.02).bfloat16()
    logits, dout = randn(a.tokens, a.experts), randn(a.tokens, a.hidden).bfloat16()

    def step():
        return backward(dout, forward(x, logits, w, a.top_k)[1])
    for _ in range(3):
        step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        step()
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) * 100
    flops = 6 * a.tokens * a.top_k * a.hidden * a.width
    print(f"forward and backward: {us:.1f} us, {flops / us / 1e6:.0f} TFLOP/s of products")


if __name__ == "__main__":
    main()
