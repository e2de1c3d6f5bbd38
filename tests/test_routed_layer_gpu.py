"""Routing, sort, copies, products and weighted sums as one layer; captured and replayed; on other streams.

Tolerances. The layer rounds to BF16 (2^-8) after the products, and after the sums: an output is off by at most
2^-8 of each expert's weighted row, of the sum, the products' FP32 sums and the weights' (k + G + 30) U. Its gradients
follow the same way: each BF16 rounding of an intermediate is 2^-8 of its terms' magnitudes.
"""
import numpy as np
import pytest
import torch

import dense_gemm_09_amd as g
from examples import routed_layer as layer
from oracle import routing as o

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8


def problem(T, G, K, N, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, w = rand(T, K).bfloat16(), (rand(G, N, K) * 0.1).bfloat16()
    logits = rand(T, G)
    logits[:, G - 1] = -float("inf")  # an expert that nobody has
    logits[T // 2] = -float("inf")    # a token of padding
    return x, logits, w, rand(T, N).bfloat16()


@pytest.mark.parametrize("score,renorm", [(o.SOFTMAX, True), (o.SOFTMAX, False), (o.SIGMOID, True)])
@pytest.mark.parametrize("T,G,k,K,N", [(1, 8, 3, 64, 96), (70, 5, 2, 256, 128), (300, 33, 6, 128, 200)])
def test_layer_and_gradients(T, G, k, K, N, score, renorm):
    x, logits, w, dout = problem(T, G, K, N)
    if T == 1:
        logits[0] = torch.randn(G, generator=torch.Generator().manual_seed(1))
    out, saved = layer.forward(x.cuda(), logits.cuda(), w.cuda(), k, None, score, renorm)
    dx, dlogits, dw = (t.double().cpu().numpy() for t in layer.backward(dout.cuda(), saved))
    out = out.double().cpu().numpy()
    X, L, W, D = (t.double().numpy() for t in (x, logits, w, dout))
    want_dx, want_dw = np.zeros_like(X), np.zeros_like(W)
    e_dx, e_dw = np.zeros_like(X), np.zeros_like(W)
    for t in range(T):
        ids = o.choose(L[t], k, score)
        weight = o.weights(L[t], ids, score, renorm, 1.0)
        y = np.array([W[e] @ X[t] if e >= 0 else np.zeros(N) for e in ids])
        mass = np.array([np.abs(W[e]) @ np.abs(X[t]) if e >= 0 else np.zeros(N) for e in ids])
        rel = (K + N + k + G + 60 + 8 * 10) * U
        want = weight @ y
        bound = weight @ (H * np.abs(y) + 2 * rel * mass) * (1 + H) + H * np.abs(want) + 1e-30
        assert (np.abs(out[t] - want) <= bound).all(), t
        # the weights' gradient sees y rounded to BF16
        dweight = y @ D[t]
        e_dweight = (H * np.abs(y) + 2 * rel * mass) @ np.abs(D[t]) + 2 * rel * (np.abs(y) @ np.abs(D[t]))
        want_l = o.grad(L[t], ids, dweight, score, renorm, 1.0)
        # the gradient is linear in dweight: a score or share of at most 1 each, times at most twice the largest
        s = np.zeros(G)
        live = ids >= 0
        e_l = (2 * e_dweight[live].sum() + 4 * rel * np.abs(dweight[live]).sum()) + s + 1e-30
        assert (np.abs(dlogits[t] - want_l) <= e_l).all(), t
        for j, e in enumerate(ids):
            if e < 0:
                continue
            dy = weight[j] * D[t]  # rounded to BF16, then two products
            want_dx[t] += dy @ W[e]
            e_dx[t] += (2 * H + 2 * rel) * (np.abs(dy) @ np.abs(W[e])) * (1 + H)
            want_dw[e] += np.outer(dy, X[t])
            e_dw[e] += (H + (T + 60) * U + 2 * rel) * np.abs(np.outer(dy, X[t]))
    assert (np.abs(dx - want_dx) <= e_dx + H * np.abs(want_dx) + 1e-30).all()
    assert (np.abs(dw - want_dw) <= e_dw + 1e-30).all()


def test_gradient_against_differences():
    """d sum(out * dout) / d logits, by central differences of the layer's own forward pass with FP64 sums of its BF16
    outputs: the outputs' rounding over the step is the bound, and h^2 / 6 of a third derivative below 6 each."""
    T, G, k, K, N = 4, 6, 3, 32, 16
    x, logits, w, dout = problem(T, G, K, N, 3)
    logits[T // 2], logits[:, G - 1] = 0.3, -9.0
    logits[T // 2, 0] = 1.0
    f = lambda l: layer.forward(x.cuda(), l.cuda(), w.cuda(), k)  # noqa: E731
    out, saved = f(logits)
    _, dlogits, _ = layer.backward(dout.cuda(), saved)
    dlogits = dlogits.cpu().double()
    y = saved[1].double().cpu()
    h = 2.0 ** -4
    size = (out.double().cpu().abs() * dout.double().abs()).sum(1)
    mass = y.abs().max() * dout.double().abs().sum(1)
    for e in range(G):
        up, down = logits.clone(), logits.clone()
        up[:, e] += h
        down[:, e] -= h
        (a, sa), (b, sb) = f(up), f(down)
        diff = ((a.double().cpu() - b.double().cpu()) * dout.double()).sum(1) / (2 * h)
        for t in range(T):
            if sorted(sa[3][t].tolist()) == sorted(sb[3][t].tolist()) == sorted(saved[3][t].tolist()):
                bound = 2 * H * size[t] / h + mass[t] * h * h + 2 * H * mass[t]
                assert (diff[t] - dlogits[t, e]).abs() <= bound, (t, e)


def test_captured_and_replayed():
    """Forward and backward in one graph, replayed with other inputs between eager work; nothing is synchronised."""
    T, G, k, K, N = 130, 9, 4, 128, 64
    x, logits, w, dout = (t.cuda() for t in problem(T, G, K, N))
    layer.backward(dout, layer.forward(x, logits, w, k)[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, saved = layer.forward(x, logits, w, k)
        grads = layer.backward(dout, saved)
    for i in range(4):
        fresh = [t.cuda() for t in problem(T, G, K, N, 10 + i)]
        for dst, src in zip((x, logits, w, dout), fresh):
            dst.copy_(src)
        graph.replay()
        want, kept = layer.forward(*fresh[:3], k)
        expected = layer.backward(fresh[3], kept)
        live = int(kept[6][-1])
        assert torch.equal(saved[6], kept[6]) and torch.equal(saved[5], kept[5])
        assert torch.equal(saved[0][:live], kept[0][:live])
        assert torch.equal(out, want)
        assert all(torch.equal(a, b) for a, b in zip(grads, expected))


@pytest.mark.parametrize("M", [9, 40, 300])
def test_adapters_captured_and_replayed(M):
    N, K, G, R = 512, 1024, 7, 16
    gen = torch.Generator("cuda").manual_seed(M)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    a, b, down, up = rand(M, K), rand(N, K), rand(G, R, K), rand(G, N, R)
    ids = torch.zeros(M, device="cuda", dtype=torch.int32)
    c = torch.empty(M, N, device="cuda")

    def run(c):
        g.gemm_lora_bf16(M, N, K, G, R, 1.0, a, K, b, K, ids, down, K, R * K, up, R, N * R, None, 0.0, c, N, g.OUT_F32)
        return c
    run(c)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(c)
    for i in range(4):
        ids.copy_(torch.randint(-1, G, (M,), device="cuda", generator=gen, dtype=torch.int32))
        a.copy_(rand(M, K))
        graph.replay()
        assert torch.equal(c, run(torch.empty_like(c)))


def test_two_streams_at_once():
    """Calls with workspaces of their own, on two streams together, as on one."""
    T, G, k = 20000, 64, 4
    gen = torch.Generator("cuda").manual_seed(0)
    ids = [torch.randint(0, G, (T, k), device="cuda", generator=gen, dtype=torch.int32) for _ in range(2)]
    a = torch.randn(64, 2048, device="cuda", generator=gen).bfloat16()
    b = torch.randn(1024, 2048, device="cuda", generator=gen).bfloat16()
    down = torch.randn(8, 16, 2048, device="cuda", generator=gen).bfloat16()
    up = torch.randn(8, 1024, 16, device="cuda", generator=gen).bfloat16()
    row = (torch.arange(64, device="cuda") % 8).int()

    def run(i, stream=None):
        off = torch.empty(G + 1, device="cuda", dtype=torch.int32)
        pos, order = torch.empty_like(ids[i]), torch.empty_like(ids[i])
        c = torch.empty(64, 1024, device="cuda")
        torch.cuda.synchronize()
        g.route_order(T * k, G, ids[i], off, pos, order, stream=stream)
        g.gemm_lora_bf16(64, 1024, 2048, 8, 16, 1.0, a, 2048, b, 2048, row, down, 2048, 16 * 2048, up, 16, 1024 * 16,
                         None, 0.0, c, 1024, g.OUT_F32, stream=stream)
        return off, pos, order, c
    want = [run(0), run(1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [run(i, s) for i, s in enumerate(streams)]
        torch.cuda.synchronize()
        for w, v in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(w, v))


def test_a_host_workspace_is_refused():
    ids = torch.zeros(100000, device="cuda", dtype=torch.int32)
    with pytest.raises(ValueError, match="workspace must be a device tensor"):
        g.route_order(100000, 4, ids, torch.empty(5, device="cuda", dtype=torch.int32), torch.empty_like(ids), None,
                      torch.empty(1 << 20, dtype=torch.uint8))
