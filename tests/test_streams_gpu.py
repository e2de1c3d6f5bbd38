"""Routing, rows and adapters on two streams whose work overlaps: nothing is synchronised between the calls.

Each stream has inputs and outputs of its own, and the calls allocate their workspaces, all of which the calls of both
streams use in turn. Calls are many, and the first ones of each stream large, so that both streams have work queued
while the other's runs."""
import pytest
import torch

import dense_gemm_09_amd as g

pytestmark = pytest.mark.gpu

T, E, K_TOP, N = 30000, 96, 4, 512
M, LN, LK, G, R = 64, 1024, 4096, 8, 16


class Work:
    """Inputs of one stream, and fresh outputs for every repetition."""

    def __init__(self, seed, repeats):
        gen = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.logits, self.bias = rand(T, E), rand(E) * 0.1
        self.x = rand(T, N).bfloat16()
        self.a, self.b = rand(M, LK).bfloat16(), rand(LN, LK).bfloat16()
        self.down, self.up = rand(G, R, LK).bfloat16(), rand(G, LN, R).bfloat16()
        self.row = torch.randint(-1, G, (M,), device="cuda", generator=gen, dtype=torch.int32)
        self.out = [self.outputs() for _ in range(repeats)]

    @staticmethod
    def outputs():
        i32 = lambda *s: torch.full(s, -7, device="cuda", dtype=torch.int32)  # noqa: E731
        return dict(expert=i32(T, K_TOP), weight=torch.zeros(T, K_TOP, device="cuda"), offsets=i32(E + 1),
                    position=i32(T, K_TOP), order=i32(T * K_TOP),
                    rows=torch.zeros(T * K_TOP, N, device="cuda", dtype=torch.bfloat16),
                    drows=torch.zeros(T * K_TOP, N, device="cuda", dtype=torch.bfloat16),
                    back=torch.zeros(T, N, device="cuda"), dweight=torch.zeros(T, K_TOP, device="cuda"),
                    dlogits=torch.zeros(T, E, device="cuda"), c=torch.zeros(M, LN, device="cuda"))

    def enqueue(self, o, stream=None):
        S = T * K_TOP
        g.route(T, E, K_TOP, self.logits, E, g.OUT_F32, g.SCORE_SIGMOID, self.bias, 8, 4, 2, True, 1.0, o["expert"],
                o["weight"], stream=stream)
        g.gemm_lora_bf16(M, LN, LK, G, R, 1.0, self.a, LK, self.b, LK, self.row, self.down, LK, R * LK, self.up, R,
                         LN * R, None, 0.0, o["c"], LN, g.OUT_F32, stream=stream)
        g.route_order(S, E, o["expert"], o["offsets"], o["position"], o["order"], stream=stream)
        g.dispatch_rows(T, K_TOP, S, N, self.x, N, 2, o["position"], o["rows"], N, stream=stream)
        g.combine_rows(T, K_TOP, S, N, o["rows"], N, g.OUT_BF16, o["position"], o["weight"], 0.0, o["back"], N,
                       g.OUT_F32, stream=stream)
        g.combine_rows_grad(T, K_TOP, S, N, o["back"], N, g.OUT_F32, o["rows"], N, g.OUT_BF16, o["position"],
                            o["weight"], o["drows"], N, o["dweight"], stream=stream)
        g.route_grad(T, E, K_TOP, self.logits, E, g.OUT_F32, g.SCORE_SIGMOID, True, 1.0, o["expert"], o["dweight"],
                     o["dlogits"], E, stream=stream)


def test_overlapping_streams():
    repeats = 6
    works = [Work(1, repeats), Work(2, repeats)]
    want = []
    for w in works:
        o = w.outputs()
        w.enqueue(o)
        torch.cuda.synchronize()
        want.append(o)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    # Events on either stream show that neither was done when the other had begun.
    begin, end = ([torch.cuda.Event(enable_timing=True) for _ in streams] for _ in range(2))
    for e, s in zip(begin, streams):
        e.record(s)
    for i in range(repeats):
        for w, s in zip(works, streams):
            w.enqueue(w.out[i], s)
    for e, s in zip(end, streams):
        e.record(s)
    torch.cuda.synchronize()
    assert begin[0].elapsed_time(end[1]) > 0 and begin[1].elapsed_time(end[0]) > 0
    for w, expected in zip(works, want):
        for o in w.out:
            for name, t in o.items():
                assert torch.equal(t, expected[name]), name


def test_overlapping_graphs():
    """Two captured runs, whose workspaces come from their graphs' pools, replayed on two streams together."""
    works = [Work(3, 1), Work(4, 1)]
    want, graphs = [], []
    for w in works:
        o = w.outputs()
        w.enqueue(o)
        torch.cuda.synchronize()
        want.append(o)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.enqueue(w.out[0])
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for w in works:
            for t in w.out[0].values():
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for w, expected in zip(works, want):
            for name, t in w.out[0].items():
                assert torch.equal(t, expected[name]), name
