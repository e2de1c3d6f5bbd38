"""Grouped products, weight gradients and INT8 products with more tiles than workgroups.

Each workgroup then takes several tiles as one stream of K slices: tiles of one
slice and of many, an odd number of slices, K ending inside a 16-byte chunk,
partial rows and columns, empty groups between full ones. Operands are small
integers, so that every sum is exact in any order.
"""
import numpy as np
import pytest
import torch

import dense_gemm_09_amd as g
import oracle
import synth
from dense_gemm_09_amd import ACT_GELU_ERF, ACT_NONE, ACT_RELU, COL, OUT_BF16, OUT_F32, ROW
from oracle import grouped as og
from oracle import int8 as oi
from tests import wide

pytestmark = pytest.mark.gpu

SIZES = [1500, 0, 257, 2200, 1, 0, 2043]  # 26 row tiles of 256


def dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def offsets(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


def ints(shape, top, seed):
    return np.random.default_rng(seed).integers(-top, top + 1, shape)


def bits(x):
    return synth.to_bf16_bits(x.astype(np.float64))


def check_exact(got, want, what):
    bad = got != want
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} differ, first at {tuple(np.argwhere(bad)[0])}"


@pytest.mark.parametrize("layout", [COL, ROW])
@pytest.mark.parametrize("N,K", [(4096, 8), (3900, 77), (3841, 200), (4096, 320)])
def test_bf16(N, K, layout):
    print(f"[gpu] stream bf16 N={N} K={K} layout={layout}", flush=True)
    G, T, off = len(SIZES), sum(SIZES), offsets(SIZES)
    x, w = ints((T, K), 3, K), ints((G, N, K), 3, K + 1)
    y = np.zeros((T, N))
    for i in range(G):
        y[off[i]:off[i + 1]] = x[off[i]:off[i + 1]].astype(np.float64) @ w[i].T.astype(np.float64)
    wd = dev(bits(w if layout == COL else w.transpose(0, 2, 1)))
    ld = K if layout == COL else N
    xd, od = dev(bits(x)), dev(off)
    c = torch.full((T, N), 2.0, device="cuda")
    g.gemm_grouped_bf16(G, T, N, K, 2.0, xd, K, od, wd, ld, layout, N * K, -1.0, c, N, OUT_F32)
    check_exact(c.cpu().numpy(), 2 * y - 2, "alpha and beta, FP32")
    b = ints((G, N), 5, 9)
    cb = torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
    g.gemm_grouped_bf16(G, T, N, K, 1.0, xd, K, od, wd, ld, layout, N * K, 0.0, cb, N, OUT_BF16,
                        dev(bits(b)), ACT_RELU)
    want = y + b[np.repeat(np.arange(G), SIZES)]
    want = torch.from_numpy(np.maximum(want, 0)).to(torch.bfloat16)  # integers below 2^24: one rounding
    check_exact(cb.cpu().float().numpy(), want.float().numpy(), "bias and ReLU, BF16")


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("N,K", [(4096, 16), (3900, 131), (4096, 384)])
def test_8bit_scales_and_bias(N, K, kind):
    print(f"[gpu] stream {kind} N={N} K={K}", flush=True)
    G, T, off = len(SIZES), sum(SIZES), offsets(SIZES)
    rng = np.random.default_rng(K)
    x, w = ints((T, K), 3, 1), ints((G, N, K), 3, 2)
    sa = rng.uniform(0.5, 1.5, T).astype(np.float32) / 16
    sb = rng.uniform(0.5, 1.5, (G, N)).astype(np.float32)
    bias = synth.to_bf16_bits(synth.normal((G, N), 0.5, 3))
    c = torch.empty(T, N, device="cuda")
    if kind == "int8":
        za = rng.integers(-3, 4, T).astype(np.int32)
        sums = w.sum(2).astype(np.int32)
        g.gemm_grouped_int8_scaled(G, T, N, K, 1.0, dev(x.astype(np.int8)), K, dev(off), dev(w.astype(np.int8)), K,
                                   COL, N * K, dev(sa), dev(za), dev(sb), dev(sums), 0.0, c, N, OUT_F32, dev(bias),
                                   ACT_GELU_ERF)
        xv = x - za[:, None]
    else:
        code = lambda v: synth.to_e4m3_bits(v.astype(np.float64))  # noqa: E731
        g.gemm_grouped_fp8_scaled(G, T, N, K, 1.0, dev(code(x)), K, dev(off), dev(code(w)), K, COL, N * K, dev(sa),
                                  dev(sb), 0.0, c, N, OUT_F32, dev(bias), ACT_GELU_ERF)
        xv = x
    y, z, mass, _ = og.grouped(xv, off, w.transpose(0, 2, 1), np.zeros((T, N)), scale_a=sa, scale_b=sb,
                               bias=oracle.decode_bf16(bias), act=ACT_GELU_ERF)
    e = wide.bound(y, z, mass, 0, ACT_GELU_ERF, False, np.abs(oracle.decode_bf16(bias)).max())
    wide.check(c.cpu().numpy(), y, e, kind)


@pytest.mark.parametrize("K", [64, 201])
def test_int8_dense(K):
    M, N = 4200, 4500
    print(f"[gpu] stream int8 dense K={K}", flush=True)
    a, b = ints((M, K), 9, 1).astype(np.int8), ints((N, K), 9, 2).astype(np.int8)
    za = ints((M,), 9, 3).astype(np.int32)
    one = torch.ones(max(M, N), device="cuda")
    c = torch.empty(M, N, device="cuda")
    g.gemm_int8_scaled(M, N, K, 1.0, dev(a), K, ROW, dev(b), K, COL, one, dev(za), one,
                       dev(b.astype(np.int32).sum(1).astype(np.int32)), 0.0, c, N, OUT_F32)
    y, _, _ = oi.gemm_int8_scaled(a, b, np.ones(M), za, np.ones(N))
    check_exact(c.cpu().numpy(), y, "int8 dense")


@pytest.mark.parametrize("G,rows", [(130, 200), (1024, 70), (1100, 70)])
def test_many_groups(G, rows):
    """More groups than one wave's lanes, as many as the table holds, and more."""
    N, K = 300, 24
    print(f"[gpu] stream G={G}", flush=True)
    sizes = np.random.default_rng(G).integers(0, 2 * rows, G)
    T, off = int(sizes.sum()), offsets(sizes)
    x, w = ints((T, K), 3, 1), ints((G, N, K), 3, 2)
    c = torch.empty(T, N, device="cuda")
    g.gemm_grouped_bf16(G, T, N, K, 1.0, dev(bits(x)), K, dev(off), dev(bits(w)), K, COL, N * K, 0.0, c, N, OUT_F32)
    y = np.concatenate([x[off[i]:off[i + 1]].astype(np.float64) @ w[i].T for i in range(G)])
    check_exact(c.cpu().numpy(), y, "many groups")


@pytest.mark.parametrize("N,K,G", [(512, 2048, 40), (1700, 2500, 7)])
@pytest.mark.parametrize("out", [OUT_F32, OUT_BF16])
def test_weight_gradient(N, K, G, out):
    """Groups without rows, of one slice, an odd and an even number of slices; the second shape has
    tile counts that eight XCDs do not divide."""
    print(f"[gpu] stream wgrad N={N} K={K} G={G} out={out}", flush=True)
    sizes = [(0, 1, 63, 64, 65, 129, 190)[i % 7] for i in range(G)]
    T, off = sum(sizes), offsets(sizes)
    d, x = ints((T, N), 2, 1), ints((T, K), 2, 2)
    c = torch.full((G, N, K), 3.0, device="cuda", dtype=torch.float32 if out == OUT_F32 else torch.bfloat16)
    g.gemm_grouped_bf16_wgrad(G, T, N, K, 1.0, dev(bits(d)), N, dev(bits(x)), K, dev(off), 1.0, c, K, N * K, out)
    for i in range(G):
        r = slice(off[i], off[i + 1])
        y = torch.from_numpy(d[r].T.astype(np.float64) @ x[r].astype(np.float64) + 3)
        y = y.float() if out == OUT_F32 else y.to(torch.bfloat16).float()
        check_exact(c[i].float().cpu().numpy(), y.numpy(), f"group {i}")


def test_k_zero_and_no_rows():
    """K = 0 leaves act(beta C + bias); a weight gradient over no rows is zero."""
    G, N, T, off = len(SIZES), 4096, sum(SIZES), offsets(SIZES)
    c = torch.full((T, N), 2.0, device="cuda")
    b = ints((G, N), 5, 3)
    g.gemm_grouped_bf16(G, T, N, 0, 1.0, None, 1, dev(off), None, 1, COL, 0, -1.0, c, N, OUT_F32, dev(bits(b)), ACT_RELU)
    check_exact(c.cpu().numpy(), np.maximum(b[np.repeat(np.arange(G), SIZES)] - 2, 0), "K = 0")
    dw = torch.full((3, 2048, 4096), float("nan"), device="cuda")
    g.gemm_grouped_bf16_wgrad(3, 0, 2048, 4096, 1.0, None, 2048, None, 4096, dev(offsets([0, 0, 0])), 0.0, dw, 4096,
                              2048 * 4096, OUT_F32)
    assert torch.all(dw == 0).item()


def test_a_nan_stays_in_its_own_rows_and_its_own_expert():
    """A NaN token spoils its row alone, a NaN weight its group alone, an infinite row of no group nothing."""
    G, N, K, T, off = len(SIZES), 3900, 64, sum(SIZES) + 5, offsets(SIZES)
    x, w = ints((T, K), 2, 1).astype(np.float64), ints((G, N, K), 2, 2).astype(np.float64)
    x[-5:] = np.inf
    x[1600, 3] = np.nan
    w[0, 7, 5] = np.nan
    c = torch.full((T, N), 8.0, device="cuda")
    g.gemm_grouped_bf16(G, T, N, K, 1.0, dev(synth.to_bf16_bits(x)), K, dev(off), dev(synth.to_bf16_bits(w)), K, COL,
                        N * K, 0.0, c, N, OUT_F32)
    c = c.cpu().numpy()
    assert np.all(c[-5:] == 8)
    want = np.zeros((sum(SIZES), N), bool)
    want[1600] = True
    want[:1500, 7] = True
    assert np.array_equal(np.isnan(c[:-5]), want)


@pytest.mark.parametrize("bad", [[0, 9000, 100], [-70, 4000, 100], [5000, 10, 4000], [0, 1 << 30, 0]])
def test_offsets_out_of_order_or_range_stay_inside(bad):
    T, N, K, G = 5000, 4096, 64, 2
    a, b = dev(bits(ints((T, K), 2, 1))), dev(bits(ints((G * N, K), 2, 2)))
    buf = torch.full((T + 600, N), 5.0, device="cuda")
    g.gemm_grouped_bf16(G, T, N, K, 1.0, a, K, dev(np.array(bad, np.int32)), b, K, COL, N * K, 0.0,
                        buf[300:300 + T], N, OUT_F32)
    torch.cuda.synchronize()
    assert torch.all(buf[:300] == 5).item() and torch.all(buf[300 + T:] == 5).item()


def test_same_bits_under_capture_with_other_sizes():
    """The groups' sizes are data: one captured launch, replayed with other offsets, between eager calls."""
    G, N, K = 4, 4096, 128
    T = 6000
    a, b = dev(synth.to_bf16_bits(synth.normal((T, K), 1.0, 1))), dev(synth.to_bf16_bits(synth.normal((G * N, K), 1.0, 2)))
    off = dev(offsets([1500] * 4))
    c = torch.empty(T, N, device="cuda", dtype=torch.bfloat16)

    def call():
        g.gemm_grouped_bf16(G, T, N, K, 1.0, a, K, off, b, K, COL, N * K, 0.0, c, N, OUT_BF16, None, ACT_NONE)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for sizes in ([1500] * 4, [6000, 0, 0, 0], [1, 2999, 0, 3000], [256, 512, 768, 4464]):
        off.copy_(dev(offsets(sizes)))
        call()
        torch.cuda.synchronize()
        want = c.clone()
        c.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want)
