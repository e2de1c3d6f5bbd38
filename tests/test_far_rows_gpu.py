"""INT8 and grouped products whose operands are too far apart for 32-bit copies: they are loaded through registers."""
import pytest
import torch

import dense_gemm_09_amd as g
from dense_gemm_09_amd import ACT_RELU, COL, OUT_BF16, OUT_F32, QOUT_INT8, ROW

pytestmark = pytest.mark.gpu


def ints(shape, seed, top=3):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda", dtype=torch.int8)


def spread(x, ld, kind):
    """The rows of x, ld elements apart, in an array of their own type: (array, values)."""
    t = {"int8": torch.int8, "fp8": torch.float8_e4m3fn, "bf16": torch.bfloat16}[kind]
    rows, cols = x.shape
    buf = torch.zeros((rows - 1) * ld + cols, dtype=t, device="cuda")
    as_bytes = buf.view(torch.int8 if kind != "bf16" else torch.int16)
    as_bytes.as_strided((rows, cols), (ld, 1)).copy_(x.to(t).view(as_bytes.dtype))
    return buf


def offsets(sizes):
    return torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", ["int8", "fp8", "bf16"])
def test_grouped_rows_far_apart(kind):
    sizes, N, K = [3, 0, 6, 1], 130, 77
    T, G, ld = sum(sizes), len(sizes), (1 << 22) if kind == "bf16" else (1 << 23)
    x, w = ints((T, K), 1), ints((G * N, K), 2)
    xd, wd, off = spread(x, ld, kind), spread(w, K, kind), offsets(sizes)
    one_t, one_n = torch.ones(T, device="cuda"), torch.ones(G * N, device="cuda")
    c = torch.full((T, N), 2.0, device="cuda")
    if kind == "bf16":
        g.gemm_grouped_bf16(G, T, N, K, 1.0, xd, ld, off, wd, K, COL, N * K, 1.0, c, N, OUT_F32)
    elif kind == "fp8":
        g.gemm_grouped_fp8_scaled(G, T, N, K, 1.0, xd, ld, off, wd, K, COL, N * K, one_t, one_n, 1.0, c, N, OUT_F32)
    else:
        g.gemm_grouped_int8_scaled(G, T, N, K, 1.0, xd, ld, off, wd, K, COL, N * K, one_t, None, one_n, None, 1.0, c,
                                   N, OUT_F32)
    o = off.tolist()
    W = w.double().view(G, N, K)
    want = torch.cat([x[o[i]:o[i + 1]].double() @ W[i].t() for i in range(G)]) + 2
    assert torch.equal(c.double(), want)


@pytest.mark.parametrize("layout", [COL, ROW])
def test_a_weight_of_2_gib(layout):
    """Past 2^31 bytes from a weight's first element to its last."""
    T, N, K = 9, 130, 129
    ld = 1 << 23
    x, w = ints((T, K), 1), ints((N, K), 2)
    wd = spread(w if layout == COL else w.t(), ld, "bf16")
    c = torch.empty(T, N, device="cuda")
    g.gemm_grouped_bf16(1, T, N, K, 1.0, x.bfloat16(), K, offsets([T]), wd, ld, layout, 0, 0.0, c, N, OUT_F32)
    assert torch.equal(c.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("out", [OUT_F32, OUT_BF16])
def test_weight_gradient_rows_far_apart(out):
    sizes, N, K, ld = [3, 0, 6, 1], 131, 70, 1 << 24
    T, G = sum(sizes), len(sizes)
    d, x = ints((T, N), 1), ints((T, K), 2)
    c = torch.full((G, N, K), 2.0, device="cuda", dtype=torch.float32 if out == OUT_F32 else torch.bfloat16)
    g.gemm_grouped_bf16_wgrad(G, T, N, K, 1.0, spread(d, ld, "bf16"), ld, x.bfloat16(), K, offsets(sizes), 1.0, c, K,
                              N * K, out)
    o = offsets(sizes).tolist()
    want = torch.stack([d[o[i]:o[i + 1]].double().t() @ x[o[i]:o[i + 1]].double() for i in range(G)]) + 2
    assert torch.equal(c.double(), want)  # below 2^8: BF16 values


@pytest.mark.parametrize("M,N,K", [(40, 300, 8192), (200, 600, 257)])
def test_int8_rows_far_apart(M, N, K):
    """The first shape is split along K, the second is not."""
    assert (g.plan(M, N, K, True).split_k > 1) == (K == 8192)
    ld = 1 << (26 if M == 40 else 24)
    a, b = ints((M, K), 1, 9), ints((N, K), 2, 9)
    ad = spread(a, ld, "int8")
    za = ints((M,), 3, 9).int()
    sums = b.sum(1, dtype=torch.int32)
    one = torch.ones(max(M, N), device="cuda")
    want = a.double() @ b.double().t() - za.double()[:, None] * b.double().sum(1)
    c = torch.full((M, N), 2.0, device="cuda")
    g.gemm_int8_scaled(M, N, K, 1.0, ad, ld, ROW, b, K, COL, one, za, one, sums, -1.0, c, N, OUT_F32)
    assert torch.equal(c.double(), want - 2)
    h = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    g.gemm_int8_scaled(M, N, K, 1.0, ad, ld, ROW, b, K, COL, one, za, one, sums, 0.0, h, N, OUT_BF16, None, ACT_RELU)
    assert torch.equal(h, want.clamp(min=0).float().bfloat16())
    q = torch.empty(M, N, device="cuda", dtype=torch.int8)
    scale = torch.full((M,), 2.0 ** -7, device="cuda")
    g.gemm_int8_scaled_quant(M, N, K, 1.0, ad, ld, ROW, b, K, COL, one, za, one, sums, None, 0, scale, None, q, N,
                             QOUT_INT8)
    assert torch.equal(q.double(), (want / 128).round().clamp(-128, 127))
