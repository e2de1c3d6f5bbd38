"""The projection with low-rank adapters against the float64 definition.

Tolerance. The main product is a sum of K terms in FP32 (at most 16 partial sums of it are added): (K + 16) U of its
magnitudes. An adapter's h is a sum of K terms and a scale: (K + 2) U, kept to 2^-16 of itself (BF16 high part and
remainder, each off by at most 2^-8 of what it represents), its second product a sum of 2 R terms, added to the
main sum: together (K + 2 R + 20) U + 2^-16 (1 + 2^-8) of the magnitudes of both factors' products. Then alpha,
beta C, bias, activation and output as for the other products (tests/wide.py).
"""
import numpy as np
import pytest
import torch

import dense_gemm_09_amd as g
from oracle import lora as oracle
from tests import tolerance, wide

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def bound(y, z, mags, K, R, act, bf16):
    main, low, add = mags
    n, m = (K + 20) * U, (K + 2 * R + 24) * U
    e = n / (1 - n) * main + (m / (1 - m) + 2.0 ** -16 * (1 + 2.0 ** -7)) * low + 4 * U * (np.abs(z) + add + main + low)
    e = e * tolerance.slope_bound(z, e, act) + (tolerance.ACT_REL[act] + U) * np.abs(y)
    if bf16:
        e = e * (1 + 2.0 ** -7) + (2.0 ** -8 + (2.0 ** -16 if act in tolerance.ACT_GELU else 0)) * np.abs(y) + 2.0 ** -134
    return e + 2.0 ** -149


def block(rows, ld, cols, std, seed, shift=0):
    """BF16 rows of `cols` values in a leading dimension ld, NaN between them, `shift` elements into an allocation."""
    flat = torch.full((shift + rows * ld,), float("nan"), dtype=torch.bfloat16)
    v = flat[shift:].view(rows, ld)
    v[:, :cols] = (torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)) * std).bfloat16()
    return v[:, :cols].double().numpy(), flat.cuda()[shift:]


def problem(M, N, K, G, R, adapter, out="bf16", bias=True, act=0, alpha=1.0, beta=0.0, pad=0, shift=0, up_pad=0,
            scale=True, low=1.0):
    a, da = block(M, K + pad, K, 1.0, 1, shift)
    b, db = block(N, K + pad, K, 0.05, 2, shift)
    down, ddown = block(G * R, K + pad, K, 0.05 * low, 3, shift)
    up, dup = block(G * N, R + up_pad, R, 0.3, 4, shift if up_pad else 0)
    gen = torch.Generator().manual_seed(5)
    s = torch.rand(G, generator=gen) + 0.5
    bv = (torch.randn(N, generator=gen) * 0.2).bfloat16()
    ot = torch.float32 if out == "f32" else torch.bfloat16
    c = torch.randn(M, N + 3, generator=gen).to(ot)
    dc = c.cuda() if beta else torch.full((M, N + 3), float("nan"), dtype=ot, device="cuda")
    ids = torch.from_numpy(np.asarray(adapter, np.int32))
    g.gemm_lora_bf16(M, N, K, G, R, alpha, da, K + pad, db, K + pad, ids.cuda(), ddown, K + pad, R * (K + pad), dup,
                     R + up_pad, N * (R + up_pad), s.cuda() if scale else None, beta, dc, N + 3,
                     g.OUT_F32 if out == "f32" else g.OUT_BF16, bv.cuda() if bias else None, act)
    got = dc.cpu().double().numpy()
    assert (np.isnan(got[:, N:]) if not beta else got[:, N:] == c.double().numpy()[:, N:]).all()
    y, z, mags = oracle.lora(a, b.T, adapter, down.reshape(G, R, K), up.reshape(G, N, R),
                             s.numpy() if scale else None, c.double().numpy()[:, :N], alpha, beta,
                             bv.double().numpy() if bias else None, act)
    wide.check(got[:, :N], y, bound(y, z, mags, K, R, act, out == "bf16"))


def rows_of(M, G, kind, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "mixed":
        a = rng.integers(0, G, M)
    elif kind == "sorted":
        a = np.sort(rng.integers(0, G, M))
    elif kind == "one":
        a = np.full(M, G - 1)
    else:
        a = np.full(M, -1)
    if kind in ("mixed", "sorted"):
        a[rng.random(M) < 0.15] = rng.choice([-1, G, 1 << 30, -(1 << 31)])
    return a.astype(np.int32)


@pytest.mark.parametrize("kind", ["mixed", "sorted", "one", "none"])
@pytest.mark.parametrize("M,N,K,G,R", [
    (1, 256, 256, 3, 16), (2, 64, 4096, 2, 8), (7, 1000, 512, 9, 4), (16, 512, 1024, 16, 16), (16, 528, 8192, 5, 32),
    (17, 300, 520, 4, 16), (33, 256, 2048, 33, 64), (64, 640, 4096, 20, 16), (64, 4096, 1024, 8, 128),
    (65, 260, 256, 6, 20), (100, 512, 2048, 7, 1), (128, 384, 640, 40, 24), (256, 512, 512, 3, 16),
    (300, 520, 264, 300, 8), (600, 768, 1024, 10, 40), (1000, 256, 128, 2, 128)])
def test_parity(M, N, K, G, R, kind):
    problem(M, N, K, G, R, rows_of(M, G, kind))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("M,N,K", [(5, 272, 512), (16, 1040, 8192), (40, 260, 1031), (200, 516, 257), (520, 300, 64)])
def test_epilogue(M, N, K, act, out):
    problem(M, N, K, 4, 16, rows_of(M, 4, "mixed"), out, act=act, alpha=0.75, beta=-0.5)


@pytest.mark.parametrize("M", [1, 3, 16, 30, 150])
@pytest.mark.parametrize("N,K,R,pad,shift,up_pad", [
    (37, 41, 5, 0, 0, 0), (64, 100, 16, 3, 1, 1), (129, 4099, 13, 0, 1, 0), (50, 8, 3, 8, 0, 5), (96, 1, 2, 0, 0, 0),
    (33, 65, 17, 1, 3, 2), (256, 256, 8, 0, 4, 4), (70, 40, 8, 8, 8, 8), (40, 4104, 127, 0, 0, 1)])
def test_odd_sizes_and_strides(M, N, K, R, pad, shift, up_pad):
    problem(M, N, K, 6, R, rows_of(M, 6, "mixed", M), "f32", pad=pad, shift=shift, up_pad=up_pad, scale=M % 2 == 0)


@pytest.mark.parametrize("M", [4, 16, 48, 200])
def test_an_adapter_that_outweighs_the_projection(M):
    problem(M, 256, 512, 3, 16, rows_of(M, 3, "mixed"), "f32", low=100.0)


@pytest.mark.parametrize("M", [6, 50, 140])
def test_no_adapters_and_no_k(M):
    a, da = block(M, 64, 64, 1.0, 1)
    b, db = block(128, 64, 64, 0.1, 2)
    ids = torch.zeros(M, device="cuda", dtype=torch.int32)
    for G, R in ((0, 16), (4, 0)):
        c = torch.empty(M, 128, device="cuda")
        g.gemm_lora_bf16(M, 128, 64, G, R, 1.0, da, 64, db, 64, ids if G == 0 else None, None, 64, 0, None, 16, 0, None,
                         0.0, c, 128, g.OUT_F32)
        y = a @ b.T
        wide.check(c.cpu().numpy(), y, wide.bound(y, y, np.abs(a) @ np.abs(b.T), 64 + 16, 0, False))
    up = torch.ones(4 * 128 * 8, device="cuda", dtype=torch.bfloat16)
    c = torch.full((M, 128), 3.0, device="cuda")
    g.gemm_lora_bf16(M, 128, 0, 4, 8, 1.0, None, 1, None, 1, ids, None, 1, 0, up, 8, 128 * 8, None, 0.5, c, 128, g.OUT_F32)
    assert (c == 1.5).all()


@pytest.mark.parametrize("M", [12, 60, 200])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["down", "up", "a"])
@pytest.mark.parametrize("R", [8, 16, 5])
def test_a_bad_adapter_stays_in_its_rows(M, R, where, what):
    N, K, G = 160, 256, 4
    gen = torch.Generator("cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    a, b, down, up = rand(M, K), rand(N, K), rand(G, R, K), rand(G, N, R)
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % (G + 1)  # G: none

    def run():
        c = torch.empty(M, N, device="cuda")
        g.gemm_lora_bf16(M, N, K, G, R, 1.0, a, K, b, K, ids, down, K, R * K, up, R, N * R, None, 0.0, c, N, g.OUT_F32)
        return c
    good = run()
    if where == "a":
        a[7] = what
        bad = torch.arange(M, device="cuda") == 7
    else:
        (down if where == "down" else up)[2] = what
        bad = ids == 2
    c = run()
    assert torch.equal(c[~bad], good[~bad]) and not c[bad].isfinite().any()


def test_rows_do_not_depend_on_their_neighbours():
    """A request's rows are the same bits whoever shares the batch with it, while the kernel is the same."""
    N, K, G, R = 512, 1024, 8, 16
    gen = torch.Generator("cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    a, b, down, up = rand(48, K), rand(N, K), rand(G, R, K), rand(G, N, R)

    def run(ids):
        c = torch.empty(48, N, device="cuda")
        g.gemm_lora_bf16(48, N, K, G, R, 1.0, a, K, b, K, ids, down, K, R * K, up, R, N * R, None, 0.0, c, N, g.OUT_F32)
        return c
    ids = torch.arange(48, device="cuda", dtype=torch.int32) % G
    other = ids.clone()
    other[::2] = 3
    assert torch.equal(run(ids)[1::2], run(other)[1::2])


def test_shared_and_far_adapters():
    """Strides of zero (one adapter for all) and adapters further apart than 2^31 elements."""
    M, N, K, R = 20, 64, 64, 8
    gen = torch.Generator("cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    a, b = rand(M, K), rand(N, K)
    far = (1 << 31) + 64
    down, up = torch.zeros(far + R * K, device="cuda", dtype=torch.bfloat16), torch.zeros(far + N * R, device="cuda", dtype=torch.bfloat16)
    down[:R * K] = rand(R * K)
    up[:N * R] = rand(N * R)
    down[far:], up[far:] = down[:R * K], up[:N * R]
    ids = (torch.arange(M, device="cuda", dtype=torch.int32) % 2).contiguous()

    def run(stride_down, stride_up):
        c = torch.empty(M, N, device="cuda")
        g.gemm_lora_bf16(M, N, K, 2, R, 1.0, a, K, b, K, ids, down, K, stride_down, up, R, stride_up, None, 0.0, c, N, g.OUT_F32)
        return c
    assert torch.equal(run(0, 0), run(far, far))
