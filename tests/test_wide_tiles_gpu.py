"""Row copies on 256x256 tiles: contraction lengths that fill their last slice, columns that do not fill a chunk."""
import pytest
import torch

import dense_gemm_09_amd as g
from dense_gemm_09_amd import COL, OUT_BF16, OUT_F32, ROW
from tests import host
from tests.test_grouped_gpu import gradient, product

pytestmark = pytest.mark.gpu

SIZES = [700, 0, 513, 256, 900]


@pytest.mark.parametrize("N", [4097, 4098, 4100, 4103])
@pytest.mark.parametrize("K", [64, 128, 192])
def test_weight_along_its_rows(N, K):
    assert host.lib().grouped_tile(len(SIZES), sum(SIZES), N, 1) == 256
    product(SIZES, N, K, layout=ROW, ints=4)


@pytest.mark.parametrize("sizes,N,K", [([64, 0, 128], 2050, 2047), ([320, 1, 64], 2044, 2049),
                                       ([64, 64, 192], 1801, 2046), ([128], 4090, 4087)])
def test_gradient_of_whole_slices(sizes, N, K):
    assert host.lib().wgrad_tile(len(sizes), N, K) == 256
    gradient(sizes, N, K, OUT_F32, ints=3)
    gradient(sizes, N, K, OUT_BF16, seed=2, pad=1)


def test_a_weight_of_few_rows_far_apart():
    """Eight rows of 2^26 elements: what follows them in a slice is zero, not one of them, though one holds an infinity."""
    T, N, K, ld = 2369, 4096, 8, 1 << 26
    assert host.lib().grouped_tile(1, T, N, 1) == 256
    w = torch.zeros((K - 1) * ld + N, dtype=torch.bfloat16, device="cuda")
    rows = torch.as_strided(w, (K, N), (ld, 1))
    rows.copy_(torch.randint(-3, 4, (K, N), device="cuda", generator=torch.Generator("cuda").manual_seed(1)))
    rows[0, 5] = float("inf")
    x = torch.randint(1, 4, (T, K), device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(torch.bfloat16)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    c = torch.empty(T, N, device="cuda")
    g.gemm_grouped_bf16(1, T, N, K, 1.0, x, K, off, w, ld, ROW, 0, 0.0, c, N, OUT_F32)
    want = x.cpu().double() @ rows.cpu().double()
    assert torch.equal(c.cpu().double(), want)


@pytest.mark.parametrize("K", [4, 8, 61, 63, 64, 66, 77, 130])
def test_an_infinite_weight_in_any_row(K):
    """0 * Inf enters no sum: the chunk that K ends inside is multiplied once, by its own values."""
    N = 4096
    T = sum(SIZES)
    off = torch.tensor([0, *torch.tensor(SIZES).cumsum(0).tolist()], dtype=torch.int32)
    gen = torch.Generator().manual_seed(K)
    x = torch.randint(1, 4, (T, K), generator=gen).double()
    w = torch.randint(-3, 4, (len(SIZES), K, N), generator=gen).double()
    for i in range(len(SIZES)):
        w[i, K - 1, 3 + i] = float("inf")
        w[i, max(K - 7, 0), 300 + i] = -float("inf")
        w[i, 0, 600 + i] = float("inf")
    want = torch.cat([x[off[i]:off[i + 1]] @ w[i] for i in range(len(SIZES))])
    assert host.lib().grouped_tile(len(SIZES), T, N, 1) == 256
    c = torch.empty(T, N, device="cuda")
    for layout in (ROW, COL):
        wd = (w if layout == ROW else w.transpose(1, 2)).to(torch.bfloat16).cuda().contiguous()
        g.gemm_grouped_bf16(len(SIZES), T, N, K, 1.0, x.to(torch.bfloat16).cuda(), K, off.cuda(), wd,
                            N if layout == ROW else K, layout, N * K, 0.0, c, N, OUT_F32)
        assert torch.equal(c.cpu().double(), want), layout


@pytest.mark.parametrize("sizes,N", [([0, 1, 5, 0, 64, 65, 2], 200), ([130, 0, 257, 300, 1], 2048), ([130, 0, 257], 8192)])
@pytest.mark.parametrize("K", [61, 77])
def test_an_infinite_weight_on_smaller_tiles(sizes, N, K):
    """The same weight gives the same infinities whatever tile the call is planned on."""
    G, T = len(sizes), sum(sizes)
    assert host.lib().grouped_tile(G, T, N, 1) == 128
    gen = torch.Generator().manual_seed(K)
    x = torch.randint(1, 4, (T, K), generator=gen).double()
    w = torch.randint(-3, 4, (G, K, N), generator=gen).double()
    w[:, K - 1, 3] = float("inf")
    w[:, K - 5, 100] = -float("inf")
    off = [0, *torch.tensor(sizes).cumsum(0).tolist()]
    want = torch.cat([x[off[i]:off[i + 1]] @ w[i] for i in range(G)])
    c = torch.empty(T, N, device="cuda")
    g.gemm_grouped_bf16(G, T, N, K, 1.0, x.to(torch.bfloat16).cuda(), K, torch.tensor(off, dtype=torch.int32).cuda(),
                        w.to(torch.bfloat16).cuda(), N, ROW, N * K, 0.0, c, N, OUT_F32)
    assert torch.equal(c.cpu().double(), want)
