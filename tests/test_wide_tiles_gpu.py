"""Row copies on 256x256 tiles: contraction lengths that fill their last slice, columns that do not fill a chunk."""
import pytest

from dense_gemm_09_amd import OUT_BF16, OUT_F32, ROW
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
