"""The tiles that BF16 plans have: the projection with adapters is compiled for these alone."""
import random

import dense_gemm_09_amd as g


def test_tiles_of_plans():
    """256x128 tiles have a split K in every plan (at most 64 rows take 64-row tiles)."""
    rng = random.Random(0)
    seen = set()
    shapes = [(100, 512, 2048), (100, 512, 2046)]
    for _ in range(6000):
        shapes.append(tuple(int(2 ** rng.uniform(lo, hi)) for lo, hi in ((4.1, 15), (0, 16), (0, 16))))
    for M, N, K in shapes:
        p = g.plan(M, N, K, False)
        tile = (p.tile_m, p.tile_n)
        assert tile in {(64, 256), (64, 128), (256, 256), (128, 128), (256, 128)}
        assert tile != (256, 128) or p.split_k > 1, (M, N, K)
        seen.add((tile, p.split_k > 1))
    assert ((256, 128), True) in seen and ((256, 256), True) in seen and ((128, 128), False) in seen
