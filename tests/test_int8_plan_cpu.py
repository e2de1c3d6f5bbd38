"""Plans of the 8-bit types that the INT8 kernels have to have (no GPU)."""
import itertools
import random

import dense_gemm_09_amd as g

# Rows, columns of the tiles that the INT8 product has kernels for.
INT8_TILES = {(64, 256), (64, 128), (128, 128), (256, 256)}


def test_every_plan_has_an_int8_kernel():
    rng = random.Random(5)
    even = itertools.product((65, 128, 129, 256, 300, 512, 1000, 2048, 4096, 8192, 20000), repeat=2)
    shapes = [(m, n, k) for m, n in even for k in (1, 128, 1000, 1920, 2048, 2100, 4096, 14336, 131071)]
    shapes += [tuple(int(2 ** rng.uniform(0, top)) for top in (16, 16, 17)) for _ in range(40000)]
    seen = set()
    for m, n, k in shapes:
        p = g.plan(m, n, k, True)
        if p.kernel == 0:
            seen.add((p.tile_m, p.tile_n))
    assert seen == INT8_TILES
