"""Groups by the sum of their two best scores where that sum is beyond FP32: biases near the end of its range."""
import numpy as np
import pytest

from oracle import routing as o
from tests.test_route_gpu import check, logits, run

import torch

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("score", [o.SOFTMAX, o.SIGMOID])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("E,groups", [(64, 8), (60, 6), (256, 4)])
def test_sums_beyond_fp32(E, groups, sign, score):
    """Every sum of two is beyond FP32 (of one sign); the best groups are not the first ones."""
    per = E // groups
    b = np.full(E, 1.8e38 * sign, np.float32)
    for i in range(groups):  # later groups' best are larger
        b[i * per] = (2e38 + 1e37 * i) * sign
        b[i * per + 1] = 1.9e38 * sign
    if sign < 0:
        b = b[::-1].copy()
    x = logits(20, E, torch.float32, E)
    x[3, : E // 2] = -INF
    x[4, ::2] = -INF
    x[5] = -INF
    x[6, 2:] = -INF
    for top in (1, 2, groups - 1):
        k = min(4, per * top)
        ids, w = run(x, k, score, b, groups, top, 2, True)
        check(x, k, score, ids, w, b, groups, top, 2, True)


def test_a_sum_below_the_range_is_no_empty_group():
    """Group 0 is masked; group 1's sum is below FP32's range, and is chosen before it."""
    x = logits(3, 16, torch.float32, 1)
    x[:, :8] = -INF
    b = np.full(16, -3e38, np.float32)
    ids, w = run(x, 2, o.SIGMOID, b, 2, 1, 2)
    check(x, 2, o.SIGMOID, ids, w, b, 2, 1, 2)
    assert (ids >= 8).all()
