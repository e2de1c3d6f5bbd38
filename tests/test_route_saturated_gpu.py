"""Scores that 64 bits do not tell apart are equal, and go to the lowest index; logits, which a choice without bias and
with one best per group compares, are always told apart."""
import numpy as np
import pytest
import torch

from oracle import routing as o
from tests.test_route_gpu import check, run

pytestmark = pytest.mark.gpu


def rows(score):
    """Eight experts in two groups: expert 0's logit is the lowest of those that saturate, expert 3's the highest."""
    x = torch.full((2, 8), -5.0)
    if score == o.SIGMOID:
        x[:, :4] = torch.tensor([40.0, 50.0, 45.0, 60.0])  # all 1
    else:
        x[:, 0] = 0.0
        x[:, 1:] = torch.tensor([-800.0, -790.0, -780.0, -900.0, -760.0, -1000.0, -750.0])  # all 0 next to it
    x[1] = x[1].flip(0)
    return x


@pytest.mark.parametrize("score", [o.SOFTMAX, o.SIGMOID])
@pytest.mark.parametrize("bias,best", [(True, 1), (True, 2), (False, 2)])
def test_scores(score, bias, best):
    x = rows(score)
    b = np.zeros(8, np.float32) if bias else None
    for groups, top in ((1, 1), (2, 2), (2, 1)):
        if groups == 1 and not bias:
            continue  # one group: its score is not needed, and logits are compared
        ids, w = run(x, 4, score, b, groups, top, best)
        check(x, 4, score, ids, w, b, groups, top, best)
    if score == o.SIGMOID:
        assert ids.tolist() == [[0, 1, 2, 3], [4, 5, 6, 7]]


@pytest.mark.parametrize("score", [o.SOFTMAX, o.SIGMOID])
@pytest.mark.parametrize("groups,top,best", [(1, 1, 1), (2, 2, 1), (2, 1, 1)])
def test_logits(score, groups, top, best):
    x = rows(score)
    ids, w = run(x, 4, score, None, groups, top, best)
    check(x, 4, score, ids, w, None, groups, top, best)
    want = torch.sort(x[0, :4] if groups == 2 and top == 1 else x[0], descending=True).indices[:4]
    assert ids[0].tolist() == want.tolist()
