"""Softmax weights of logits far below the largest.

The largest logit is alone: the other scores are below 2^-60, so the sum is 1 to a last bit or two (two of E terms).
A weight is then an exponential (1 step of 2^-23), corrected for the difference's rounding (two operations), divided,
and for shares divided by their sum (E operations): 3 + 2 + 2 + 2 E roundings of U = 2^-24, all of one size, whatever the
distance. The difference's own rounding alone would be up to 64 U at these distances. Its square, below 2^-36, is nothing.
"""
import numpy as np
import pytest
import torch

from oracle import routing as o
from tests.test_route_gpu import run

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E", [4, 6])
def test_far_logits(E, bias, renorm):
    T = 500
    gen = torch.Generator().manual_seed(E)
    x = torch.rand(T, E, generator=gen) * 30
    x[:, 0] = 75 + torch.rand(T, generator=gen) * 5
    b = np.zeros(E, np.float32) if bias else None
    ids, w = run(x, E, o.SOFTMAX, b, renorm=renorm)
    X = x.double().numpy()
    for t in range(T):
        want = o.weights(X[t], ids[t], o.SOFTMAX, renorm, 1.0)
        assert sorted(ids[t].tolist()) == list(range(E))
        assert (np.abs(w[t] - want) <= (7 + 2 * E) * U * want).all(), (t, (np.abs(w[t] - want) / want / U).max())
