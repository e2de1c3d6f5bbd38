"""Pins of the oracles of routing, row movements and adapters: worked examples and central differences."""
import numpy as np
import pytest

from oracle import lora as lora_oracle
from oracle import routing as o

INF = np.inf


def test_choice_by_hand():
    x = [0.0, 2.0, 2.0, -INF, 1.0]
    assert o.choose(x, 3, o.SOFTMAX).tolist() == [1, 2, 4]  # the tie goes to the lower expert
    assert o.choose(x, 5, o.SIGMOID).tolist() == [1, 2, 4, 0, -1]
    # sigmoid 0.5, 0.881, 0.881, -, 0.731: a bias moves expert 0 to the front
    assert o.choose(x, 2, o.SIGMOID, [0.5, 0, 0, 9, 0]).tolist() == [0, 1]
    assert o.choose(x, 2, o.SIGMOID, [-INF, np.nan, 0, 0, 0]).tolist() == [2, 4]
    assert o.choose([-INF] * 3, 2, o.SOFTMAX).tolist() == [-1, -1]
    assert o.choose([0, np.nan], 1, o.SIGMOID) is None and o.choose([0, INF], 1, o.SOFTMAX) is None
    assert o.choose([0, INF], 1, o.SIGMOID).tolist() == [1]


def test_groups_by_hand():
    x = np.log([4.0, 1.0, 3.0, 3.0])  # softmax 4/11, 1/11, 3/11, 3/11
    assert o.choose(x, 2, o.SOFTMAX, None, 2, 1, 1).tolist() == [0, 1]
    assert o.choose(x, 2, o.SOFTMAX, np.zeros(4), 2, 1, 2).tolist() == [2, 3]  # 6/11 beats 5/11
    # a group with one expert left counts that one
    assert o.choose([5.0, -INF, 1.0, 1.0], 2, o.SOFTMAX, np.zeros(4), 2, 1, 2).tolist() == [0, -1]


def test_weights_by_hand():
    x = np.log([4.0, 1.0, 3.0, 2.0])
    assert np.allclose(o.weights(x, [0, 2, -1], o.SOFTMAX, False, 1.0), [0.4, 0.3, 0.0])
    assert np.allclose(o.weights(x, [0, 2, -1], o.SOFTMAX, True, 2.0), [8 / 7, 6 / 7, 0.0])
    # scores that are nothing in float64 still have shares
    assert np.allclose(o.weights([-800.0, -800.0, -801.0], [0, 1], o.SIGMOID, True, 1.0), [0.5, 0.5])


@pytest.mark.parametrize("score", [o.SOFTMAX, o.SIGMOID])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradient_against_differences(score, renormalise):
    rng = np.random.default_rng(3)
    x, ids, dw = rng.standard_normal(9), np.array([4, 0, -1, 7]), rng.standard_normal(4)
    f = lambda v: (o.weights(v, ids, score, renormalise, 1.7) * dw).sum()  # noqa: E731
    h = 1e-6
    want = [(f(x + h * e) - f(x - h * e)) / (2 * h) for e in np.eye(9)]
    assert np.allclose(o.grad(x, ids, dw, score, renormalise, 1.7), want, rtol=1e-7, atol=1e-9)


def test_order_and_rows_by_hand():
    offsets, position, order = o.order([2, 0, -1, 2, 0, 5], 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert position.tolist() == [2, 0, -1, 3, 1, -1] and order.tolist() == [1, 4, 0, 3, -1, -1]
    y = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    c, mass = o.combine(y, np.array([[2, 0], [-1, 1]]), [[0.5, -2.0], [7.0, 1.0]], np.ones((2, 2)), 10.0)
    assert c.tolist() == [[10.5, 9.0], [13.0, 14.0]] and mass.tolist() == [[14.5, 17.0], [13.0, 14.0]]


def test_row_gradients_against_differences():
    rng = np.random.default_rng(4)
    y, w, d = rng.standard_normal((4, 3)), rng.standard_normal((2, 2)), rng.standard_normal((2, 3))
    pos = np.array([[3, 0], [-1, 1]])
    dy, written, dw, _ = o.combine_grad(d, y, pos, w)
    assert written.tolist() == [True, True, False, True] and dw[1, 0] == 0
    f = lambda y_, w_: (o.combine(y_, pos, w_)[0] * d).sum()  # noqa: E731
    h = 1e-6
    for i in np.ndindex(y.shape):
        e = np.zeros_like(y)
        e[i] = h
        assert np.isclose((f(y + e, w) - f(y - e, w)) / (2 * h), dy[i], atol=1e-8)
    for i in np.ndindex(w.shape):
        e = np.zeros_like(w)
        e[i] = h
        assert np.isclose((f(y, w + e) - f(y, w - e)) / (2 * h), dw[i], atol=1e-8)


def test_lora_by_its_whole_weight():
    rng = np.random.default_rng(5)
    a, b = rng.standard_normal((4, 5)), rng.standard_normal((5, 3))
    down, up, scale = rng.standard_normal((2, 2, 5)), rng.standard_normal((2, 3, 2)), [0.5, 3.0]
    c, bias = rng.standard_normal((4, 3)), rng.standard_normal(3)
    y, z, (main, low, add) = lora_oracle.lora(a, b, [1, -1, 0, 2], down, up, scale, c, 2.0, -1.0, bias, 1)
    for m, g in enumerate([1, None, 0, None]):
        w = b if g is None else b + scale[g] * (up[g] @ down[g]).T
        want = 2.0 * a[m] @ w - c[m] + bias
        assert np.allclose(z[m], want) and np.allclose(y[m], np.maximum(want, 0))
    assert (low[[1, 3]] == 0).all() and (main + low + add >= np.abs(z) - 1e-12).all()
