"""Routing and its gradient against the float64 definition.

Tolerances. An FP32 operation is off by at most U = 2^-24 of its result; expf, log1pf and the division by at most
4 U. A softmax score exp(x - top) / sum: the difference is off by U |x - top|, which the exponential turns into
a relative error, its own error is 4 U, the sum of E positive terms adds E U and the terms' own errors (a term
t exp(-t) U stays below U), then a division and the scale: (|x - top| + E + 16) U. log sigmoid is off by at most
(|log s| + 8) U absolute (a sum of two terms of one sign, log1p of at most log 2), a share of the chosen from
their logarithms l by those errors, the difference's (|l| + |top|), the exponential, a sum of k and a division.
Below FP32's smallest normal number a result may be off by that number.
"""
import numpy as np
import pytest
import torch

import dense_gemm_09_amd as g
from oracle import routing as o

pytestmark = pytest.mark.gpu

INF = float("inf")
U = 2.0 ** -24
TINY = 2.0 ** -126


def run(x, k, score, bias=None, groups=1, top=1, best=1, renorm=False, scale=1.0, ld=None):
    """x: CPU tensor FP32 or BF16 [T, E] -> expert, weight (numpy)."""
    T, E = x.shape
    ld = E if ld is None else ld
    buf = torch.full((T, ld), float("nan"), dtype=x.dtype)
    buf[:, :E] = x
    kind = g.OUT_F32 if x.dtype == torch.float32 else g.OUT_BF16
    ids = torch.full((T * k + 1,), 77, device="cuda", dtype=torch.int32)
    w = torch.full((T * k + 1,), 77.0, device="cuda")
    b = None if bias is None else torch.as_tensor(bias, dtype=torch.float32).cuda()
    g.route(T, E, k, buf.cuda(), ld, kind, score, b, groups, top, best, renorm, scale, ids, w)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    assert ids[-1] == 77 and w[-1] == 77  # nothing behind the last row
    return ids[:-1].reshape(T, k), w[:-1].reshape(T, k)


def weight_bound(x, ids, score, renorm, scale, want):
    """|computed - want| of one row's weights."""
    E, k = len(x), len(ids)
    logs = o.log_scores(x, score)
    live = ids >= 0
    if not live.any():
        return np.zeros(k)
    far = np.abs(logs[ids[live]])
    if renorm:
        if score == o.SOFTMAX:  # from the logits themselves
            far = np.abs(x[ids[live]])
        rel = 2 * (2 * far.max() + 8) + k + 16
    elif score == o.SIGMOID:
        rel = far.max() + 24
    else:
        top = x[x > -INF].max()
        rel = np.abs(x[ids[live]] - top).max() + E + 16
    return rel * U * np.abs(want) + TINY * scale


def check(x, k, score, ids, w, bias=None, groups=1, top=1, best=1, renorm=False, scale=1.0):
    X = x.double().numpy()
    for t in range(len(X)):
        want = o.choose(X[t], k, score, bias, groups, top, best)
        if want is None:
            assert (ids[t] == -1).all() and np.isnan(w[t]).all(), t
            continue
        assert ids[t].tolist() == want.tolist(), (t, ids[t], want)
        y = o.weights(X[t], want, score, renorm, scale)
        e = weight_bound(X[t], want, score, renorm, scale, y)
        assert (np.abs(w[t] - y) <= e).all(), (t, w[t], y, e)
        assert (w[t][want < 0] == 0).all()


def logits(T, E, dtype, seed, std=2.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=gen) * std).to(dtype)


SHAPES = [(1, 1, 1), (1, 64, 6), (3, 2, 2), (5, 60, 4), (70, 64, 8), (9, 65, 5), (33, 128, 8), (17, 256, 8),
          (6, 257, 32), (5, 512, 10), (4, 1000, 7), (3, 1024, 32), (2, 33, 32), (130, 8, 2), (67, 16, 4),
          (40, 17, 3), (21, 384, 6)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [(o.SOFTMAX, False), (o.SOFTMAX, True), (o.SIGMOID, False),
                                          (o.SIGMOID, True)])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_parity(T, E, k, score, renorm, dtype):
    x = logits(T, E, dtype, 100 * E + k)
    x[torch.rand(T, E, generator=torch.Generator().manual_seed(E)) < 0.1] = -INF
    ids, w = run(x, k, score, renorm=renorm, scale=2.5, ld=E + 3)
    check(x, k, score, ids, w, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", [o.SOFTMAX, o.SIGMOID])
@pytest.mark.parametrize("E,groups,top,best,k", [(256, 8, 4, 2, 8), (64, 4, 2, 1, 6), (60, 6, 2, 2, 5), (128, 64, 3, 1, 4),
                                                 (24, 1, 1, 2, 3), (160, 8, 3, 2, 6), (512, 16, 1, 2, 8),
                                                 (1024, 32, 5, 2, 11), (16, 8, 8, 2, 16), (10, 5, 2, 2, 4),
                                                 (256, 4, 4, 1, 8), (96, 3, 1, 2, 8)])
@pytest.mark.parametrize("bias", [False, True])
def test_groups(E, groups, top, best, k, score, bias):
    T = 41
    x = logits(T, E, torch.float32, E + groups)
    x[torch.rand(T, E, generator=torch.Generator().manual_seed(5)) < 0.3] = -INF
    x[7] = -INF
    x[8, 1:] = -INF
    b = (np.random.default_rng(E).standard_normal(E) * 0.3).astype(np.float32) if bias else None
    ids, w = run(x, k, score, b, groups, top, best, True, 1.0)
    check(x, k, score, ids, w, b, groups, top, best, True, 1.0)


@pytest.mark.parametrize("score", [o.SOFTMAX, o.SIGMOID])
@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
@pytest.mark.parametrize("E,groups,top,best", [(64, 1, 1, 1), (256, 8, 3, 2), (40, 4, 2, 1)])
def test_equal_scores_go_to_the_lowest_index(E, groups, top, best, score, bias):
    """Three values only: nearly everything is a tie."""
    x = torch.randint(0, 3, (50, E), generator=torch.Generator().manual_seed(E)).float()
    x[3] = 1.0
    b = None if bias is None else np.full(E, bias, np.float32)
    if b is None and best == 2:
        b = np.zeros(E, np.float32)
    ids, w = run(x, 6, score, b, groups, top, best)
    check(x, 6, score, ids, w, b, groups, top, best)


def test_scores_that_differ_in_their_last_bits():
    """With a bias: sigmoids 2^-30 apart, far below an FP32 step of the scores, are told apart."""
    E = 64
    x = torch.zeros(2, E)
    # neighbours of 0 in FP32 have sigmoids 2^-151 apart: take steps of 2^-28, sigmoid' = 1/4
    x[0] = torch.arange(E).flip(0).float() * 2.0 ** -28
    x[1] = torch.arange(E).float() * 2.0 ** -28
    b = np.full(E, 0.5, np.float32)
    ids, w = run(x, 8, o.SIGMOID, b, renorm=True)
    assert ids[0].tolist() == list(range(8)) and ids[1].tolist() == list(range(63, 55, -1))
    check(x, 8, o.SIGMOID, ids, w, b, renorm=True)


@pytest.mark.parametrize("score", [o.SOFTMAX, o.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_whose_mask_leaves_little(score, renorm, dtype):
    E, low = 48, torch.finfo(dtype).min
    x = logits(10, E, dtype, 2)
    x[0] = -INF          # nothing left
    x[1] = low           # the type's lowest value is a logit like any other
    x[2, 3:] = low
    x[3, 1:] = -INF      # one expert
    x[4, 5] = float("nan")
    x[5, 6] = INF        # the best by far (softmax: no scores)
    x[6] = -200.0        # sigmoids below FP32
    x[7, ::2] = -INF
    x[8] = torch.finfo(dtype).max
    for bias in (None, np.zeros(E, np.float32)):
        ids, w = run(x, 4, score, bias, renorm=renorm)
        check(x, 4, score, ids, w, bias, renorm=renorm)


def test_bias_that_is_not_a_number():
    x = logits(20, 32, torch.float32, 4)
    b = np.zeros(32, np.float32)
    b[[1, 5]], b[7], b[[9, 20]] = -np.inf, np.nan, np.inf
    ids, w = run(x, 5, o.SIGMOID, b)
    check(x, 5, o.SIGMOID, ids, w, b)
    assert (ids[:, :2] == [9, 20]).all()


# ---------------------------------------------------------------- gradient

def run_grad(x, ids, dw, score, renorm, scale, ld):
    T, E = x.shape
    kind = g.OUT_F32 if x.dtype == torch.float32 else g.OUT_BF16
    out = torch.full((T, ld), 9.0, device="cuda", dtype=x.dtype)
    g.route_grad(T, E, ids.shape[1], x.cuda(), E, kind, score, renorm, scale, torch.as_tensor(ids).int().cuda(),
                 torch.as_tensor(dw).cuda(), out, ld)
    out = out.cpu()
    assert (out[:, E:] == 9).all()
    return out[:, :E].double().numpy()


def grad_bound(x, ids, dw, score, renorm, scale, bf16):
    """Every term of an element's gradient is a product of a score or share (relative error as above), a dweight
    and factors; terms are summed: their magnitudes times the relative error."""
    E, k = len(x), len(ids)
    live = (ids >= 0) & (ids < E)
    out = np.zeros(E)
    if not live.any():
        return out
    s = np.exp(o.log_scores(x, score))
    finite = x[x > -INF]
    far = np.abs(finite).max() if len(finite) else 0.0
    rel = (4 * far + 2 * E + 3 * k + 64) * U
    d = np.abs(scale * dw[live])
    if renorm:
        p = o.weights(x, ids[live], score, True, 1.0)
        term = p * (d + (d * p).sum())
    else:
        term = s[ids[live]] * d
    np.add.at(out, ids[live], term)
    if score == o.SOFTMAX and not renorm:
        out += s * term.sum()
    out = rel * out + TINY
    if bf16:
        out = out * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(o.grad(x, ids, dw, score, renorm, scale)) + 2.0 ** -134
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [(o.SOFTMAX, False), (o.SOFTMAX, True), (o.SIGMOID, False),
                                          (o.SIGMOID, True)])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gradient(T, E, k, score, renorm, dtype):
    x = logits(T, E, dtype, 7 * E + k)
    x[torch.rand(T, E, generator=torch.Generator().manual_seed(E + 1)) < 0.1] = -INF
    x[T // 2, : E // 2] = -INF
    ids = np.stack([o.choose(r, k, score) for r in x.double().numpy()])
    rng = np.random.default_rng(k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dw[ids < 0] = np.nan  # slots without an expert are not looked at
    got = run_grad(x, ids, dw, score, renorm, 2.5, E + 1)
    for t, row in enumerate(x.double().numpy()):
        want = o.grad(row, ids[t], dw[t].astype(np.float64), score, renorm, 2.5)
        e = grad_bound(row, ids[t], np.nan_to_num(dw[t].astype(np.float64)), score, renorm, 2.5, dtype == torch.bfloat16)
        assert (np.abs(got[t] - want) <= e).all(), (t, np.abs(got[t] - want).max(), e.max())


@pytest.mark.parametrize("score,renorm", [(o.SOFTMAX, False), (o.SOFTMAX, True), (o.SIGMOID, False),
                                          (o.SIGMOID, True)])
def test_gradient_of_odd_rows(score, renorm):
    """No expert, experts out of range, one named twice, sigmoids that are nothing in FP32."""
    E = 70
    x = logits(6, E, torch.float32, 1)
    ids = np.array([[-1, -1, -1], [3, 70, -5], [4, 4, 4], [69, 0, 64], [1, 2, 3], [1 << 30, 5, 6]], np.int32)
    x[0], x[4] = -INF, -150.0
    dw = np.random.default_rng(0).standard_normal((6, 3)).astype(np.float32)
    got = run_grad(x, ids, dw, score, renorm, 1.0, E)
    for t, row in enumerate(x.double().numpy()):
        want = o.grad(row, ids[t], dw[t].astype(np.float64), score, renorm, 1.0)
        e = grad_bound(row, ids[t], dw[t].astype(np.float64), score, renorm, 1.0, False)
        assert (np.abs(got[t] - want) <= e).all(), (t, got[t], want)
    assert (got[0] == 0).all()


@pytest.mark.parametrize("score,renorm", [(o.SOFTMAX, False), (o.SOFTMAX, True), (o.SIGMOID, False),
                                          (o.SIGMOID, True)])
def test_gradient_against_differences_of_the_kernel(score, renorm):
    """Central differences of route's own weights with h = 2^-6. Their error: h^2 / 6 times a third derivative, which
    for these functions is at most 6 |dw| in all (each derivative of a score or share is a sum of at most six products
    of numbers below one), and the weights' rounding over h."""
    T, E, k = 3, 24, 4
    x = logits(T, E, torch.float32, 11, 1.0)
    ids, w = run(x, k, score, renorm=renorm)
    dw = np.random.default_rng(1).standard_normal((T, k)).astype(np.float32)
    got = run_grad(x, ids, dw, score, renorm, 1.0, E)
    h = 2.0 ** -6
    mass = np.abs(dw).sum(1)
    for e in range(E):
        f = []
        for sign in (1, -1):
            y = x.clone()
            y[:, e] += sign * h
            at, w = run(y, k, score, renorm=renorm)
            # the same experts' weights, wherever the order has put them
            same = [sorted(a) == sorted(b) for a, b in zip(at.tolist(), ids.tolist())]
            f.append([(sum(w[t][at[t].tolist().index(i)] * float(d) for i, d in zip(ids[t], dw[t])))
                      if same[t] else None for t in range(T)])
        for t in range(T):
            if f[0][t] is not None and f[1][t] is not None:
                err = mass[t] * (6 * h * h / 6 + (E + 64) * U / h)
                assert abs((f[0][t] - f[1][t]) / (2 * h) - got[t, e]) <= err, (t, e)
