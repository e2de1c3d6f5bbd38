"""Routing of tokens to experts and their rows' way there and back. TEST INFRASTRUCTURE ONLY.

Written from the definition in float64, a token at a time. Pinned by
tests/test_oracle_routing.py (worked examples, gradients against central differences).
"""
from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1


def log_scores(x, score):
    """log of a row's scores; x: float64[E], without NaN."""
    x = np.asarray(x, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        if score == SIGMOID:
            return np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))
        top = x.max()
        if top == -np.inf:
            return np.full_like(x, -np.inf)
        return x - top - np.log(np.exp(x - top).sum())


def choose(x, k, score, bias=None, groups=1, top_groups=1, best=1):
    """Experts of one row, in order; -1 where none is left. None for a row that has no scores."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or (score == SOFTMAX and (x == np.inf).any()):
        return None
    if bias is None and best == 1:
        c = x.copy()
    else:
        c = np.exp(log_scores(x, score)) + (0.0 if bias is None else np.asarray(bias, np.float64))
    c[(x == -np.inf) | np.isnan(c)] = -np.inf
    per = len(x) // groups
    if groups > 1:
        total = np.full(groups, -np.inf)
        for g in range(groups):
            v = sorted((float(u) for u in c[g * per:(g + 1) * per] if u > -np.inf), reverse=True)[:best]
            if v:
                total[g] = sum(v)
        kept = [g for g in sorted(range(groups), key=lambda g: (-total[g], g)) if total[g] > -np.inf][:top_groups]
        for g in range(groups):
            if g not in kept:
                c[g * per:(g + 1) * per] = -np.inf
    ids = [e for e in sorted(range(len(x)), key=lambda e: (-c[e], e)) if c[e] > -np.inf][:k]
    return np.array(ids + [-1] * (k - len(ids)))


def weights(x, ids, score, renormalise, scale):
    """The weights of one row's slots."""
    ids = np.asarray(ids)
    logs = log_scores(x, score)
    w = np.zeros(len(ids))
    live = ids >= 0
    if not live.any():
        return w
    chosen = logs[ids[live]]
    if renormalise:
        # (A row whose chosen logits are all -inf has no shares.)
        s = np.exp(chosen - chosen.max()) if chosen.max() > -np.inf else np.zeros(len(chosen))
        w[live] = s / s.sum() if s.sum() > 0 else 0.0
    else:
        w[live] = np.exp(chosen)
    return scale * w


def grad(x, ids, dw, score, renormalise, scale):
    """d sum_j dw_j w_j / dx of one row, by the chain rule on the formulas."""
    x, ids, dw = np.asarray(x, np.float64), np.asarray(ids), np.asarray(dw, np.float64)
    out = np.zeros(len(x))
    live = (ids >= 0) & (ids < len(x))
    ids, dw = ids[live], scale * dw[live]
    if not len(ids):
        return out
    s = np.exp(log_scores(x, score))
    if renormalise:
        p = weights(x, ids, score, True, 1.0)
        ds = p * (dw - (dw * p).sum())  # d / d log s
    else:
        ds = s[ids] * dw
    if score == SIGMOID:
        ds = ds * np.exp(log_scores(-x[ids], SIGMOID))  # d log s / dx = 1 - s
        np.add.at(out, ids, ds)
    else:
        np.add.at(out, ids, ds)
        out -= s * (0.0 if renormalise else ds.sum())
    return out


def order(expert, G):
    """offsets, position, order of slots by expert (stable)."""
    expert = np.asarray(expert).reshape(-1)
    rows = [s for g in range(G) for s in np.flatnonzero(expert == g)]
    position = np.full(len(expert), -1)
    position[rows] = np.arange(len(rows))
    offsets = np.concatenate([[0], np.cumsum([int((expert == g).sum()) for g in range(G)])]).astype(int)
    return offsets, position, np.array(rows + [-1] * (len(expert) - len(rows)), dtype=int)


def combine(y, position, weight, c=None, beta=0.0):
    """(C, sum of |terms|); position: T x k, weight: T x k or None."""
    y, position = np.asarray(y, np.float64), np.asarray(position)
    weight = None if weight is None else np.asarray(weight, np.float64)
    T, k = position.shape
    out, mass = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            r = position[t, j]
            if 0 <= r < len(y):
                term = (1.0 if weight is None else float(weight[t, j])) * y[r]
                out[t] += term
                mass[t] += np.abs(term)
        if beta != 0.0:
            out[t] += beta * np.asarray(c, np.float64)[t]
            mass[t] += np.abs(beta * np.asarray(c, np.float64)[t])
    return out, mass


def combine_grad(d, y, position, weight):
    """(dY, rows written, dweight, sum of |products| of dweight)."""
    d, y, position = np.asarray(d, np.float64), np.asarray(y, np.float64), np.asarray(position)
    weight = None if weight is None else np.asarray(weight, np.float64)
    T, k = position.shape
    dy, written = np.zeros(y.shape), np.zeros(len(y), bool)
    dw, mass = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = position[t, j]
            if 0 <= r < len(y):
                dy[r] = (1.0 if weight is None else float(weight[t, j])) * d[t]
                written[r] = True
                dw[t, j] = (d[t] * y[r]).sum()
                mass[t, j] = np.abs(d[t] * y[r]).sum()
    return dy, written, dw, mass
