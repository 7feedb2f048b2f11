"""Sampling under a request's limits written out in 64 bits (test
infrastructure)."""
from __future__ import annotations

import math

import numpy as np


def row(x, u, T, k, p, m):
    """(token, probability, distance of the nearest border in units of the sum) of one row."""
    x = np.asarray(x, np.float64)
    V = x.size
    nan = np.isnan(x)
    if nan.any():
        return int(nan.argmax()), math.nan, 1.0
    top = x.max()
    if np.isneginf(top):
        return -1, 0.0, 1.0
    if not T >= 1e-5 or np.isposinf(top):
        return int((x == top).argmax()), 1.0, 1.0
    order = np.lexsort((np.arange(V), -x))
    order = order[~np.isneginf(x[order])]
    with np.errstate(over="ignore", under="ignore"):
        w = np.exp((x[order] - top) / T) if np.isfinite(T) else np.ones(order.size)
    if 0 < k < V:
        order, w = order[:k], w[:k]
    near = 1.0
    if m > 0:
        m = min(m, 1.0)
        apart = np.abs(w - m)
        near = min(near, apart[apart > 0].min(initial=1.0))
        n = max(int((w >= m).sum()), 1)
        order, w = order[:n], w[:n]
    total = math.fsum(w)
    if p < 1:
        upto = np.cumsum(w)
        before = np.concatenate([[0.0], upto[:-1]])
        near = min(near, np.abs(upto[:-1] - p * total).min(initial=total) / total)
        n = max(int((before < p * total).sum()), 1)
        order, w = order[:n], w[:n]
    total = math.fsum(w)
    by = np.argsort(order)
    upto = np.cumsum(w[by])
    target = min(max(u, 0.0), 1.0 - 2.0 ** -24) * total
    near = min(near, np.abs(upto[:-1] - target).min(initial=total) / total)
    i = min(int((upto <= target).sum()), order.size - 1)
    return int(order[by][i]), w[by][i] / total, near
