"""The distillation loss and its gradient written out in 64 bits (test
infrastructure), with how far a kernel that streams its sums in fp32 may be
from them."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24


def valid(ids, t, V):
    return (ids >= 0) & (ids < V) & ~np.isneginf(t)


def row(x, ids, t, tau, g):
    """(loss, tolerance of the loss, gradient [V], tolerance of the gradient) of one row."""
    x, t = np.asarray(x, np.float64), np.asarray(t, np.float64)
    V = x.size
    ok = valid(ids, t, V)
    grad, gtol = np.zeros(V), np.zeros(V)
    if not ok.any():
        return 0.0, 0.0, grad, gtol
    if np.isneginf(x).all():
        return np.inf, 0.0, grad, gtol
    if np.isnan(x).any() or np.isposinf(x).any():
        return np.nan, 0.0, np.full(V, np.nan), gtol
    ids, t = ids[ok], t[ok]
    d = (x - x.max()) / tau
    e = np.exp(d)
    z = e.sum()
    p = e / z
    u = (t - t.max()) / tau
    q = np.exp(u)
    q = q / q.sum()
    with np.errstate(divide="ignore", invalid="ignore"):
        logp = d - np.log(z)
        terms = np.where(q > 0, q * (np.log(q) - logp[ids]), 0.0)
    loss = tau * tau * terms.sum()
    # A weight 2^((x - m) kappa): the difference, kappa and their product are
    # rounded, the exponential is good to a step (2^-23).  The sum: every
    # thread adds V / 256 weights, rescaled at each of its V / 8192 turns, then
    # eight joins, each a product with a weight and an addition.
    big = np.where(np.isfinite(d), np.abs(d), 0.0)
    own = 3 * U32 * big + 2 * U32
    turns = V / 8192 + 10
    zrel = (p * own).sum() + (V / 256 + 3 * turns) * U32 + turns * (2 * U32 + 3 * U32 * big[p > 0].max())
    ltol = tau * tau * zrel
    scale = abs(g) * tau
    # past the weight: z itself, g tau, their quotient and the product are rounded
    gtol = scale * (p * (own + zrel + 5 * U32) + 2.0 ** -126)
    grad = g * tau * p
    for j, i in enumerate(ids):
        grad[i] -= g * tau * q[j]
        gtol[i] += scale * 3 * U32 * q[j]  # the list's sum and the entry's weight in fp32, the result in fp32
        gtol[i] += 2 * U32 * abs(grad[i])
    return loss, ltol * 1.001, grad, gtol * 1.001


def block(x, ids, t, tau, g):
    """The same of [B, M, ...] arrays."""
    B, M, V = x.shape
    loss, ltol = np.zeros((B, M)), np.zeros((B, M))
    grad, gtol = np.zeros((B, M, V)), np.zeros((B, M, V))
    for b in range(B):
        for m in range(M):
            loss[b, m], ltol[b, m], grad[b, m], gtol[b, m] = row(x[b, m], ids[b, m], t[b, m], tau, g[b, m])
    return loss, ltol, grad, gtol
