"""Sampling straight from its definition, row by row in 64 bits (numpy)."""

import numpy as np


def distribution(x, t=1.0, k=0, p=1.0, least=0.0):
    """Token ids and weights that may come, ids rising; greedy and empty rows: one id or none, weight 1."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64)) + 0.0
    top = x.max()
    if top == -np.inf:
        return np.array([], int), np.array([])
    if not t > 0:
        return np.flatnonzero(x == top)[:1], np.ones(1)

    def weights(v):
        if top == np.inf:
            return (v == np.inf).astype(np.float64)
        w = np.exp((v - top) / t) if np.isfinite(t) else np.ones_like(v)
        return np.where(v == -np.inf, 0.0, w)

    ids = np.lexsort((np.arange(x.size), -x))
    if 0 < k < x.size:
        ids = ids[:k]
    w = weights(x[ids])
    if p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        keep = before < p * w.sum()
        keep[0] = True
        ids, w = ids[keep], w[keep]
    if least > 0:
        keep = w >= min(least, 1.0)
        ids, w = ids[keep], w[keep]
    order = np.argsort(ids)
    return ids[order], w[order]


def sample(x, u, **kw):
    """Token and its probability."""
    ids, w = distribution(x, **kw)
    if ids.size == 0:
        return -1, 0.0
    u = 0.0 if np.isnan(u) else min(max(u, 0.0), 1.0 - 2.0 ** -24)
    sums = np.cumsum(w)
    at = int(np.searchsorted(sums, u * sums[-1], side="right"))
    return int(ids[at]), w[at] / sums[-1]


def border(x, u, **kw):
    """How near u is to a border of the distribution over how near two right answers can be: a weight is a multiple
    of 2^-S of the largest (S = min(51, 62 - log2 vocab)), so a border lies off by at most vocab 2^-(S+1) of that, twice
    that where tiles are rounded too, and 2^-38 of the sum for the exponentials (good to 2^-39). Below 1 either neighbour is right.
    Equal weights are whole multiples: nothing is lost."""
    ids, w = distribution(x, **kw)
    if ids.size == 0 or (w == w[0]).all():
        return np.inf
    shift = min(51, 62 - max(0, int(np.ceil(np.log2(x.size)))))
    off = 2 * x.size * 2.0 ** -(shift + 1) * w.max() / w.sum() + 2.0 ** -38
    return float(np.abs(np.cumsum(w) / w.sum() - u).min()) / off
