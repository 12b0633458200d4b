"""Sampling of one token from a row of logits, in fp64, by sorting the row.

``sample`` is the definition: rank by (logit, lowest index), keep a prefix of
the ranking (top-k, min-p, top-p), draw by the running weight in index order.
"""

import math

import numpy as np


def kept(row, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """-> (indices of the kept tokens in rank order, their weights); empty without a logit above -inf."""
    x = np.where(np.isnan(row), -np.inf, np.asarray(row, dtype=np.float64))
    V = x.size
    order = np.lexsort((np.arange(V), -x))
    top = x[order[0]]
    if top == -np.inf:
        return order[:0], np.zeros(0)
    if not temperature > 0:
        return order[:1], np.ones(1)
    with np.errstate(over="ignore", invalid="ignore"):
        w = np.where(x[order] == top, 1.0, np.exp((x[order] - top) / temperature))
    w[x[order] == -np.inf] = 0.0
    n = V if top_k <= 0 or top_k > V else int(top_k)
    n = max(1, min(n, int(np.count_nonzero(w >= min_p)))) if min_p <= 1 else 1
    if not top_p >= 1:
        before = np.concatenate([[0.0], np.cumsum(w[:n])[:-1]])
        n = max(1, int(np.count_nonzero(before < top_p * math.fsum(w[:n]))))
    return order[:n], w[:n]


def sample(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """-> (token, logprob); (-1, -inf) without a logit above -inf."""
    order, w = kept(row, temperature, top_k, top_p, min_p)
    if order.size == 0:
        return -1, -math.inf
    by_index = np.argsort(order)
    idx, w = order[by_index], w[by_index]
    idx, w = idx[w > 0], w[w > 0]
    total = math.fsum(w)
    u = min(max(u, 0.0), 1.0 - 2.0 ** -24) if u == u else 0.0
    run = np.cumsum(w)
    i = min(int(np.searchsorted(run, u * total, side="right")), idx.size - 1)
    return int(idx[i]), math.log(w[i] / total)
