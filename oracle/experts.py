"""Experts and adapters in fp64: routing, products grouped by expert, their weighted sum, low-rank updates.

Each function is the definition, row by row; the products also give the sum of
their terms' magnitudes, which error bounds are stated in.
"""

import numpy as np


def route(logits, k, renormalize=True):
    """-> (experts [T, k], weights [T, k], offsets [E + 1], rows [T k], places [T, k])."""
    x = np.asarray(logits, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    T, E = x.shape
    experts, weights = np.full((T, k), -1, np.int64), np.zeros((T, k))
    members = [[] for _ in range(E + 1)]
    for t in range(T):
        order = np.lexsort((np.arange(E), -x[t]))
        top = x[t, order[0]]
        with np.errstate(invalid="ignore"):
            w = np.where(x[t] == top, 1.0, np.exp(x[t] - top))
        w[x[t] == -np.inf] = 0.0
        chosen = [e for e in order[:k] if x[t, e] > -np.inf]
        total = sum(w[e] for e in chosen) if renormalize else w.sum()
        for j in range(k):
            if j < len(chosen):
                experts[t, j], weights[t, j] = chosen[j], w[chosen[j]] / total
                members[chosen[j]].append(t * k + j)
            else:
                members[E].append(t * k + j)
    rows = np.array([p for m in members for p in m], np.int64)
    offsets = np.concatenate([[0], np.cumsum([len(m) for m in members[:E]])]).astype(np.int64)
    places = np.full(T * k, -1, np.int64)
    places[rows[:offsets[E]]] = np.arange(offsets[E])
    return experts, weights, offsets, rows, places.reshape(T, k)


def product(A, W, offsets, rows=None, bias=None):
    """A [T, K], W [E, N, K] -> (C [P, N] with NaN where no expert has the row, sums of magnitudes)."""
    A, W = np.asarray(A, np.float64), np.asarray(W, np.float64)
    P = len(rows) if rows is not None else A.shape[0]
    fan = P // A.shape[0]
    C, mag = np.full((P, W.shape[1]), np.nan), np.zeros((P, W.shape[1]))
    for e in range(W.shape[0]):
        for p in range(offsets[e], offsets[e + 1]):
            a = A[rows[p] // fan if rows is not None else p]
            C[p] = W[e] @ a
            mag[p] = np.abs(W[e]) @ np.abs(a)
            if bias is not None:
                C[p] += bias[e]
                mag[p] += np.abs(bias[e])
    return C, mag


def gated(C):
    """gate / (1 + exp(-gate)) * up of the two halves of a row."""
    g, u = np.split(C, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def combine(y, places, weights, add=None):
    T, k = places.shape
    out = np.zeros((T, y.shape[1])) if add is None else np.array(add, np.float64)
    for t in range(T):
        for j in range(k):
            if 0 <= places[t, j] < y.shape[0]:
                out[t] += float(weights[t, j]) * y[places[t, j]]
    return out


def lora(x, base, A, B, ids, scale=None):
    """-> (out [T, N], x A^T [T, r] of each row's adapter)."""
    out = np.array(base, np.float64)
    h = np.zeros((x.shape[0], A.shape[1]))
    for t, l in enumerate(ids):
        if 0 <= l < A.shape[0]:
            h[t] = A[l] @ x[t]
            out[t] += (1.0 if scale is None else float(scale[l])) * (B[l] @ h[t])
    return out, h
