"""Attention of new tokens over a paged cache, in fp64, one query row at a time.

``attend`` gathers the keys a row sees (causal, window, sinks, pages that
exist) before it computes anything, so what a row does not see cannot touch
it.  Beside the results it returns, for the tolerance, the weighted mean of
|v| and a bound on the rounding of the row's scores.
"""

import numpy as np


def visible(p, kv, window, sinks):
    """Indices of the keys position p sees among kv keys."""
    j = np.arange(min(max(p, -1) + 1, kv))
    return j if not window else j[(p - j < window) | (j < sinks)]


def attend(q, k_cache, v_cache, table, cu, kv, scale, window=0, sinks=0):
    """-> dict of out [T, Hq, D], lse [T, Hq], mag (sum of weight * |v|), smag (bound of sum |q k| and |score|), wmax.

    Rows of no request are nan (not written)."""
    T, Hq, D = q.shape
    pages, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    out, mag = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D))
    lse, smag, wmax = np.full((T, Hq), np.nan), np.zeros((T, Hq)), np.zeros((T, Hq, D))
    for b in range(len(kv)):
        n = int(cu[b + 1] - cu[b])
        for i in range(n):
            j = visible(int(kv[b]) - n + i, int(kv[b]), window, sinks)
            j = j[j // page < table.shape[1]]
            ids = table[b, j // page]
            ok = (ids >= 0) & (ids < pages)
            j, ids = j[ok], ids[ok]
            for h in range(Hq):
                t = int(cu[b]) + i
                if j.size == 0:
                    out[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                x = q[t, h].astype(np.float64)
                k = k_cache[ids, h // G, j % page].astype(np.float64)
                v = v_cache[ids, h // G, j % page].astype(np.float64)
                s = (k @ x) * scale
                m = s.max()
                w = np.exp(s - m)
                z = w.sum()
                with np.errstate(invalid="ignore"):
                    out[t, h] = (w[:, None] * v).sum(0) / z
                    mag[t, h] = (w[:, None] * np.abs(v)).sum(0) / z
                    wmax[t, h] = np.abs(v).max(0) * j.size / z
                lse[t, h] = m + np.log(z)
                smag[t, h] = (np.abs(k) @ np.abs(x)).max() * abs(scale)
    return {"out": out, "lse": lse, "mag": mag, "smag": smag, "wmax": wmax}
