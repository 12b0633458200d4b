"""Inputs and error bounds of the experts' and adapters' tests.

Bounds count what the operators round.  A product sums K exact products in fp32: each of at most K + 32 additions (the
matrix cores' own, the waves' and the groups') is off by at most 2^-23 of a partial sum, and no partial sum passes the sum
of the terms' magnitudes, so the sum is off by (K + 32) 2^-23 of that.  (A half step would be 2^-24; the matrix cores may
cut instead of rounding.)  Where a group's scale multiplies its sum, that is one more such rounding a group, counted in the
32 and the K.  The result is then rounded once to its type: half a step, u = eps / 2 of the value, and half the smallest
subnormal.
"""
import numpy as np

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}
DT = {"f16": "float16", "bf16": "bfloat16"}


def sum_bound(K, mag):
    return (K + 32) * 2.0 ** -23 * mag


def rounded(dt, bound, out):
    """The bound of a value that is off by `bound` and then rounded to dt."""
    return bound * (1 + U[dt]) + U[dt] * np.abs(out) + TINY[dt]


def gated_bound(K, C, mag):
    """gate / (1 + exp(-gate)) * up of sums that are off by sum_bound: the first factor's slope is below 1.1, exp, the sum, the
    quotient and the product are each within 4 steps of 2^-24 of the value; exp(-gate) is off by |gate| 2^-24 besides."""
    g, u = np.split(C, 2, axis=1)
    dg, du = np.split(sum_bound(K, mag), 2, axis=1)
    with np.errstate(over="ignore"):
        s = g / (1.0 + np.exp(-g))
    return 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + (16 + np.abs(g)) * 2.0 ** -24 * np.abs(s * u) + 2.0 ** -126


def experts(fmt, E, N, K, rng, zeros=False):
    """-> (dict of packed numpy arrays, fp64 weights [E, N, K])."""
    if fmt == "ternary":
        c = rng.integers(0, 3, (E, N, K // 4, 4))
        scale = (rng.random((E, N)) * 0.03 + 0.005).astype(np.float16)
        W = (c.reshape(E, N, K) - 1) * scale.astype(np.float64)[:, :, None]
        codes = (c * np.array([1, 4, 16, 64])).sum(-1).astype(np.uint8)
        return {"w": codes, "scale": scale, "zeros": None}, W
    q = rng.integers(0, 16, (E, N, K // 8, 8))
    scale = (rng.random((E, N, K // 128)) * 0.01 + 0.001).astype(np.float16)
    z = rng.integers(0, 16, (E, N, K // 128)).astype(np.uint8) if zeros else np.full((E, N, K // 128), 8, np.uint8)
    W = (q.reshape(E, N, K // 128, 128) - z.astype(np.int64)[..., None]) * scale.astype(np.float64)[..., None]
    words = (q.astype(np.uint64) << (4 * np.arange(8, dtype=np.uint64))).sum(-1).astype(np.uint32).view(np.int32)
    return {"w": words, "scale": scale, "zeros": z if zeros else None}, W.reshape(E, N, K)


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def to_dev(x, dev, dt=None):
    import torch
    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.to(getattr(torch, DT[dt])) if dt else t).to(dev)


def values(t):
    return t.double().cpu().numpy()


def assert_within(got, want, bound, label):
    """got within bound of want; equal where want is not finite."""
    got, want = np.asarray(got), np.asarray(want)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), f"{label}: values that are not finite differ"
    err = np.abs(got[fine] - want[fine])
    b = np.broadcast_to(bound, want.shape)[fine]
    bad = ~(err <= b)
    if bad.any():
        i = int(np.argmax(np.where(bad, np.where(np.isfinite(err), err, np.inf), -1)))
        raise AssertionError(f"{label}: {bad.sum()} of {bad.size} outside; worst {got[fine][i]} for {want[fine][i]}, bound {b[i]}")
