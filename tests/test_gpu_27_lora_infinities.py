"""Infinite activations and weights in tq_lora: with A of one sign and each row of B of one sign, the result is +inf or -inf.

Ranks that fill the matrix tiles and ranks that do not must agree, and so must few rows and prompts: no rank that is not
there may bring a NaN into the sums.
"""
import numpy as np
import pytest

import oracle.experts as OE
from gpu_common import log, require_gpu
from moe_common import DT, assert_within, to_dev, values
from test_gpu_24_lora import bound_of

pytestmark = pytest.mark.gpu


def signed(T, K, N, L, r, dt, seed):
    """x, base, A > 0, B of one sign a row; ids; scale > 0: device tensors and their fp64 values."""
    import torch
    dev = require_gpu()
    rng = np.random.default_rng(seed)
    sign = rng.choice([-1.0, 1.0], (L, N, 1))
    host = [rng.standard_normal((T, K)), rng.standard_normal((T, N)), (rng.random((L, r, K)) + 0.25) / K, sign * (rng.random((L, N, r)) + 0.25)]
    d = [torch.from_numpy(v).to(getattr(torch, DT[dt])).to(dev) for v in host]
    ids = rng.integers(0, L, T).astype(np.int32)
    scale = (rng.random(L) + 0.5).astype(np.float32)
    return d, ids, scale


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T, N", [(1, 40), (7, 41), (40, 72), (300, 72), (300, 41), (2100, 72), (2100, 41)])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 48, 64, 72, 136, 256])
def test_infinite_activations(T, N, r, dt):
    import torch
    import bit_weight_only_tq_amd as tq
    log(f"lora infinities T={T} N={N} r={r} {dt}")
    K = 136
    (x, base, A, B), ids, scale = signed(T, K, N, 2, r, dt, T + N + r)
    inf = float("inf")
    x[0, 3] = inf
    if T > 1:
        x[T // 2, K - 1] = -inf        # in the columns behind the last whole step
        x[T - 1, 64] = x[T - 1, 100] = inf
    dev = x.device
    got = tq.tq_lora(x, base, A, B, to_dev(ids, dev), scale=to_dev(scale, dev))
    torch.cuda.synchronize()
    h = [values(x), values(base), values(A), values(B), ids, scale.astype(np.float64)]
    want = OE.lora(*h)[0]
    rows = sorted({0, T // 2, T - 1})
    assert np.isinf(want[rows]).all()
    assert np.array_equal(values(got)[rows], want[rows])
    keep = np.setdiff1d(np.arange(T), rows)
    if len(keep):
        h = [h[0][keep], h[1][keep], h[2], h[3], ids[keep], h[5]]
        want, bound = bound_of(h, dt, K, r)
        assert_within(values(got)[keep], want, bound, "rows beside them")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T, N", [(1, 40), (40, 41), (300, 72), (2100, 72), (2100, 41)])
@pytest.mark.parametrize("r", [8, 16, 24, 64, 104, 256])
def test_infinite_weights(T, N, r, dt):
    """Infinities in columns of B, and in a rank of one adapter's A, reach their columns and rows and no others."""
    import torch
    import bit_weight_only_tq_amd as tq
    log(f"lora infinite weights T={T} N={N} r={r} {dt}")
    K = 136
    (x, base, A, B), ids, scale = signed(T, K, N, 3, r, dt, T + N + r)
    x = x.abs() + 0.125
    ids[0] = 0
    for n, j in ((0, 0), (5, r - 1), (N - 1, 3)):
        B[:2, n, j] = torch.sign(B[:2, n, j]) * float("inf")
    A[1, 4, 9] = float("inf")
    dev = x.device
    got = tq.tq_lora(x, base, A, B, to_dev(ids, dev), scale=to_dev(scale, dev))
    torch.cuda.synchronize()
    h = [values(x), values(base), values(A), values(B), ids, scale.astype(np.float64)]
    want = OE.lora(*h)[0]
    assert np.isinf(want[ids == 0][:, [0, 5, N - 1]]).all() and np.isinf(want[ids == 1]).all() and np.isfinite(want[ids == 2]).all()
    assert np.isfinite(np.delete(want[ids == 0], [0, 5, N - 1], 1)).all()
    wide = np.isinf(want)
    assert np.array_equal(values(got)[wide], want[wide])
    h[2], h[3] = (np.where(np.isinf(v), 0.0, v) for v in h[2:4])  # finite results take no infinite value
    rest, bound = bound_of(h, dt, K, r)
    assert_within(values(got)[~wide], rest[~wide], bound[~wide], "the others")
