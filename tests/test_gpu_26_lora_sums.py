"""The sums x A^T enter the second product of tq_lora whole: differences of sums of 24 bits come out exact.

Every x A^T here is a whole number below 2^24 made of three exact products, B subtracts neighbouring ranks, and the
differences, with the base, stay below 2^8: all partial sums are whole numbers of at most 24 bits, so the result has no
rounding at all, in either type.  Sums held in 16 bits (two numbers of bf16) or 22 give other values.
"""
import numpy as np
import pytest

from gpu_common import log, require_gpu
from moe_common import DT, to_dev, values

pytestmark = pytest.mark.gpu


def case(T, N, r, L, seed):
    """x [T, 64], base [T, N], A [L, r, 64], B [L, N, r], ids [T] and what must come out, all fp64 and whole."""
    rng = np.random.default_rng(seed)
    K = 64
    x = np.zeros((T, K))
    x[:, 0], x[:, 17], x[:, 63] = 256.0, 1.0, 1.0
    first = rng.integers(1 << 16, 1 << 24, (L, r // 2)) - 128
    sums = np.stack([first, first - rng.integers(-100, 101, (L, r // 2))], -1).reshape(L, r)
    A = np.zeros((L, r, K))
    A[:, :, 0], A[:, :, 17], A[:, :, 63] = (sums >> 16) * 256, ((sums >> 8) & 255) * 256, sums & 255
    B = np.zeros((L, N, r))
    pair = rng.integers(0, r // 2, (L, N))
    for l in range(L):
        B[l, np.arange(N), 2 * pair[l]], B[l, np.arange(N), 2 * pair[l] + 1] = 1.0, -1.0
    base = rng.integers(-100, 101, (T, N)).astype(np.float64)
    ids = rng.integers(0, L, T).astype(np.int32)
    diff = (sums[:, 0::2] - sums[:, 1::2])[np.arange(L)[:, None], pair]
    return x, base, A, B, ids, base + diff[ids]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T, N, r", [(1, 40, 8), (1, 41, 16), (20, 72, 24), (20, 40, 32), (50, 40, 64), (9, 64, 136), (300, 64, 64),
                                     (2100, 40, 16), (2100, 64, 32), (2100, 41, 16), (2100, 41, 32), (2100, 41, 64), (2100, 40, 104),
                                     (30, 48, 104), (2050, 24, 256)])
def test_differences_of_long_sums(T, N, r, dt):
    import torch
    import bit_weight_only_tq_amd as tq
    log(f"lora whole sums T={T} N={N} r={r} {dt}")
    dev = require_gpu()
    x, base, A, B, ids, want = case(T, N, r, 3, T + N + r)
    d = [to_dev(v, dev, dt) for v in (x, base, A, B)]
    for host, t in zip((x, base, A, B), d):
        assert np.array_equal(values(t), host), f"not whole in {DT[dt]}"
    got = tq.tq_lora(*d, to_dev(ids, dev))
    torch.cuda.synchronize()
    assert np.array_equal(values(got), want)
