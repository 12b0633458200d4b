"""Offsets and rows that no routing writes: what a call may write, and what it must.

An expert's rows are its offsets held to [0, P].  A row of no expert stays as it was; a row of one expert alone is that
expert's product, or has values left as they were where the offsets name more than P rows in all; rows of several are not
looked at.
"""
import numpy as np
import pytest

import oracle.experts as OE
from gpu_common import log
from moe_common import assert_within, rounded, sum_bound, to_dev, values
from test_gpu_23_experts import FMTS, call, make

pytestmark = pytest.mark.gpu


def ranges(off, P):
    """[(first row, row behind the last)] of each expert."""
    lo = np.clip(np.asarray(off[:-1], np.int64), 0, P)
    return list(zip(lo, np.clip(np.maximum(off[1:], lo), 0, P)))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("E, rows, N, K", [(4, 8, 48, 256), (8, 300, 272, 640), (8, 700, 144, 640), (16, 3000, 48, 128)])
def test_rows_of_sound_experts(E, rows, N, K, fmt, dt):
    import torch
    log(f"experts {fmt} {dt} E={E} rows={rows} N={N} K={K} offsets of any values")
    d, h = make(fmt, E, N, K, [rows] * E, dt, 31, fan=2)
    dev, P = d["A"].device, h["P"]
    pairs = h["rows"].copy()
    pairs[3], pairs[9] = -7, 1 << 30
    held = np.clip(pairs, 0, P - 1)
    big = torch.full((P + 64, N), 77.0, dtype=d["A"].dtype, device=dev)
    sound = np.arange(E + 1, dtype=np.int64) * rows
    for change in ({2: 1 << 30}, {0: -5, E: P + 99}, {0: rows, 1: 0, E - 1: -1}, {1: P, 2: 0, E: P}, {2: rows, 3: rows}, {E: 3 * rows - 1},
                   {0: 5, E: P - 3}):
        off = sound.copy()
        for i, v in change.items():
            off[i] = v
        big.fill_(77.0)
        call(d["A"], d["packed"], to_dev(off.astype(np.int32), dev), rows=to_dev(pairs, dev), out=big[32:-32])
        torch.cuda.synchronize()
        assert (big[:32] == 77.0).all() and (big[-32:] == 77.0).all()
        got = values(big[32:-32])
        r = ranges(off, P)
        owners = np.zeros(P, np.int64)
        for lo, hi in r:
            owners[lo:hi] += 1
        assert (got[owners == 0] == 77.0).all(), "rows of no expert were written"
        whole = sum(hi - lo for lo, hi in r) <= P
        right = 0
        for e, (lo, hi) in enumerate(r):
            at = np.arange(lo, hi)[owners[lo:hi] == 1]
            if len(at) > 40:
                at = np.unique(np.r_[at[:6], at[-6:], at[:: len(at) // 28]])
            if not len(at):
                continue
            C, mag = OE.product(h["A"][held[at] // 2], h["W"][e:e + 1], np.array([0, len(at)]))
            bound = rounded(dt, sum_bound(K, mag), C)
            there = np.full(C.shape, True) if whole else got[at] != 77.0
            assert_within(got[at][there], C[there], bound[there], f"expert {e}")
            right += there.sum()
        assert right > 0 or not whole
