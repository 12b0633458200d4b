"""Paged attention where most of the weight is in many keys of small weight each, behind a key that outweighs every one
of them, against the fp64 oracle.

The weights are rounded to the cache's type before the product with the values.  fp16 has its full step down to 2^-14
and none below 2^-25, so weights are held 2^7 times larger than the largest key's being 1 would have them: a weight of
r times the largest is off by half a step of 2^-11 r, or by 2^-25 / 2^7 = 2^-32 at most where it is smaller than 2^-21.
The other terms are the ones derived in test_gpu_11_attention.
"""
import numpy as np
import pytest
import torch

import oracle.attention as OA
from gpu_common import log
from test_gpu_11_attention import Case, _bounds, _share

pytestmark = pytest.mark.gpu


def _bound(ref, D, n, dt):
    if dt == torch.bfloat16:
        return _bounds(ref, D, n, dt)[0]
    half = torch.finfo(dt).eps / 2
    e = (D + 14) * 2.0 ** -23 * ref["smag"] + 2.0 ** -21
    acc = (n / 32 + 64) * 2.0 ** -23
    out = ref["mag"] * (2 * e[..., None] + half + 2 * acc) + 2.0 ** -32 * ref["wmax"]
    return out + half * (np.abs(ref["out"]) + out) + 2.0 ** -25


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("below", [9.0, 14.5, 17.5])
@pytest.mark.parametrize("qn", [[1], [1, 3], [20], [140]])
def test_many_small_weights(qn, below, D, dt):
    """The first key's score is `below` above all others'; its value is 0 and theirs 1, so the output is their share."""
    log(f"small weights qn={qn} below={below} D={D} {dt}")
    kv = [6001 if n == 140 else 20001 for n in qn]
    c = Case(qn, kv, 1, 1, D, 64, dt, spare=1)
    c.q.zero_(), c.k.zero_()
    c.q[..., 0] = 1.0
    c.v.fill_(1.0)
    for b in range(len(qn)):
        first = int(c.table[b, 0])
        c.k[first, :, 0, 0] = below
        c.v[first, :, 0] = 0.0
    f = lambda t: t.double().numpy()  # noqa: E731
    ref = OA.attend(f(c.q), f(c.k), f(c.v), c.table.numpy(), c.cu.tolist(), c.kvl, 1.0)
    tol = _bound(ref, D, max(kv), c.dt)
    for ws in ("auto", None):
        out, lse = [x.double().cpu().numpy() for x in c.run(scale=1.0, workspace=ws)]
        err = _share(np.abs(out - ref["out"]), tol)
        assert err <= 1, f"out {err} of its tolerance"
        assert np.abs(lse - ref["lse"]).max() <= 2.0 ** -21 + (max(kv) / 32 + 64) * 2.0 ** -23 + 2.0 ** -22 * below + 2.0 ** -20


@pytest.mark.parametrize("value", [6.0e4, -3.0e4])
@pytest.mark.parametrize("qn", [[1], [40]])
def test_large_values(value, qn):
    """fp16 values at the type's upper end with scores that rise and fall along the keys: nothing overflows on the way."""
    log(f"large values {value} qn={qn}")
    c = Case(qn, [3000], 1, 1, 64, 16, "f16")
    c.v.fill_(value)
    for j in range(3000):
        c.k[int(c.table[0, j // 16]), 0, j % 16] = (1 if j < 1500 else -1) * (j % 1500) * 0.01
    c.q = c.q.abs()
    c.check(c.run())
    c.check(c.run(workspace=None))
