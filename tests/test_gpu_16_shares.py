"""Even shares of decoding requests: batches and lengths at which the division of the work changes, against the fp64
oracle (tolerances derived in test_gpu_11_attention)."""
import pytest

from test_gpu_11_attention import Case, _go

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [1, 2, 63, 255, 256, 257, 300])
@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
def test_batches(B, dt, D):
    """Ragged lengths, requests that rest, have no keys, or bring a few tokens."""
    kv = [(0, 1, 700, 33, 257, 90, 1500, 31, 64, 5)[(7 * b) % 10] for b in range(B)]
    qn = [(1, 1, 0, 2, 1, 4, 1)[b % 7] for b in range(B)]
    if sum(qn) == 0 or max(kv) == 0:
        qn[0], kv[0] = 1, 600
    _go(qn, kv, 4, 1, D, 16, dt)


def test_more_requests_than_shares_hold():
    _go([1] * 1100, [(37 * b) % 300 + 1 for b in range(1100)], 2, 1, 64, 16, "bf16")


@pytest.mark.parametrize("kv", [[33], [257], [320, 320], [20000, 1, 1, 1], [5000, 0, 9000, 256, 2048]])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (16, 1), (8, 8)])
def test_lengths(kv, Hq, Hkv):
    """Requests in one share, in many, and shares of many requests; the same bits each time."""
    import torch
    c, got = _go([1] * len(kv), kv, Hq, Hkv, 128, 64, "bf16")
    again = c.run()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("qn", [[16, 1], [17, 1], [64, 3], [65, 16, 17, 1]])
def test_either_kernel(qn):
    """Row counts at which a request changes from one kernel to the other, one head a group."""
    _go(qn, [n + 600 for n in qn], 1, 1, 64, 16, "f16")
    _go(qn, [n + 600 for n in qn], 1, 1, 128, 16, "f16", 100, 5)


def test_small_workspace_means_none():
    """A workspace too small for the partial results: one workgroup a request, within tolerance."""
    import torch
    from gpu_common import require_gpu
    c = Case([1, 1], [3000, 100], 8, 2, 128, 16, "bf16")
    c.check(c.run(workspace=torch.zeros(20000, dtype=torch.uint8, device=require_gpu())))
