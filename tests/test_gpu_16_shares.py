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


@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
def test_both_kernels_in_one_call(dt, D):
    """A chunk beside decoding requests over more than 12288 keys: two launches, one workspace, captured as well."""
    import torch
    import bit_weight_only_tq_amd as tq
    from gpu_common import require_gpu
    dev = require_gpu()
    qn, kv = [1, 90, 0, 16, 1], [13000, 300, 5, 2000, 50]
    c, got = _go(qn, kv, 2, 2, D, 16, dt)
    ws = tq.new_workspace(tq.tq_paged_attention_workspace_bytes(sum(qn), 2, 2, D, 5, 90, 13000), dev)
    d = [t.to(dev) for t in (c.q, c.k, c.v, c.table, c.cu, c.kv)]
    out = torch.empty_like(got[0])
    call = lambda: tq.tq_paged_attention(*d, 90, 13000, out=out, return_lse=True, workspace=ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, lse = call()
    for i in range(4):
        out.fill_(0), lse.fill_(0)
        torch.randn(1000, device=dev).sum()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got[0]) and torch.equal(lse, got[1]), f"replay {i}"
    assert int(ws[:tq.TQ_WORKSPACE_FLAG_BYTES].count_nonzero()) == 0
    if D == 64:  # with a window that leaves little to read, one kernel does it all
        c.check(c.run(1000, 4), 1000, 4)
        c.check(c.run(12500, 4), 12500, 4)
