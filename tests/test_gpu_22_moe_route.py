"""Routing against the fp64 oracle: experts, offsets, rows and places are equal, weights within their rounding.

A weight is exp(x - max) over a sum: the difference is rounded once (2^-24 of it, so exp is off by |x - max| 2^-24), exp is
within 2 steps of 2^-24, the sum of E terms within E 2^-24 of itself, the quotient half a step.
"""
import numpy as np
import pytest

import oracle.experts as OE
from gpu_common import log, require_gpu
from moe_common import values

pytestmark = pytest.mark.gpu

TYPES = {"f32": "float32", "f16": "float16", "bf16": "bfloat16"}


def check(x, k, renorm=True, **kw):
    """x: CPU tensor [T, E]."""
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    r = tq.tq_moe_route(x.to(dev), k, renormalize=renorm, **kw)
    torch.cuda.synchronize()
    compare(r, x, k, renorm)
    return r


def compare(r, x, k, renorm=True):
    rows = x.double().numpy()
    e, w, off, order, places = OE.route(rows, k, renorm)
    T, E = rows.shape
    assert np.array_equal(r.experts.cpu().numpy(), e)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.rows.cpu().numpy(), order)
    assert np.array_equal(r.places.cpu().numpy(), places)
    finite = np.where(np.isfinite(rows), rows, 0.0)
    spread = finite.max(1, keepdims=True) - finite.min(1, keepdims=True)
    err = np.abs(values(r.weights) - w)
    assert (err <= w * (E + 8 + 2 * spread) * 2.0 ** -24 + 2.0 ** -140).all(), err.max()


def logits(T, E, dt, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * 2).to(getattr(torch, TYPES[dt]))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("E, k", [(1, 1), (2, 1), (3, 3), (8, 2), (15, 4), (16, 16), (17, 5), (64, 6), (65, 8), (128, 8), (100, 17),
                                  (255, 8), (256, 16), (257, 3), (512, 10), (1000, 64), (1024, 8)])
@pytest.mark.parametrize("T", [1, 5, 64, 65, 200])
def test_sizes(T, E, k, dt):
    log(f"route T={T} E={E} k={k} {dt}")
    check(logits(T, E, dt, T * 31 + E), k, renorm=(T + E) % 2 == 0)


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("E, k", [(8, 3), (128, 8), (600, 8)])
def test_ties(T, E, k):
    """Rows of few distinct logits, zeros of both signs among them: the lowest index first."""
    import torch
    log(f"route ties T={T} E={E}")
    x = torch.randint(-1, 2, (T, E), generator=torch.Generator().manual_seed(E)).float()
    x[::2] *= -1.0
    check(x, k)
    check(x.bfloat16(), k, renorm=False)


@pytest.mark.parametrize("T", [9, 130])
def test_masked_and_infinite_rows(T):
    import torch
    log(f"route masks T={T}")
    inf = float("inf")
    x = logits(T, 16, "f32", 5)
    x[0] = -inf                       # nothing to choose
    x[1] = float("nan")
    x[2, 3:] = -inf                   # fewer than k
    x[3, ::2] = float("nan")
    x[4, 5] = inf
    x[5, [2, 9, 11]] = inf            # infinities share the weight
    x[6] = -3.0e38
    x[6, 7] = 3.0e38
    x[7] = torch.finfo(torch.float32).min
    x[8, 1:] = torch.finfo(torch.float32).min
    for renorm in (True, False):
        check(x, 4, renorm)
        check(x, 1, renorm)
    y = x.clamp(-6.0e4, 6.0e4).half()
    y[7] = -65504.0
    check(y, 4)


def test_all_rows_masked():
    import torch
    log("route all masked")
    for T in (3, 100):
        r = check(torch.full((T, 8), float("-inf")), 2)
        assert r.offsets.cpu().tolist() == [0] * 9


def test_one_expert_takes_all():
    import torch
    log("route one expert")
    for T in (64, 1000):
        x = logits(T, 128, "bf16", 3)
        x[:, 77] = 100.0
        r = check(x, 1)
        assert r.offsets.cpu().tolist() == [0] * 78 + [T] * 51


def test_many_tokens():
    """More chunks than one pass of the sorting reads, and chunks of more than 64 tokens."""
    log("route 20000 tokens")
    check(logits(20000, 24, "f16", 9), 3)
    check(logits(16385, 8, "f32", 10), 2)


def test_strided_rows_and_given_outputs():
    import torch
    import bit_weight_only_tq_amd as tq
    log("route strides, out")
    dev = require_gpu()
    for T in (33, 70):
        wide = logits(T, 50, "f16", 4)
        view = wide.to(dev)[:, 3:42]
        out = tq.MoeRoute(*(torch.full(s, 99, dtype=d, device=dev) for s, d in (
            ((T, 4), torch.int32), ((T, 4), torch.float32), ((40,), torch.int32), ((T * 4,), torch.int32), ((T, 4), torch.int32))))
        ws = torch.full((tq.tq_moe_route_workspace_bytes(T, 39, 4),), 255, dtype=torch.uint8, device=dev)
        r = tq.tq_moe_route(view, 4, out=out, workspace=ws)
        torch.cuda.synchronize()
        assert r is out
        compare(r, wide[:, 3:42], 4)


def test_graph_and_stream():
    """Captured on a side stream and replayed on other logits."""
    import torch
    import bit_weight_only_tq_amd as tq
    log("route graph")
    dev = require_gpu()
    for T in (7, 500):
        x = logits(T, 64, "bf16", 1).to(dev)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            tq.tq_moe_route(x, 6)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = tq.tq_moe_route(x, 6)
        for seed in (2, 3, 4):
            new = logits(T, 64, "bf16", seed)
            x.copy_(new.to(dev))
            graph.replay()
            torch.cuda.synchronize()
            compare(r, new, 6)
