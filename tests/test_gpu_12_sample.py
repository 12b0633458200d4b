"""Sampling against the fp64 oracle: tokens are equal, log probabilities within their rounding.

A log probability is fp64 until its one rounding to fp32 (half a step: 2^-24 of it); the kernel's weights and their
total differ from the oracle's by less than 2^-40, the kept total being at least 1.
"""
import numpy as np
import pytest

import oracle.sampling as OS
from gpu_common import log, require_gpu

pytestmark = pytest.mark.gpu

DT = {"f16": "float16", "bf16": "bfloat16", "f32": "float32"}


def _run(x, u, T=None, k=None, p=None, m=None):
    """x: CPU tensor [B, V]; the others None, a value, or B values."""
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    B = x.shape[0]
    t = lambda v, d: None if v is None else torch.as_tensor(v, dtype=d).expand(B).contiguous().to(dev)  # noqa: E731
    r = tq.tq_sample(x if x.is_cuda else x.to(dev), t(u, torch.float32), temperature=t(T, torch.float32),
                     top_k=t(k, torch.int32), top_p=t(p, torch.float32), min_p=t(m, torch.float32))
    torch.cuda.synchronize()
    return r[0].tolist(), r[1].double().cpu().numpy()


def _check(x, u, T=None, k=None, p=None, m=None):
    f = lambda v, b, d: d if v is None else float(np.float32(v[b] if np.ndim(v) else v))  # noqa: E731
    tok, lp = _run(x, u, T, k, p, m)
    rows = x.double().cpu().numpy()
    for b in range(rows.shape[0]):
        want, wlp = OS.sample(rows[b], f(u, b, 0.0), f(T, b, 1.0), int(f(k, b, 0)), f(p, b, 1.0), f(m, b, 0.0))
        assert tok[b] == want, f"row {b}: token {tok[b]}, oracle {want}"
        if wlp == -np.inf:
            assert lp[b] == -np.inf
        else:
            assert abs(lp[b] - wlp) <= 2.0 ** -24 * abs(wlp) + 2.0 ** -38, f"row {b}: logprob {lp[b]}, oracle {wlp}"


def _logits(B, V, dt, seed=0, peaks=20):
    import torch
    g = torch.Generator().manual_seed(seed * 977 + V + B)
    x = torch.randn((B, V), generator=g) * 2
    at = torch.randint(0, V, (B, peaks), generator=g)
    x.scatter_add_(1, at, torch.rand((B, peaks), generator=g) ** 2 * 14)
    return x.to(getattr(torch, DT[dt]))


PARAMS = [(None, None, None, None), (0.0, 50, 0.9, 0.1), (1.0, 1, None, None), (0.7, 50, None, None), (1.0, None, 0.9, None),
          (1.3, None, 0.5, None), (0.8, None, None, 0.05), (1.0, 20, 0.8, 0.02), (2.0, 1000, 0.95, None),
          (0.6, 7, 0.99, 0.3), (50.0, None, 0.7, None), (0.05, 100, 0.9, None), (3.0, 3000, 0.999, 0.001)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 3, 63, 64, 65, 255, 257, 511, 513, 1000, 4097, 32000, 129281])
def test_sizes_and_filters(V, dt):
    B = 3
    for i, (T, k, p, m) in enumerate(PARAMS):
        log(f"sample V={V} {dt} T={T} k={k} p={p} min_p={m}")
        u = np.random.default_rng(V + i).random(B).astype(np.float32)
        _check(_logits(B, V, dt, i), u, T, k, p, m)


def test_rows_of_different_requests():
    """Every row its own temperature and filters, 300 rows."""
    log("mixed rows")
    rng = np.random.default_rng(8)
    B = 300
    _check(_logits(B, 5003, "f32"), rng.random(B).astype(np.float32), rng.choice([0.0, 0.3, 1.0, 1.7], B),
           rng.choice([0, 1, 5, 50, 4000], B), rng.choice([0.1, 0.6, 0.95, 1.0], B), rng.choice([0.0, 0.01, 0.2, 1.0], B))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("values", [1, 2, 5, 40])
def test_ties(dt, values):
    """Rows of few distinct logits: cuts fall inside ties, which go to the lowest index."""
    import torch
    rng = np.random.default_rng(values)
    for V in (1, 65, 1000, 9001):
        x = torch.tensor(rng.integers(0, values, (6, V)) / 4.0).to(getattr(torch, DT[dt]))
        log(f"ties {values} {dt} V={V}")
        for T, k, p, m in ((1.0, 1 + V // 3, None, None), (0.5, None, 0.3, None), (1.0, 1 + V // 2, 0.77, None),
                           (2.0, None, 0.9, 0.3), (1.0, None, None, 1.0), (0.9, V, 0.01, None)):
            _check(x, rng.random(6).astype(np.float32), T, k, p, m)


def test_equal_logits_cut_exactly():
    """All weights 1: top-p of one half keeps exactly half, and u walks through them."""
    import torch
    log("equal logits")
    x = torch.zeros((64, 64))
    u = (np.arange(64) / 64).astype(np.float32)
    tok, lp = _run(x, u, 1.0, None, 0.5, None)
    assert tok == [i // 2 for i in range(64)] and np.allclose(lp, -np.log(32), atol=1e-6)
    tok, _ = _run(x, u, 1.0, 16, None, None)
    assert tok == [i // 4 for i in range(64)]


def test_frequencies():
    """Evenly spaced random numbers draw every token as often as its probability says."""
    import torch
    log("frequencies")
    x = _logits(1, 333, "f32", 3).expand(5000, 333).contiguous()
    u = ((np.arange(5000) + 0.5) / 5000).astype(np.float32)
    tok, lp = _run(x, u, 1.5, 100, 0.95, None)
    order, w = OS.kept(x[0].double().numpy(), 1.5, 100, float(np.float32(0.95)), 0.0)
    p = np.zeros(333)
    p[order] = w / w.sum()
    assert np.abs(np.bincount(tok, minlength=333) / 5000 - p).max() <= 1.001 / 5000
    assert np.allclose(lp, np.log(p[tok]), atol=1e-5)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_infinities_and_nan(dt):
    import torch
    log(f"infinities {dt}")
    inf, nan = float("inf"), float("nan")
    V = 700
    x = _logits(7, V, dt)
    x[0] = -inf                              # nothing to sample
    x[1] = nan
    x[2, ::2], x[2, 1::4] = -inf, nan
    x[3, [5, 600, 601]] = inf                # equal infinities share the weight
    x[4], x[4, 77] = -inf, -3.0              # one token
    x[5] = torch.finfo(x.dtype).min          # masks of the lowest value everywhere: all alike
    x[6, 10:] = torch.finfo(x.dtype).min
    for T, k, p, m in PARAMS:
        for u in (0.0, 0.3, 0.999):
            _check(x, u, T, k, p, m)


def test_ends_of_u():
    log("u")
    import torch
    x = _logits(8, 3001, "f32", 5)
    u = [0.0, 1e-30, 2.0 ** -24, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, float("nan")]
    _check(x, u)
    _check(x, u, 0.7, 40, 0.9)
    # u = 0 takes the first kept token of positive weight, however small
    far = torch.full((1, 900), -80.0)
    far[0, 500] = 0.0
    assert _run(far, 0.0)[0] == [0] and _run(far, 0.0, None, None, 0.9)[0] == [500]


def test_values_out_of_their_ranges():
    """Negative and huge k, p and min_p outside [0, 1], temperatures that are not positive."""
    log("ranges")
    x = _logits(5, 999, "bf16", 6)
    u = np.random.default_rng(1).random(5).astype(np.float32)
    big = 2**31 - 1
    _check(x, u, 1.0, [-5, -big - 1, big, 998, 999])
    _check(x, u, 1.0, None, [1.5, 0.0, -2.0, 1e-20, float("inf")])
    _check(x, u, 1.0, None, None, [1.5, -3.0, 1.0, 1e-30, float("inf")])
    _check(x, u, [-1.0, -0.0, float("nan"), 1e-30, 1e30], 30)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_strided_and_unaligned_rows(dt):
    import torch
    log(f"strides {dt}")
    dev = require_gpu()
    x = _logits(5, 1003, dt)
    wide = torch.full((5, 1003 + 9), 99.0, dtype=x.dtype, device=dev)
    for off in (0, 1, 3, 7):
        view = wide[:, off:off + 1003]
        wide.fill_(99.0)
        view.copy_(x)
        u = np.random.default_rng(off).random(5).astype(np.float32)
        _check(view, u, 0.9, 30, 0.9)
        _check(view, u)


def test_largest_vocabulary():
    log("V = 2^20")
    x = _logits(2, 1 << 20, "f32", 9)
    _check(x, [0.2, 0.9], 1.0)
    _check(x, [0.2, 0.9], 1.0, 5000, 0.9)
    _check(x.half(), [0.4, 0.7], 2.0, None, 0.8)


def test_graph_and_none():
    """Captured, replayed with new logits and numbers in place; B = 0 does nothing."""
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    log("graph")
    x = _logits(4, 32000, "f32").to(dev)
    u = torch.full((4,), 0.5, device=dev)
    k = torch.full((4,), 40, dtype=torch.int32, device=dev)
    out = (torch.empty(4, dtype=torch.int32, device=dev), torch.empty(4, device=dev))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tq.tq_sample(x, u, top_k=k, out=out)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_sample(x, u, top_k=k, out=out)
    for i in range(4):
        x.copy_(_logits(4, 32000, "f32", i))
        u.fill_(0.2 * i)
        want = tq.tq_sample(x, u, top_k=k)
        out[0].fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), f"replay {i}"
    assert tq.tq_sample(x[:0], u[:0])[0].numel() == 0
