"""Low-rank updates and the experts' weighted sum against the fp64 oracle.

The update's bound: x A^T is off by (K + 32) 2^-23 of its terms' magnitudes, and enters the second product as two 16-bit numbers
that are off by u^2 of the value (u: half a step of the type) or, in fp16, by half its smallest subnormal (2^-25) of twice the
row's largest value; the second product sums twice the rank; scale, product and sum with the base are fp32 roundings.
"""
import numpy as np
import pytest

import oracle.experts as OE
from gpu_common import log, require_gpu
from moe_common import U, assert_within, rounded, sum_bound, to_dev, values

pytestmark = pytest.mark.gpu


def make(T, K, N, L, r, dt, seed, ids=None):
    import torch
    dev = require_gpu()
    rng = np.random.default_rng(seed)
    half = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(getattr(torch, {"f16": "float16", "bf16": "bfloat16"}[dt]))  # noqa: E731
    x, base, A, B = half(T, K), half(T, N), half(L, r, K) / K ** 0.5, half(L, N, r) / r ** 0.5
    if ids is None:
        ids = rng.integers(-1, L + 1, T)
    ids = np.asarray(ids, np.int32)
    scale = (rng.random(L) + 0.5).astype(np.float32)
    d = [t.to(dev) for t in (x, base, A, B)] + [to_dev(ids, dev), to_dev(scale, dev)]
    return d, [x.double().numpy(), base.double().numpy(), A.double().numpy(), B.double().numpy(), ids, scale.astype(np.float64)]


def bound_of(h, dt, K, r):
    x, base, A, B, ids, scale = h
    want, hid = OE.lora(*h)
    bound = np.zeros_like(want)
    for t, l in enumerate(ids):
        if 0 <= l < A.shape[0]:
            dh = sum_bound(K, np.abs(A[l]) @ np.abs(x[t]))
            split = U[dt] ** 2 * np.abs(hid[t]) + (2.0 ** -24 * np.abs(hid[t]).max() if dt == "f16" else 0.0)
            b = np.abs(B[l])
            bound[t] = scale[l] * (b @ (dh + split) + (2 * r + 32) * 2.0 ** -23 * (b @ np.abs(hid[t])) * 1.01)
            bound[t] += 2.0 ** -23 * (np.abs(base[t]) + 2 * np.abs(want[t] - base[t]))
    out = rounded(dt, bound, want)
    out[~((ids >= 0) & (ids < A.shape[0]))] = 0.0  # rows without an adapter are copied
    return want, out


def check(T, K, N, L, r, dt, seed=0, ids=None):
    import torch
    import bit_weight_only_tq_amd as tq
    d, h = make(T, K, N, L, r, dt, seed, ids)
    x, base, A, B, ids_d, scale = d
    got = tq.tq_lora(x, base, A, B, ids_d, scale=scale)
    torch.cuda.synchronize()
    want, bound = bound_of(h, dt, K, r)
    assert_within(values(got), want, bound, f"lora T={T} K={K} N={N} L={L} r={r} {dt}")
    again = base.clone()
    assert tq.tq_lora(x, again, A, B, ids_d, scale=scale, out=again) is again
    torch.cuda.synchronize()
    assert torch.equal(again, got), "in place"


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 104, 128, 136, 256])
@pytest.mark.parametrize("T", [1, 3, 16, 17, 50])
def test_ranks(T, r, dt):
    log(f"lora T={T} r={r} {dt}")
    check(T, 256, 192, 3, r, dt, seed=T + r)


@pytest.mark.parametrize("K, N", [(8, 8), (24, 1), (64, 7), (72, 31), (136, 33), (520, 100), (1000, 513), (4096, 1025), (14336, 40)])
@pytest.mark.parametrize("T", [2, 70])
def test_odd_sizes(T, K, N):
    log(f"lora T={T} K={K} N={N}")
    for dt in ("f16", "bf16"):
        check(T, K, N, 2, 16, dt, seed=K)


@pytest.mark.parametrize("T, L", [(1, 1), (64, 1), (64, 100), (300, 7), (1000, 3), (257, 40)])
def test_mixtures(T, L):
    log(f"lora T={T} L={L}")
    check(T, 320, 264, L, 16, "bf16", seed=T)
    cuts = np.sort(np.random.default_rng(T).integers(0, T, 4))
    check(T, 320, 264, L, 64, "f16", seed=L, ids=np.searchsorted(cuts, np.arange(T), side="right") % L)


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 256])
def test_long_prompts(r):
    """From 2048 rows on: whole and ragged columns, K that ends inside a step, blocks of several adapters, rows without one."""
    log(f"lora prompts r={r}")
    ids = np.repeat([0, 2, -1, 1, 5, 0], [700, 13, 64, 1000, 200, 100])[:2055]
    assert len(ids) == 2055
    check(2055, 200, 520, 3, r, "bf16", seed=r, ids=ids)
    check(2055, 64, 72, 3, r, "f16", seed=r, ids=ids)
    check(2048, 1096, 1032, 2, r, "f16", seed=r + 1)


def test_ids_of_any_values():
    log("lora ids")
    check(9, 64, 48, 2, 8, "f16", ids=[0, -1, 1, 2, -2 ** 31, 2 ** 31 - 1, 1, 0, -2])
    check(40, 64, 48, 2, 8, "bf16", ids=[-1] * 40)


def test_strides_scale_and_none():
    """Views of a fused projection's output, no scales, and rows around the views left alone."""
    import torch
    import bit_weight_only_tq_amd as tq
    log("lora strides")
    (x, base, A, B, ids, scale), h = make(37, 128, 64, 3, 16, "bf16", 2)
    for pad in (8, 3):
        wide = torch.full((37, 64 + 2 * pad), 55.0, dtype=x.dtype, device=x.device)
        xs = torch.zeros((37, 160), dtype=x.dtype, device=x.device)
        xs[:, 16:144] = x
        view = wide[:, pad:pad + 64]
        view.copy_(base)
        got = tq.tq_lora(xs[:, 16:144], view, A, B, ids, out=view)
        assert got is view
        torch.cuda.synchronize()
        want, bound = bound_of(h[:5] + [np.ones(3)], "bf16", 128, 16)
        assert_within(values(view), want, bound, "strided")
        assert (wide[:, :pad] == 55.0).all() and (wide[:, pad + 64:] == 55.0).all()
    out = torch.full((37, 80), 55.0, dtype=x.dtype, device=x.device)
    got = tq.tq_lora(x, base, A, B, ids, scale=scale, out=out[:, 5:69])
    torch.cuda.synchronize()
    assert torch.equal(got, tq.tq_lora(x, base, A, B, ids, scale=scale))
    assert (out[:, :5] == 55.0).all() and (out[:, 69:] == 55.0).all()


@pytest.mark.parametrize("dt, big", [("f16", 2.0 ** 15), ("bf16", 2.0 ** 100), ("bf16", 2.0 ** -100), ("f16", 2.0 ** -12)])
def test_large_and_small_inner_values(dt, big):
    """x A^T past the type's range, or near its smallest values, where the result is ordinary."""
    import torch
    import bit_weight_only_tq_amd as tq
    log(f"lora inner values {dt} {big}")
    (x, base, A, B, ids, scale), h = make(20, 512, 64, 2, 16, dt, 6, ids=[0, 1] * 10)
    x2, B2 = (x * 8 if big > 1 else x / 8), B
    A2 = A * big if dt == "bf16" else A * (big / 8 if big > 1 else big)
    s2 = (1.0 / (big * (8.0 if big > 1 else 0.125))) if dt == "bf16" else (1.0 / big if big > 1 else 8.0 / big)
    scale2 = (scale.double() * s2).float()
    got = tq.tq_lora(x2, base, A2, B2, ids, scale=scale2)
    torch.cuda.synchronize()
    hh = [values(x2), h[1], values(A2), h[3], h[4], values(scale2)]
    want, bound = bound_of(hh, dt, 512, 16)
    assert_within(values(got), want, bound, "inner")


def test_values_that_are_not_finite_stay_in_their_row():
    import torch
    import bit_weight_only_tq_amd as tq
    log("lora not finite")
    (x, base, A, B, ids, scale), _ = make(12, 128, 72, 2, 16, "f16", 3, ids=[0, 1, 0, 1, 1, 0, -1, 0, 1, 0, 1, 1])
    clean = tq.tq_lora(x, base, A, B, ids)
    x = x.clone()
    x[2, 3], x[5, 9], x[6] = float("nan"), float("inf"), float("nan")
    got = tq.tq_lora(x, base, A, B, ids)
    torch.cuda.synchronize()
    assert got[2].isnan().all() and not got[5].isfinite().any()
    assert torch.equal(got[6], base[6])  # no adapter: x is not looked at
    keep = [0, 1, 3, 4, 7, 8, 9, 10, 11]
    assert torch.equal(got[keep], clean[keep])


def test_lora_graph():
    import torch
    import bit_weight_only_tq_amd as tq
    log("lora graph")
    (x, base, A, B, ids, scale), _ = make(33, 256, 128, 4, 16, "bf16", 8)
    out = torch.empty_like(base)
    tq.tq_lora(x, base, A, B, ids, scale=scale, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_lora(x, base, A, B, ids, scale=scale, out=out)
    for shift in (1, 2, 3):
        ids.copy_(torch.roll(ids, shift))
        want = tq.tq_lora(x, base, A, B, ids, scale=scale)
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T, k, N", [(1, 1, 1), (1, 2, 4096), (3, 8, 100), (50, 3, 257), (700, 2, 64), (9, 17, 72)])
def test_combine(T, k, N, dt):
    """k fp32 products and sums: each within 2^-24 of a partial sum, itself at most the magnitudes' sum."""
    import torch
    import bit_weight_only_tq_amd as tq
    log(f"combine T={T} k={k} N={N} {dt}")
    dev = require_gpu()
    rng = np.random.default_rng(T * k + N)
    ty = getattr(torch, {"f16": "float16", "bf16": "bfloat16"}[dt])
    P = T * k
    y = torch.from_numpy(rng.standard_normal((P, N)).astype(np.float32)).to(ty)
    wide = torch.from_numpy(rng.standard_normal((T, N + 5)).astype(np.float32)).to(ty)
    places = rng.permutation(P).reshape(T, k).astype(np.int32)
    places[rng.random((T, k)) < 0.2] = rng.choice([-1, P, 2 ** 31 - 1, -2 ** 31])  # adds nothing
    w = rng.standard_normal((T, k)).astype(np.float32)
    for add in (None, wide[:, :N].contiguous(), wide[:, 5:]):
        want = OE.combine(values(y), places, w.astype(np.float64), None if add is None else values(add))
        mag = OE.combine(np.abs(values(y)), places, np.abs(w).astype(np.float64), None if add is None else np.abs(values(add)))
        a = None if add is None else wide.to(dev)[:, 5:] if add.stride(0) != N and T > 1 else add.to(dev)
        got = tq.tq_moe_combine(y.to(dev), to_dev(places, dev), to_dev(w, dev), add=a)
        torch.cuda.synchronize()
        assert_within(values(got), want, rounded(dt, (k + 1) * 2.0 ** -23 * mag, want), "combine")
        if a is not None and a.is_contiguous():
            assert tq.tq_moe_combine(y.to(dev), to_dev(places, dev), to_dev(w, dev), add=a, out=a) is a
            torch.cuda.synchronize()
            assert torch.equal(a, got)
