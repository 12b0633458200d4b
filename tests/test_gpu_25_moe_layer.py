"""The experts' operators one after another as a layer uses them, in the sizes of every cut of a call, and calls at once.

Each stage of the layer is held against the fp64 formula of the values that the stage before it wrote, within the bounds
of moe_common.py; the whole layer replayed from a graph gives the eager layer's bits.
"""
import numpy as np
import pytest

import oracle.experts as OE
from gpu_common import log, require_gpu
from moe_common import assert_within, experts, gated_bound, rounded, sum_bound, to_dev, values
from test_gpu_23_experts import call, check
from test_gpu_24_lora import bound_of, make as make_lora, test_combine as combine_within

pytestmark = pytest.mark.gpu


def uneven(experts_, rows, seed):
    """Counts of `experts_` experts around `rows` each, with their sum experts_ * rows."""
    if rows == 1:
        return [1] * experts_
    return np.random.default_rng(seed).multinomial(experts_ * rows, np.full(experts_, 1.0 / experts_)).tolist()


# (format, experts, rows of each, N, K): few and many rows, weight rows and columns, so that a call is cut into blocks of
# 4, 16, 32, 64 and 128 rows and its columns go to one wave, two, four and eight.
CUTS = [("ternary", 2, 1, 17772, 832), ("ternary", 35, 1, 519, 2048), ("ternary", 3, 1, 34, 4160), ("ternary", 1, 2, 34, 192),
        ("ternary", 6, 9, 1032, 576), ("ternary", 2, 20, 33, 1088), ("ternary", 12, 700, 33, 128), ("ternary", 24, 700, 33, 128),
        ("ternary", 12, 700, 528, 128), ("ternary", 40, 3, 2080, 320),
        ("w4", 35, 1, 519, 1408), ("w4", 3, 1, 34, 4224), ("w4", 1, 2, 33, 128), ("w4", 6, 9, 1032, 640), ("w4", 2, 20, 33, 512),
        ("w4", 12, 700, 33, 128), ("w4", 5, 3200, 16, 128), ("w4", 12, 2539, 142, 768), ("w4", 40, 3, 2080, 384),
        ("w4z", 12, 1, 2080, 512), ("w4z", 3, 1, 34, 4224), ("w4z", 8, 1, 2080, 128), ("w4z", 12, 1, 2080, 256),
        ("w4z", 2, 20, 33, 512), ("w4z", 24, 700, 33, 128), ("w4z", 48, 400, 33, 128), ("w4z", 7, 2773, 385, 128)]


@pytest.mark.parametrize("fmt, E, rows, N, K", CUTS)
def test_cuts(fmt, E, rows, N, K):
    log(f"experts {fmt} E={E} rows={rows} N={N} K={K}")
    counts = uneven(E, rows, N)
    check(fmt, E, N, K, counts, "bf16" if N % 2 else "f16", seed=E, bias=True)
    check(fmt, E, N + N % 2, K, counts, "f16" if N % 2 else "bf16", seed=E + 1, fan=1, gated=True)


def layer(x, logits, residual, up, down, k):
    import bit_weight_only_tq_amd as tq
    r = tq.tq_moe_route(logits, k)
    h = call(x, up, r.offsets, rows=r.rows, gated=True)
    y = call(h, down, r.offsets)
    return r, h, y, tq.tq_moe_combine(y, r.places, r.weights, add=residual)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["ternary", "w4", "w4z"])
@pytest.mark.parametrize("T", [1, 13, 300])
def test_layer(T, fmt, dt):
    """Routing, gated up and down products, the weighted sum; token 0 of several tokens has one expert alone."""
    import torch
    log(f"layer T={T} {fmt} {dt}")
    dev = require_gpu()
    E, k, H, F = 8, 2, 256, 384
    rng = np.random.default_rng(T)
    up, W13 = experts("ternary" if fmt == "ternary" else "w4", E, 2 * F, H, rng, zeros=fmt == "w4z")
    down, W2 = experts("ternary" if fmt == "ternary" else "w4", E, H, F, rng, zeros=fmt == "w4z")
    up, down = ({n: to_dev(v, dev) for n, v in p.items()} for p in (up, down))
    x, residual = (to_dev(rng.standard_normal((T, H)).astype(np.float32), dev, dt) for _ in range(2))
    logits = rng.standard_normal((T, E)).astype(np.float32)
    if T > 1:
        logits[0, 1:] = -np.inf
    logits = to_dev(logits, dev, dt)

    r, h, y, out = layer(x, logits, residual, up, down, k)
    torch.cuda.synchronize()
    off, rows, places = (t.cpu().numpy() for t in (r.offsets, r.rows, r.places))
    n = off[-1]
    want = OE.route(values(logits), k)
    for got, right in zip((r.experts, r.offsets, r.places), (want[0], want[2], want[4])):
        assert np.array_equal(got.cpu().numpy(), right)
    assert n == (2 * T if T == 1 else 2 * T - 1)
    C, mag = OE.product(values(x), W13, off, rows)
    assert_within(values(h)[:n], OE.gated(C[:n]), rounded(dt, gated_bound(H, C[:n], mag[:n]), OE.gated(C[:n])), "up")
    C, mag = OE.product(values(h), W2, off)
    assert_within(values(y)[:n], C[:n], rounded(dt, sum_bound(F, mag[:n]), C[:n]), "down")
    w = r.weights.double().cpu().numpy()
    C = OE.combine(values(y), places, w, values(residual))
    mag = OE.combine(np.abs(values(y)), places, np.abs(w), np.abs(values(residual)))
    assert_within(values(out), C, rounded(dt, (k + 1) * 2.0 ** -23 * mag, C), "combine")

    # replayed: other tokens and other experts every time, a row of no expert among them
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = layer(x, logits, residual, up, down, k)
    for step in range(4):
        x.copy_(to_dev(rng.standard_normal((T, H)).astype(np.float32), dev, dt))
        logits.copy_(to_dev(rng.standard_normal((T, E)).astype(np.float32), dev, dt))
        if step == 2:
            logits[T // 2] = -float("inf")
        eager = layer(x, logits, residual, up, down, k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        n = int(eager[0].offsets[-1])
        for a, b in zip(again[0], eager[0]):
            if a.dim() == 1 and a.numel() == T * k:  # rows: only those of an expert are told
                a, b = a[:n], b[:n]
            assert torch.equal(a, b)
        assert torch.equal(again[1][:n], eager[1][:n]) and torch.equal(again[2][:n], eager[2][:n])
        assert torch.equal(again[3], eager[3])
        if step == 2:
            assert torch.equal(eager[3][T // 2], residual[T // 2])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_adapters_beside_a_packed_projection(dt):
    """The projection's output takes the adapters' update in place, eager and from a graph."""
    import torch
    import bit_weight_only_tq_amd as tq
    log(f"projection with adapters {dt}")
    T, K, N, L, r = 21, 256, 264, 5, 16
    (x, _, A, B, ids, scale), h = make_lora(T, K, N, L, r, dt, 4)
    packed, W = experts("ternary", 1, N, K, np.random.default_rng(1))
    codes, s = to_dev(packed["w"][0], x.device), to_dev(packed["scale"][0], x.device)

    def run():
        out = tq.tq_gemm(x, codes, s)
        plain = out.clone()
        return plain, tq.tq_lora(x, out, A, B, ids, scale=scale, out=out)

    base, got = run()
    torch.cuda.synchronize()
    want, bound = bound_of([h[0], values(base)] + h[2:], dt, K, r)
    assert_within(values(got), want, bound, "projection")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, again = run()
    for shift in (1, 5):
        ids.copy_(torch.roll(ids, shift))
        x.mul_(-0.5)
        _, eager = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, eager)


@pytest.mark.parametrize("r", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("T, N", [(1, 520), (9, 1031), (64, 520), (300, 520), (300, 523), (2055, 264), (2055, 131)])
def test_adapters_give_the_same_bits_again(T, N, r):
    """Calls one after another and two at once: no value depends on the waves' or the workgroups' order."""
    import torch
    import bit_weight_only_tq_amd as tq
    log(f"lora again T={T} N={N} r={r}")
    (x, base, A, B, ids, scale), _ = make_lora(T, 328, N, 3, r, "f16" if r % 16 else "bf16", T + r)
    want = tq.tq_lora(x, base, A, B, ids, scale=scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        with torch.cuda.stream(side):
            other = tq.tq_lora(x, base, A, B, ids, scale=scale)
        again = tq.tq_lora(x, base, A, B, ids, scale=scale)
        torch.cuda.synchronize()
        assert torch.equal(again, want) and torch.equal(other, want)


@pytest.mark.parametrize("K, N", [(328, 1), (64, 9), (200, 31), (328, 265), (1096, 1030)])
@pytest.mark.parametrize("T, r", [(3, 16), (40, 64), (300, 32), (300, 64), (2100, 16), (2100, 64)])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_adapters_of_rows_at_any_address(T, r, K, N, shift):
    """Rows that begin at any value and end inside a vector, in place; what lies between the rows stays as it was."""
    import torch
    import bit_weight_only_tq_amd as tq
    log(f"lora T={T} r={r} K={K} N={N} shift={shift}")
    dt = "bf16" if shift else "f16"
    (x, base, A, B, ids, scale), h = make_lora(T, K, N, 4, r, dt, N)
    wide = torch.full((T, N + 11), 33.0, dtype=x.dtype, device=x.device)
    view = wide[:, shift:shift + N]
    view.copy_(base)
    tq.tq_lora(x, view, A, B, ids, scale=scale, out=view)
    torch.cuda.synchronize()
    want, bound = bound_of(h, dt, K, r)
    assert_within(values(view), want, bound, "rows")
    assert (wide[:, :shift] == 33.0).all() and (wide[:, shift + N:] == 33.0).all()


@pytest.mark.parametrize("N", list(range(2, 17)) + [1054, 4101])
def test_weighted_sums_of_rows_of_any_length(N):
    """Rows that end inside a vector, and so begin at any address."""
    for dt in ("f16", "bf16"):
        combine_within(5, 3, N, dt)
        combine_within(2, 9, N, dt)


def test_calls_at_once():
    """Routing with workspaces of their own and weighted sums on two streams at once."""
    import torch
    import bit_weight_only_tq_amd as tq
    log("route and combine at once")
    dev = require_gpu()
    gen = torch.Generator().manual_seed(3)
    logits = [torch.randn(1500, 60, generator=gen).to(dev) for _ in range(2)]
    y = torch.randn(6000, 136, generator=gen).to(dev, torch.bfloat16)
    want = [tq.tq_moe_route(v, 4) for v in logits]
    sums = [tq.tq_moe_combine(y, w.places, w.weights) for w in want]
    streams = [torch.cuda.Stream() for _ in logits]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for v, st in zip(logits, streams):
            with torch.cuda.stream(st):
                r = tq.tq_moe_route(v, 4)
                got.append((r, tq.tq_moe_combine(y, r.places, r.weights)))
        torch.cuda.synchronize()
        for (r, s), w, t in zip(got, want, sums):
            assert all(torch.equal(a, b) for a, b in zip(r, w)) and torch.equal(s, t)


LARGE = [("ternary", 16, 300, 144, 640), ("ternary", 8, 700, 272, 640), ("ternary", 8, 3000, 144, 640), ("w4", 8, 300, 272, 640),
         ("w4", 8, 700, 272, 640), ("w4", 16, 3000, 144, 640), ("w4z", 8, 700, 144, 640), ("w4z", 16, 700, 144, 640),
         ("w4z", 8, 3000, 144, 1024)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt, E, rows, N, K", LARGE)
def test_many_rows_scales_and_values_that_are_not_finite(fmt, E, rows, N, K, dt):
    """Blocks of 32 to 128 rows: groups whose scale is 0 (first, last, all of a row), scales from 2^-20 to 2^9 beside each
    other, a NaN and an infinity in a row, rows of no expert at the end; 40 rows of each expert against the formula."""
    import torch
    log(f"experts {fmt} {dt} E={E} rows={rows} N={N} K={K} scales")
    dev = require_gpu()
    rng = np.random.default_rng(K + rows)
    packed, W = experts("ternary" if fmt == "ternary" else "w4", E, N, K, rng, zeros=fmt == "w4z")
    old = packed["scale"].astype(np.float64)
    scale = (2.0 ** rng.integers(-20, 10, old.shape) * (1 + rng.integers(0, 4, old.shape) / 4)).astype(np.float16)
    scale[:, 5:20:3] = 0.0
    if fmt != "ternary":
        scale[:, 30:60][rng.random(scale[:, 30:60].shape) < 0.5] = 0.0
        scale[:, 60, 0] = scale[:, 61, -1] = 0.0
    W = (W.reshape(E, N, old[0, 0].size, -1) / old.reshape(E, N, -1, 1) * scale.astype(np.float64).reshape(E, N, -1, 1)).reshape(E, N, K)
    packed["scale"] = scale
    counts = uneven(E, rows, 9)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    P = int(off[-1]) + 7
    A = to_dev(rng.standard_normal((P, K)).astype(np.float32), dev, dt)
    bad_nan, bad_inf = int(off[1]) + 3, int(off[2]) - 2
    A[bad_nan, 5], A[bad_inf, K - 3] = float("nan"), float("inf")
    d = {n: to_dev(v, dev) for n, v in packed.items()}
    picked = np.unique(np.concatenate([np.r_[lo, hi - 1, rng.integers(lo, hi, 38)] for lo, hi in zip(off[:-1], off[1:])]))
    picked = picked[(picked != bad_nan) & (picked != bad_inf)]
    sub = np.searchsorted(picked, off).astype(np.int32)
    C, mag = OE.product(values(A[torch.from_numpy(picked).to(dev)]), W, sub)
    over = {"f16": 65520.0, "bf16": 3.3961775e38}[dt]
    for gated in (False, True):
        out = torch.full((P, N // 2 if gated else N), 123.0, dtype=A.dtype, device=dev)
        call(A, d, to_dev(off, dev), gated=gated, out=out)
        torch.cuda.synchronize()
        assert (out[-7:] == 123.0).all()
        assert out[bad_nan].isnan().all()
        assert gated or not out[bad_inf].isfinite().any()
        got = values(out)[picked]
        want, bound = (OE.gated(C), gated_bound(K, C, mag)) if gated else (C, sum_bound(K, mag))
        fine = np.abs(want) + bound < over
        assert_within(got[fine], want[fine], rounded(dt, bound, want)[fine], "scales")
        past = np.abs(want) - bound >= over
        assert np.array_equal(got[past], np.sign(want[past]) * np.inf)


@pytest.mark.parametrize("fmt, E, rows, N, K", LARGE)
def test_many_rows_offsets_of_any_values(fmt, E, rows, N, K):
    """Offsets and rows that no routing writes: memory around the output stays as it was."""
    import torch
    log(f"experts {fmt} E={E} rows={rows} wild offsets")
    dev = require_gpu()
    rng = np.random.default_rng(rows)
    packed, _ = experts("ternary" if fmt == "ternary" else "w4", E, N, K, rng, zeros=fmt == "w4z")
    d = {n: to_dev(v, dev) for n, v in packed.items()}
    P = E * rows
    A = to_dev(rng.standard_normal((P // 2, K)).astype(np.float32), dev, "f16")
    pairs = rng.permutation(P).astype(np.int32)
    pairs[:3] = -5, 2 ** 31 - 1, P
    pairs = to_dev(pairs, dev)
    big = torch.full((P + 64, N), 77.0, dtype=A.dtype, device=dev)
    sound = np.arange(E + 1, dtype=np.int64) * rows
    for change in ({1: 2 ** 30}, {0: -5, E: P + 99}, {0: 8, 1: 0, E - 1: -1}, {1: P, 2: 0, E: P}):
        off = sound.copy()
        for i, v in change.items():
            off[i] = v
        call(A, d, to_dev(off.astype(np.int32), dev), rows=pairs, out=big[32:-32])
        torch.cuda.synchronize()
        assert (big[:32] == 77.0).all() and (big[-32:] == 77.0).all()


# --------------------------------------------------- offsets past 32 bits

def test_experts_past_four_gigabytes():
    """72 experts of 64 MB: the last ones' codes, scales and zero points lie past 2^32 bytes."""
    import torch
    log("experts past 2^32 bytes")
    dev = require_gpu()
    E, N, K = 72, 8192, 16384
    gen = torch.Generator(device=dev).manual_seed(5)
    q = torch.randint(-2 ** 31, 2 ** 31 - 1, (E, N, K // 8), generator=gen, device=dev, dtype=torch.int32)
    scale = (torch.rand((E, N, K // 128), generator=gen, device=dev) * 0.01 + 0.001).half()
    zeros = torch.randint(0, 16, (E, N, K // 128), generator=gen, device=dev, dtype=torch.uint8)
    for counts in ({0: 2, 70: 1, 71: 3}, {3: 20, 71: 60}):
        off = np.zeros(E + 1, np.int32)
        for e, c in counts.items():
            off[e + 1:] += c
        A = torch.randn((int(off[-1]), K), generator=gen, device=dev).half()
        got = values(call(A, {"w": q, "scale": scale, "zeros": zeros}, to_dev(off, dev)))
        torch.cuda.synchronize()
        picked = np.r_[0:8, 4000:4040, N - 8:N]
        for e in counts:
            words = q[e, picked].cpu().numpy().view(np.uint32)
            W = ((words[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).reshape(len(picked), K // 128, 128).astype(np.float64)
            W = (W - zeros[e, picked].cpu().numpy()[..., None]) * scale[e, picked].double().cpu().numpy()[..., None]
            a = values(A[off[e]:off[e + 1]])
            want, mag = a @ W.reshape(len(picked), K).T, np.abs(a) @ np.abs(W).reshape(len(picked), K).T
            assert_within(got[off[e]:off[e + 1]][:, picked], want, rounded("f16", sum_bound(K, mag), want), f"expert {e}")


def test_rows_past_four_gigabytes():
    """Rows of the weighted sum and of the adapters that lie past 2^32 bytes."""
    import torch
    import bit_weight_only_tq_amd as tq
    log("rows past 2^32 bytes")
    dev = require_gpu()
    P, N = 560000, 4096
    y = torch.zeros((P, N), dtype=torch.bfloat16, device=dev)
    rows = torch.randn((4, N), generator=torch.Generator(device=dev).manual_seed(1), device=dev).bfloat16()
    for i, p in enumerate((0, 524288, P - 2, P - 1)):
        y[p] = rows[i]
    places = torch.tensor([[0, P - 1], [524288, P - 2]], dtype=torch.int32, device=dev)
    weights = torch.tensor([[0.5, 1.5], [-1.0, 0.25]], device=dev)
    got = values(tq.tq_moe_combine(y, places, weights))
    r, w = values(rows), values(weights)
    want = np.stack([w[0, 0] * r[0] + w[0, 1] * r[3], w[1, 0] * r[1] + w[1, 1] * r[2]])
    mag = np.stack([np.abs(w[0, 0] * r[0]) + np.abs(w[0, 1] * r[3]), np.abs(w[1, 0] * r[1]) + np.abs(w[1, 1] * r[2])])
    assert_within(got, want, rounded("bf16", 3 * 2.0 ** -23 * mag, want), "sum")
    del y

    # 9000 rows of 64 columns, 2^18 values from one to the next
    T, K, N, r = 9000, 64, 72, 16
    (x, base, A, B, _, scale), h = make_lora(T, K, N, 2, r, "f16", 3, ids=np.arange(T) // 4500)
    ids = to_dev(h[4], dev)
    far_x = torch.empty((T, 1 << 18), dtype=torch.float16, device=dev)[:, :K]
    far_out = torch.empty((T, 1 << 18), dtype=torch.float16, device=dev)[:, 8:8 + N]
    far_x.copy_(x)
    far_out.copy_(base)
    tq.tq_lora(far_x, far_out, A, B, ids, scale=scale, out=far_out)
    torch.cuda.synchronize()
    want, bound = bound_of(h, "f16", K, r)
    assert_within(values(far_out), want, bound, "rows")
