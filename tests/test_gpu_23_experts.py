"""Products grouped by expert against the fp64 oracle, within the bounds of moe_common.py."""
import numpy as np
import pytest

import oracle.experts as OE
from gpu_common import log, require_gpu
from moe_common import assert_within, experts, gated_bound, offsets_of, rounded, sum_bound, to_dev, values

pytestmark = pytest.mark.gpu

FMTS = ["ternary", "w4", "w4z"]


def call(A, packed, off, rows=None, bias=None, gated=False, out=None):
    import bit_weight_only_tq_amd as tq
    if packed["w"].dtype.itemsize == 1:
        return tq.tq_moe_gemm(A, packed["w"], packed["scale"], off, rows=rows, bias=bias, gated=gated, out=out)
    return tq.w4a16_moe_gemm(A, packed["w"], packed["scale"], off, rows=rows, zeros=packed["zeros"], bias=bias, gated=gated, out=out)


def make(fmt, E, N, K, counts, dt, seed, fan=0, bias=False):
    """-> device inputs, fp64 inputs.  fan 0: grouped rows; else rows of P / fan tokens in any order."""
    import torch
    dev = require_gpu()
    rng = np.random.default_rng(seed)
    packed, W = experts("ternary" if fmt == "ternary" else "w4", E, N, K, rng, zeros=fmt == "w4z")
    P = int(sum(counts))
    if fan:
        P = -(-P // fan) * fan  # rows of no expert at the end
    T = P // fan if fan else P
    A = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(getattr(torch, {"f16": "float16", "bf16": "bfloat16"}[dt]))
    rows = rng.permutation(P).astype(np.int32) if fan else None
    b = torch.from_numpy(rng.standard_normal((E, N)).astype(np.float32)).to(A.dtype) if bias else None
    d = {"A": A.to(dev), "packed": {n: to_dev(v, dev) for n, v in packed.items()}, "off": to_dev(offsets_of(counts), dev),
         "rows": to_dev(rows, dev), "bias": None if b is None else b.to(dev)}
    h = {"A": A.double().numpy(), "W": W, "off": offsets_of(counts), "rows": rows, "bias": None if b is None else b.double().numpy(),
         "P": P}
    return d, h


def check(fmt, E, N, K, counts, dt, seed=0, fan=0, bias=False, gated=False):
    import torch
    d, h = make(fmt, E, N, K, counts, dt, seed, fan, bias)
    width = N // 2 if gated else N
    out = torch.full((h["P"], width), 123.0, dtype=d["A"].dtype, device=d["A"].device)
    got = call(d["A"], d["packed"], d["off"], d["rows"], d["bias"], gated, out)
    torch.cuda.synchronize()
    assert got is out
    compare(values(out), h, K, dt, gated, f"{fmt} E={E} N={N} K={K}")


def compare(got, h, K, dt, gated, label):
    C, mag = OE.product(h["A"], h["W"], h["off"], h["rows"], h["bias"])
    n = h["off"][-1]
    assert (got[n:] == 123.0).all(), "rows behind the last expert's were written"
    C, mag, got = C[:n], mag[:n], got[:n]
    if gated:
        want = OE.gated(C)
        bound = gated_bound(K, C, mag)
    else:
        want, bound = C, sum_bound(K, mag)
    assert_within(got, want, rounded(dt, bound, want), label)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[1], [0, 1], [1, 0, 2], [3, 0, 0, 17, 1], [16, 15, 33], [70, 1, 130], [300, 5]])
def test_counts(counts, fmt, dt):
    log(f"experts {fmt} {dt} counts={counts}")
    K = 384 if fmt != "ternary" else 320
    check(fmt, len(counts), 96, K, counts, dt)
    check(fmt, len(counts), 64, 2 * K, counts, dt, seed=1, fan=2, gated=True, bias=True)


@pytest.mark.parametrize("fmt, K", [("ternary", 64), ("ternary", 128), ("ternary", 192), ("ternary", 256), ("ternary", 2112),
                                    ("w4", 128), ("w4", 256), ("w4z", 128), ("w4z", 640), ("w4", 2176)])
@pytest.mark.parametrize("N", [1, 2, 15, 17, 130, 257])
def test_odd_sizes(fmt, K, N):
    log(f"experts {fmt} N={N} K={K}")
    for dt in ("f16", "bf16"):
        check(fmt, 3, N, K, [5, 40, 18], dt, seed=N)
        check(fmt, 3, N, K, [2, 0, 1], dt, seed=N, fan=1, bias=True)
    if N % 2 == 0:
        check(fmt, 3, N, K, [1, 150, 0], "bf16", seed=N, gated=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[1, 1, 0, 1] * 2, [4] * 40, [0] * 90 + [3, 9] + [1] * 60, [33] * 12, [200, 0, 256, 1, 513], [1300]])
def test_larger(counts, fmt):
    log(f"experts {fmt} {len(counts)} experts, {sum(counts)} rows")
    check(fmt, len(counts), 272, 512, counts, "f16", fan=2)
    check(fmt, len(counts), 528, 512, counts, "bf16", gated=True, bias=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[2, 1], [40, 30], [600]])
def test_long_k(fmt, counts):
    log(f"experts {fmt} K=17408 counts={counts}")
    check(fmt, len(counts), 48, 17408, counts, "bf16")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[3, 2], [90, 40]])
def test_values_that_are_not_finite_stay_in_their_row(fmt, counts):
    import torch
    log(f"experts {fmt} not finite")
    d, h = make(fmt, 2, 80, 256, counts, "bf16", 7)
    clean = call(d["A"], d["packed"], d["off"])
    A = d["A"].clone()
    A[1, 5] = float("nan")
    A[2, 200] = float("inf")
    got = call(A, d["packed"], d["off"])
    torch.cuda.synchronize()
    assert got[1].isnan().all()
    assert not got[2].isfinite().any()  # +-inf, or NaN from a weight of 0
    keep = [r for r in range(sum(counts)) if r not in (1, 2)]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_and_rows_of_any_values(fmt):
    """What no routing writes: memory around the output stays as it was, and rows of sound experts are right."""
    import torch
    log(f"experts {fmt} wild offsets")
    d, h = make(fmt, 4, 48, 256, [8, 8, 8, 8], "f16", 11, fan=2)
    dev = d["A"].device
    big = torch.full((32 + 64, 48), 77.0, dtype=torch.float16, device=dev)
    for off in ([0, 8, 1 << 30, 16, 32], [-5, 8, 16, 24, 99], [8, 0, 8, -1, 4], [0, 32, 32, 0, 32]):
        rows = d["rows"].clone()
        rows[3], rows[9] = -7, 1 << 30
        big.fill_(77.0)
        call(d["A"], d["packed"], torch.tensor(off, dtype=torch.int32, device=dev), rows=rows, out=big[32:64])
        torch.cuda.synchronize()
        assert (big[:32] == 77.0).all() and (big[64:] == 77.0).all()


def test_zero_rows():
    import torch
    log("experts without rows")
    d, _ = make("w4", 2, 32, 128, [0, 0], "f16", 1)
    assert call(d["A"], d["packed"], d["off"]).shape == (0, 32)
    d, h = make("ternary", 2, 32, 128, [3, 2], "f16", 1)
    none = torch.zeros_like(d["off"])
    out = torch.full((5, 32), 9.0, dtype=torch.float16, device=none.device)
    call(d["A"], d["packed"], none, out=out)
    torch.cuda.synchronize()
    assert (out == 9.0).all()


@pytest.mark.parametrize("fmt", ["ternary", "w4"])
@pytest.mark.parametrize("counts", [[2, 0, 1, 3], [150, 20, 0, 90]])
def test_same_bits_again_and_in_a_graph(fmt, counts):
    """Two calls at once on two streams and a replayed graph give the eager call's bits; offsets are read at replay."""
    import torch
    log(f"experts {fmt} graph")
    d, _ = make(fmt, 4, 256, 512, counts, "bf16", 5, fan=1)
    want = call(d["A"], d["packed"], d["off"], d["rows"], gated=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(d["A"], d["packed"], d["off"], d["rows"], gated=True)
    again = call(d["A"], d["packed"], d["off"], d["rows"], gated=True)
    torch.cuda.synchronize()
    assert torch.equal(want, other) and torch.equal(want, again)
    off, out = torch.zeros_like(d["off"]), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(d["A"], d["packed"], off, d["rows"], gated=True, out=out)
    for _ in range(3):
        out.fill_(5.0)
        off.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert (out == 5.0).all()
        off.copy_(d["off"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", [[3, 2], [50, 20], [200, 3]])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_scales_of_zero_and_of_every_size(fmt, counts, dt):
    """Groups whose scale is 0 (whole rows of them, the first and the last group), and scales from 2^-24 to 2^9 beside each other."""
    import torch
    log(f"experts {fmt} {dt} scales counts={counts}")
    d, h = make(fmt, 2, 96, 1024, counts, dt, 13)
    rng = np.random.default_rng(14)
    old = values(d["packed"]["scale"])
    scale = 2.0 ** rng.integers(-24, 10, old.shape) * (1 + rng.integers(0, 4, old.shape) / 4)
    scale = scale.astype(np.float16).astype(np.float64)
    scale[:, 5:20:3] = 0.0
    if fmt != "ternary":
        scale[:, 30:60][rng.random(scale[:, 30:60].shape) < 0.5] = 0.0
        scale[:, 60, 0] = scale[:, 61, -1] = 0.0
        W = h["W"].reshape(2, 96, 8, 128) / old[..., None] * scale[..., None]
    else:
        W = h["W"] / old[..., None] * scale[..., None]
    h["W"] = W.reshape(2, 96, 1024)
    d["packed"]["scale"].copy_(torch.from_numpy(scale).half())
    for gated in (False, True):
        out = torch.full((h["P"], 48 if gated else 96), 123.0, dtype=d["A"].dtype, device=d["A"].device)
        got = values(call(d["A"], d["packed"], d["off"], gated=gated, out=out))
        C, mag = OE.product(h["A"], h["W"], h["off"])
        want, bound = (OE.gated(C), gated_bound(1024, C, mag)) if gated else (C, sum_bound(1024, mag))
        over = {"f16": 65520.0, "bf16": 3.3961775e38}[dt]
        fine = np.abs(want) + bound < over
        assert_within(got[fine], want[fine], rounded(dt, bound, want)[fine], "scales")
        past = np.abs(want) - bound >= over  # a value within the bound of want is then past the type's range
        assert np.array_equal(got[past], np.sign(want[past]) * np.inf)
