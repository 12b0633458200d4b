"""Plan of a paged step and append to the paged cache, against the oracle's loops."""
import numpy as np
import pytest

import oracle.paged as OP
from gpu_common import log, require_gpu

pytestmark = pytest.mark.gpu


def _step(rng, B, width, page, ctx_hi, new_hi, spare):
    room = width * page
    ctx = rng.integers(0, min(ctx_hi, room) + 1, B)
    new = rng.integers(0, new_hi + 1, B)
    held = np.minimum(-(-ctx // page), width)
    need = np.minimum(-(-(ctx + new) // page), width)
    ids = rng.permutation(int(held.sum() + (need - held).sum()) + spare + 5)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += int(held[b])
    return ctx, new, table, ids[at:]


def _check_plan(ctx, new, table, free, head, tokens, page, pad_cols=0):
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    ref = OP.plan(ctx, new, table, free, head, tokens, page)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)  # noqa: E731
    wide = torch.full((len(ctx), table.shape[1] + pad_cols), -77, dtype=torch.int32, device=dev)
    tab = wide[:, :table.shape[1]]
    tab.copy_(i32(table))
    args = (i32(ctx), i32(new), tab, i32(free), i32([head]), tokens)
    for again in range(2):  # a step planned again gives the same plan
        r = tq.tq_paged_plan(*args, page_size=page)
        torch.cuda.synchronize()
        for name in ("cu_q", "kv_lens", "positions", "slots", "state"):
            assert getattr(r, name).tolist() == list(ref[name]), f"{name}, pass {again}"
        assert np.array_equal(tab.cpu().numpy(), ref["table"])
    assert bool((wide[:, table.shape[1]:] == -77).all())


@pytest.mark.parametrize("B,width,page,ctx_hi,new_hi", [
    (1, 4, 16, 40, 1), (1, 1, 16, 0, 16), (3, 9, 32, 100, 120), (64, 20, 16, 200, 1), (65, 33, 16, 250, 200),
    (257, 17, 64, 700, 300), (1025, 12, 16, 100, 80), (2049, 5, 128, 500, 60),
])
@pytest.mark.parametrize("spare", [40, 0])
def test_plan_matches_oracle(B, width, page, ctx_hi, new_hi, spare):
    log(f"plan B={B} width={width} page={page} spare={spare}")
    rng = np.random.default_rng(B * 7 + page)
    ctx, new, table, free = _step(rng, B, width, page, ctx_hi, new_hi, spare)
    _check_plan(ctx, new, table, free, 3, int(new.sum()), page, pad_cols=3)


@pytest.mark.parametrize("kind", ["short_list", "empty_list", "bad_ids", "missing_held", "padding", "too_few_tokens",
                                  "negative_lengths", "head_past_end", "all_rest"])
def test_plan_edges(kind):
    """Steps that run out of pages, name none, or get more or fewer token entries than they have tokens."""
    log(f"plan edge {kind}")
    rng = np.random.default_rng(5)
    ctx, new, table, free = _step(rng, 40, 12, 16, 150, 70, 10)
    head, tokens = 2, int(new.sum())
    if kind == "short_list":
        free = free[:30]
    elif kind == "empty_list":
        free, head = free[:0], 0
    elif kind == "bad_ids":
        free = free.copy()
        free[::3] = -5
    elif kind == "missing_held":
        table[::2] = -1
    elif kind == "padding":
        tokens += 37
    elif kind == "too_few_tokens":
        tokens -= 100
        table[3] = -1
        free = free[:40]
    elif kind == "negative_lengths":
        new = new.copy()
        ctx = ctx.copy()
        new[::4], ctx[1::4] = -9, -3
        tokens = int(np.maximum(new, 0).sum())
    elif kind == "head_past_end":
        head = len(free)
    elif kind == "all_rest":
        new = new * 0
        tokens = 0
    _check_plan(ctx, new, table, free, head, tokens, 16)


def test_plan_largest_batch_and_lengths_at_the_limit():
    """16384 requests; lengths near 2^31 stay in bounds and hold at 2^31 - 1."""
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    log("plan B=16384")
    rng = np.random.default_rng(9)
    ctx, new, table, free = _step(rng, 16384, 6, 16, 80, 3, 0)
    _check_plan(ctx, new, table, free, 0, int(new.sum()), 16)
    log("plan huge lengths")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    table = torch.zeros((2, 4), dtype=torch.int32, device=dev)
    r = tq.tq_paged_plan(i32([2**31 - 1, 5]), i32([10, 2**31 - 1]), table, i32([9, 8, 7, 6]), i32([0]), 4, page_size=16)
    assert r.kv_lens.tolist() == [2**31 - 1] * 2 and r.cu_q.tolist() == [0, 10, 2**31 - 1]
    assert r.slots.tolist() == [-1] * 4 and table.tolist() == [[0] * 4, [0, 9, 8, 7]]


# ------------------------------------------------------------------- append

def _tol(ref, mag, dt):
    """Two fp32 products and a sum (three roundings of 2^-24 on the terms), then one rounding to dt:
    half a step, relative or of the smallest fp16 subnormals."""
    import torch
    half = torch.finfo(dt).eps / 2
    fp32 = 3 * 2.0 ** -24 * mag
    return fp32 + half * (np.abs(ref) + fp32) + (2.0 ** -25 if dt == torch.float16 else 0.0)


def _check_append(T, Hq, Hkv, D, page, rot, dt, inter=False, layout="fused", pages=None, slots=None, positions=None,
                  P=300, page_gap=0):
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dt]
    log(f"append T={T} Hq={Hq} Hkv={Hkv} D={D} page={page} rot={rot} {dt} inter={inter} {layout}")
    g = torch.Generator().manual_seed(T * 31 + D + rot)
    pages = pages or -(-T // page) + 2
    n = Hq + 2 * Hkv
    x = torch.randn((T, n, D), generator=g).to(dt)
    if layout == "fused":
        xd = x.to(dev)
        q, k, v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    elif layout == "odd":       # strides and start that no 16-byte vector fits
        xd = torch.zeros((T * n * (D + 3) + 1,), dtype=dt, device=dev)[1:].view(T, n, D + 3)[..., :D]
        xd.copy_(x)
        q, k, v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    else:                       # heads first
        xd = x.transpose(0, 1).contiguous().to(dev).transpose(0, 1)
        q, k, v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    body = Hkv * page * D
    caches = [torch.randn((pages, body + page_gap), generator=g).to(dt) for _ in range(2)]
    kc, vc = [c.to(dev)[:, :body].unflatten(1, (Hkv, page, D)) for c in caches]
    before = [c[:, :body].unflatten(1, (Hkv, page, D)).double().numpy() for c in caches]
    if slots is None:
        slots = torch.randperm(pages * page, generator=g)[:T]
    if positions is None:
        positions = torch.randint(0, P, (T,), generator=g, dtype=torch.int32)
    rope = ang = None
    if rot:
        ang = torch.rand((P, rot // 2), generator=g, dtype=torch.float64) * 6
        rope = torch.cat([ang.cos(), ang.sin()], 1).float()
    x64 = x.double().numpy()
    rq, mq = OP.rotate(x64[:, :Hq], None if rope is None else rope.numpy(), positions, inter)
    rk, mk = OP.rotate(x64[:, Hq:Hq + Hkv], None if rope is None else rope.numpy(), positions, inter)
    out = tq.tq_kv_append(q if Hq else None, k, v, kc, vc, slots.to(dev), positions.to(dev) if rot else None,
                          rope.to(dev) if rot else None, interleaved=inter)
    torch.cuda.synchronize()
    inside = [t for t in range(T) if 0 <= int(slots[t]) < pages * page]
    for got, want, tol in (
            (out, rq, _tol(rq, mq, dt)) if Hq else (None, None, None),
            (kc, OP.store(before[0], rk, slots), OP.store(before[0] * 0, _tol(rk, mk, dt), slots)),
            (vc, OP.store(before[1], x64[:, Hq + Hkv:], slots), np.zeros_like(before[1]))):
        if got is None:
            continue
        got = got.double().cpu().numpy()
        bad = np.isnan(want)
        assert np.isnan(got[bad]).all() and (np.abs(got - want)[~bad] <= tol[~bad]).all()
    assert not Hq or (out.is_contiguous() and out.dtype == dt)
    return inside


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,page,rot", [
    (1, 32, 8, 128, 16, 128), (3, 7, 1, 64, 32, 64), (17, 6, 2, 128, 64, 64), (129, 4, 4, 64, 128, 32),
    (700, 8, 2, 128, 16, 128), (5, 2, 1, 64, 1024, 0), (9, 3, 1, 96, 16, 48), (4, 2, 2, 80, 16, 20),
    (3, 1, 1, 7, 16, 6), (2, 5, 3, 256, 16, 256), (1, 1, 1, 1, 16, 0),
])
def test_append_matches_oracle(dt, inter, T, Hq, Hkv, D, page, rot):
    _check_append(T, Hq, Hkv, D, page, rot, dt, inter)


@pytest.mark.parametrize("layout", ["odd", "heads_first"])
@pytest.mark.parametrize("rot", [0, 64])
def test_append_strides(layout, rot):
    _check_append(33, 4, 2, 64, 16, rot, "bf16", layout=layout)
    _check_append(33, 4, 2, 64, 16, rot, "f16", inter=True, layout=layout, page_gap=8)
    _check_append(33, 4, 2, 64, 16, rot, "f16", page_gap=5)


def test_append_without_queries_and_nothing():
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    _check_append(19, 0, 2, 64, 16, 64, "f16")
    kc = torch.zeros((2, 1, 16, 64), dtype=torch.float16, device=dev)
    e = torch.empty((0, 1, 64), dtype=torch.float16, device=dev)
    assert tq.tq_kv_append(e, e, e, kc, kc.clone(), torch.empty(0, dtype=torch.int64, device=dev)).shape == (0, 1, 64)


def test_append_slots_and_positions_outside():
    """Slots of no page store nothing; positions outside the table give NaN; neither leaves the buffers."""
    import torch
    slots = torch.tensor([-1, 3, 4 * 16, 1 << 40, -(1 << 40), 63, 4 * 16 - 2, 17])
    assert _check_append(8, 2, 1, 64, 16, 0, "f16", pages=4, slots=slots) == [1, 5, 6, 7]
    pos = torch.tensor([0, -1, 299, 300, 2**31 - 1, -2**31, 5, 6], dtype=torch.int32)
    _check_append(8, 2, 1, 64, 16, 32, "bf16", pages=4, positions=pos, slots=slots)
    _check_append(8, 2, 1, 7, 16, 6, "bf16", pages=4, positions=pos, slots=slots)
    _check_append(8, 2, 1, 64, 16, 64, "f16", inter=True, pages=4, positions=pos, slots=slots)


def test_append_cache_past_32_bits():
    """Slots in the last page of a cache of more than 2^32 bytes."""
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    pages = 2**31 // (8 * 64 * 128) + 3  # more than 2^31 elements
    log(f"append {pages} pages of 8 x 64 x 128")
    kc = torch.empty((pages, 8, 64, 128), dtype=torch.bfloat16, device=dev)
    vc = torch.empty_like(kc)
    kc[-1].zero_(), vc[-1].zero_(), kc[0].zero_(), vc[0].zero_()
    k, v = [torch.randn((2, 8, 128), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    slots = torch.tensor([pages * 64 - 1, pages * 64 - 30], device=dev)
    tq.tq_kv_append(None, k, v, kc, vc, slots)
    for c, x in ((kc, k), (vc, v)):
        assert torch.equal(c[-1, :, 63], x[0]) and torch.equal(c[-1, :, 34], x[1])
        assert int(c[-1].count_nonzero()) <= 2 * 8 * 128 and int(c[0].count_nonzero()) == 0
