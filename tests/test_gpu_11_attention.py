"""Paged attention against the fp64 oracle: lengths, heads, pages, windows, empty rows, masked values that are not
finite, bad pages, strides, splits, graphs.

Tolerance of an output, from the roundings of the method (half steps; u = finfo(dt).eps / 2):
* a score sums D exact products in fp32, at most (D + 8) 2^-23 of sum |q k|, and takes part in an exponent of base 2
  with three more fp32 roundings of its size and of the maximum's (2^-23 of each), and the exponential itself is
  good to 2^-21: together `e`, relative, on each weight, in numerator and in denominator;
* each weight is rounded to dt: u, relative (fp16: at least 2^-25 of a weight of 1);
* the fp32 sums over n keys: (n / 32 + 64) 2^-23 of the sum of weight |v|;
* the output is rounded to dt: u |out| (fp16: 2^-25 for subnormals).
"""
import numpy as np
import pytest

import oracle.attention as OA
from gpu_common import log, require_gpu

pytestmark = pytest.mark.gpu


def _bounds(ref, D, n, dt):
    import torch
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    e = (D + 8) * 2.0 ** -23 * ref["smag"] + 6 * 2.0 ** -23 * ref["smag"] + 2.0 ** -21
    acc = (n / 32 + 64) * 2.0 ** -23
    out = ref["mag"] * (2 * e[..., None] + u + 2 * acc) + tiny * ref["wmax"]
    out = out + u * (np.abs(ref["out"]) + out) + tiny
    with np.errstate(invalid="ignore"):
        lse = e + acc + 2.0 ** -22 * np.abs(ref["lse"]) + 1e-6
    return out, lse


def _share(err, tol):
    """Largest error as a share of its tolerance; where none is allowed (rows of zeros) any error is infinite."""
    share = np.divide(err, tol, out=np.where(err > 0, np.inf, 0.0), where=tol > 0)
    return float(share.max()) if share.size else 0.0


class Case:
    """Requests with the given new-token counts and key counts over a shuffled paged cache (CPU tensors)."""

    def __init__(self, qn, kv, Hq, Hkv, D, page, dt, seed=0, spare=3, qscale=2.0, extra_cols=0):
        import torch
        self.dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dt]
        g = torch.Generator().manual_seed(seed * 1000 + sum(qn) + 7 * sum(kv) + D + page)
        self.qn, self.kvl, self.Hq, self.Hkv, self.D, self.page = list(qn), list(kv), Hq, Hkv, D, page
        blocks = [-(-x // page) for x in kv]
        width = max(max(blocks), 1) + extra_cols
        pages = sum(blocks) + spare
        ids = torch.randperm(pages, generator=g, dtype=torch.int32)
        self.table = torch.full((len(qn), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(blocks):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.k = torch.randn((pages, Hkv, page, D), generator=g).to(self.dt)
        self.v = torch.randn((pages, Hkv, page, D), generator=g).to(self.dt)
        self.q = (torch.randn((sum(qn), Hq, D), generator=g) * qscale).to(self.dt)
        self.cu = torch.tensor([0] + list(np.cumsum(qn)), dtype=torch.int32)
        self.kv = torch.tensor(self.kvl, dtype=torch.int32)

    def run(self, window=0, sinks=0, scale=None, workspace="auto", lse=True, q=None, caches=None, table=None, max_kv=None,
            out=None):
        import torch
        import bit_weight_only_tq_amd as tq
        dev = require_gpu()
        d = lambda t: t.to(dev)  # noqa: E731
        kc, vc = caches or (d(self.k), d(self.v))
        r = tq.tq_paged_attention(d(self.q) if q is None else q, kc, vc, d(self.table) if table is None else table,
                                  d(self.cu), d(self.kv), max(max(self.qn), 1),
                                  max(self.kvl) if max_kv is None else max_kv, scale=scale, window=window, sinks=sinks,
                                  return_lse=lse, workspace=workspace, out=out)
        torch.cuda.synchronize()
        return r

    def check(self, got, window=0, sinks=0, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        f = lambda t: t.double().numpy()  # noqa: E731
        ref = OA.attend(f(self.q), f(self.k), f(self.v), self.table.numpy(), self.cu.tolist(), self.kvl, scale, window,
                        sinks)
        out, lse = [x.double().cpu().numpy() for x in got]
        tol, ltol = _bounds(ref, self.D, max(self.kvl), self.dt)
        nan = np.isnan(ref["out"])
        assert np.array_equal(np.isnan(out), nan)
        fin = np.isfinite(ref["out"])
        assert np.array_equal(out[~fin & ~nan], ref["out"][~fin & ~nan])
        err = _share(np.abs(out - ref["out"])[fin], tol[fin])
        assert err <= 1, f"out {err} of its tolerance"
        empty = np.isneginf(ref["lse"])
        assert np.isneginf(lse[empty]).all() and (out[empty] == 0).all()
        ok = np.isfinite(ref["lse"])
        lerr = _share(np.abs(lse[ok] - ref["lse"][ok]), ltol[ok])
        assert lerr <= 1, f"lse {lerr} of its tolerance"
        print(f"  out {err:.3f} lse {lerr:.3f} of tolerance", flush=True)


def _go(qn, kv, Hq, Hkv, D, page, dt, window=0, sinks=0, **kw):
    log(f"attend qn={qn} kv={kv} Hq={Hq} Hkv={Hkv} D={D} page={page} {dt} window={window} sinks={sinks} {kw}")
    c = Case(qn, kv, Hq, Hkv, D, page, dt, **kw)
    got = c.run(window, sinks)
    c.check(got, window, sinks)
    c.check(c.run(window, sinks, workspace=None), window, sinks)
    return c, got


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (7, 1), (16, 1), (12, 4)])
def test_decode_lengths(dt, D, Hq, Hkv):
    """One token over 1 .. 600 keys: block, page and split edges."""
    kv = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 256, 257, 300, 600]
    _go([1] * len(kv), kv, Hq, Hkv, D, 16, dt)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_pages(page, dt):
    _go([1, 2, 5, 1, 40], [page, page + 1, 2 * page - 1, 777, 333], 8, 2, 128, page, dt)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (3, 1, 128), (7, 1, 64), (5, 5, 128), (32, 1, 64)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_new_tokens(Hq, Hkv, D, dt):
    """Requests of 0 .. 150 new tokens in one call: none, one, a few rows past a tile, a chunk."""
    qn = [1, 0, 2, 3, 5, 16, 17, 0, 33, 64, 150]
    kv = [50, 40, 2, 90, 5, 16, 300, 0, 33, 200, 151]
    _go(qn, kv, Hq, Hkv, D, 16, dt)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (31, 4), (32, 32), (33, 17), (100, 1), (100, 130), (5000, 4)])
@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
def test_window_and_sinks(window, sinks, dt, D):
    qn = [1, 1, 1, 4, 40, 130, 1]
    kv = [10, 300, 1000, 290, 40, 400, 101]
    _go(qn, kv, 6, 2, D, 16, dt, window, sinks)


@pytest.mark.parametrize("qn,kv", [([1], [5000]), ([3, 1], [9000, 4000]), ([2, 1, 1], [4097, 1, 2500])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3001, 5)])
def test_long_keys_split(qn, kv, window, sinks):
    """The key axis split over workgroups: within tolerance, and the same bits each time."""
    import torch
    c, got = _go(qn, kv, 8, 2, 128, 16, "bf16", window, sinks)
    again = c.run(window, sinks)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    small = c.run(window, sinks, max_kv=17)  # a wrong bound of the lengths changes the schedule, not the result
    c.check(small, window, sinks)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_rows_that_see_nothing(dt):
    """No keys, or more new tokens than keys: zeros and -inf for the rows before the first key."""
    _go([1, 3, 4, 70, 1], [0, 0, 2, 30, 20], 8, 2, 64, 16, dt)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), "lowest"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_hidden_places_hold_anything(value, dt, window, sinks):
    """Keys and values past the lengths, in unused pages and before the window are not finite: nothing shows."""
    import torch
    log(f"hidden {value} {dt} window={window}")
    c = Case([1, 3, 40, 1, 1], [77, 50, 90, 400, 1], 8, 2, 64, 16, dt)
    v = torch.finfo(c.dt).min if value == "lowest" else value
    keep = torch.zeros((c.k.shape[0], 16), dtype=torch.bool)
    for b, n in enumerate(c.kvl):
        for p in range(n - c.qn[b], n):
            for j in OA.visible(p, n, window, sinks):
                keep[int(c.table[b, j // 16]), j % 16] = True
    hide = ~keep[:, None, :, None].expand_as(c.k)
    c.k[hide], c.v[hide] = v, v
    if window:  # pages wholly before the window may be gone from the table
        for b, n in enumerate(c.kvl):
            for blk in range(n // 16):
                if not keep[int(c.table[b, blk])].any():
                    c.table[b, blk] = -1
    c.check(c.run(window, sinks), window, sinks)
    c.check(c.run(window, sinks, workspace=None), window, sinks)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("window", [0, 20])
def test_values_some_rows_see(value, dt, D, window):
    """A value that is not finite reaches the rows that see it and no other row."""
    log(f"partly hidden {value} {dt} window={window}")
    c = Case([40, 5, 300], [60, 300, 300], 4, 2, D, 16, dt)
    for b, j in ((0, 37), (0, 50), (1, 297), (2, 100), (2, 250)):
        c.v[int(c.table[b, j // 16]), :, j % 16, (j * 3) % D] = value
    c.check(c.run(window, 0), window, 0)


def test_nan_keys_and_queries():
    """NaN in a visible key or a query gives NaN in the rows that meet it, nowhere else."""
    log("nan keys and queries")
    c = Case([40, 1, 3], [60, 300, 100], 8, 2, 64, 16, "bf16")
    c.k[int(c.table[0, 2]), 0, 5] = float("nan")  # key 37 of request 0, KV head 0
    c.q[41, 3] = float("nan")
    c.check(c.run())


def test_bad_pages_count_as_absent():
    """Page ids outside the cache are never read: their keys are left out."""
    log("bad pages")
    c = Case([1, 2, 40], [200, 90, 130], 8, 2, 128, 16, "f16")
    c.table[0, 3], c.table[0, 12], c.table[1, 5], c.table[2, 0], c.table[2, 7] = -1, 2**31 - 1, c.k.shape[0], -2**31, 999999
    c.check(c.run())
    c.check(c.run(60, 20), 60, 20)


def test_table_narrower_than_the_lengths():
    """Keys past the table's width are not there."""
    log("narrow table")
    c = Case([1, 3], [200, 64], 4, 1, 64, 16, "bf16")
    c.table = c.table[:, :5].contiguous()
    c.check(c.run())


def test_offsets_outside_the_tokens_are_skipped():
    """A request whose offsets leave [0, T] is skipped and writes nothing."""
    import torch
    log("bad offsets")
    c = Case([2, 3, 1], [40, 50, 60], 4, 2, 64, 16, "f16")
    out = torch.full((6, 4, 64), 7.0, dtype=c.dt, device=require_gpu())
    c.cu = torch.tensor([-2, 3, 2, 9], dtype=torch.int32)  # negative start, negative count, end past T
    c.run(out=out)
    assert bool((out == 7).all())


@pytest.mark.parametrize("gap", [0, 8])
def test_strides(gap):
    """Queries as part of a fused projection, heads first, caches with gaps, a wider table."""
    import torch
    log(f"strides gap={gap}")
    dev = require_gpu()
    c = Case([1, 7, 33], [100, 60, 70], 4, 2, 64, 16, "bf16", extra_cols=3)
    T = c.q.shape[0]
    fused = torch.randn((T, 8, 64 + gap), device=dev).to(c.dt)
    q = fused[:, 1:5, :64]
    q.copy_(c.q)
    body = 2 * 16 * 64
    caches = []
    for x in (c.k, c.v):
        wide = torch.full((x.shape[0], body + gap), float("nan"), dtype=c.dt, device=dev)
        wide[:, :body] = x.reshape(-1, body).to(dev)
        caches.append(wide[:, :body].unflatten(1, (2, 16, 64)))
    wide = torch.full((3, c.table.shape[1] + 5), 1 << 30, dtype=torch.int32, device=dev)
    table = wide[:, :c.table.shape[1]]
    table.copy_(c.table)
    c.check(c.run(q=q, caches=caches, table=table))
    qh = c.q.to(dev).transpose(0, 1).contiguous().transpose(0, 1)
    c.check(c.run(q=qh))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 20.0])
def test_scales(dt, scale):
    """From near-uniform weights to one key that takes all; scores of hundreds."""
    log(f"scale {scale} {dt}")
    c = Case([1, 3, 50], [500, 40, 90], 8, 2, 64, 16, dt)
    c.check(c.run(scale=scale), scale=scale)


def test_growing_scores():
    """Maxima that rise along the keys (every block rescales) and fall (none does)."""
    import torch
    for sign in (1, -1):
        log(f"growing {sign}")
        c = Case([1, 40], [2000, 700], 4, 1, 64, 16, "bf16")
        for b, n in enumerate(c.kvl):
            for j in range(n):
                c.k[int(c.table[b, j // 16]), 0, j % 16] = sign * j * 0.02
        c.q = (c.q.abs() + 0.5).to(torch.bfloat16)
        c.check(c.run())


def test_cache_past_32_bits():
    """Pages at the end of a cache of more than 2^31 elements."""
    import torch
    dev = require_gpu()
    c = Case([1, 5], [100, 300], 8, 8, 128, 64, "bf16")
    pages = 2**31 // (8 * 64 * 128) + 20
    log(f"attend {pages} pages of 8 x 64 x 128")
    big = [torch.empty((pages, 8, 64, 128), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    n = c.k.shape[0]
    for x, src in zip(big, (c.k, c.v)):
        x[-n:] = src.to(dev)
    table = torch.where(c.table >= 0, c.table + (pages - n), c.table).to(dev)
    c.check(c.run(caches=big, table=table))


def test_other_stream_and_graph():
    """On a side stream, and captured with one workspace: every replay equals the eager call."""
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    log("stream and graph")
    c = Case([1, 1, 20], [3000, 700, 500], 8, 2, 128, 16, "bf16")
    eager = c.run()
    ws = tq.new_workspace(tq.tq_paged_attention_workspace_bytes(22, 8, 2, 128, 3, 20, 3000), dev)
    d = [t.to(dev) for t in (c.q, c.k, c.v, c.table, c.cu, c.kv)]
    out = torch.empty_like(eager[0])
    call = lambda: tq.tq_paged_attention(*d, 20, 3000, out=out, return_lse=True, workspace=ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _, lse = call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, lse = call()
    for i in range(4):
        out.fill_(0), lse.fill_(0)
        torch.randn(1000, device=dev).sum()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1]), f"replay {i}"
    if ws is not None:
        assert int(ws[:tq.TQ_WORKSPACE_FLAG_BYTES].count_nonzero()) == 0


def test_no_tokens_and_no_lse():
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    c = Case([2], [40], 4, 2, 64, 16, "f16")
    full = c.run()
    assert torch.equal(c.run(lse=False), full[0])
    d = [t.to(dev) for t in (c.q[:0], c.k, c.v, c.table, torch.zeros(2, dtype=torch.int32), c.kv)]
    assert tq.tq_paged_attention(*d, 1, 40).shape == (0, 4, 64)
