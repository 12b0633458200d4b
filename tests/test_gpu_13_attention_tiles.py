"""Paged attention of prompt chunks (more than 64 rows of a KV head: the 128-row matrix-core kernel) against the fp64
oracle, with the tolerances derived in test_gpu_11_attention: row and key tile edges, batches, splits, windows, values
that are not finite, bad pages and offsets, strides, graphs."""
import pytest

import oracle.attention as OA
from gpu_common import log, require_gpu
from test_gpu_11_attention import Case, _go

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [64, 65, 96, 97, 127, 128, 129, 191, 257])
def test_row_edges(n, D, dt):
    """One head a group: rows are tokens; alone and beside a decoding request, over a context of odd length."""
    _go([n], [n + 77], 2, 2, D, 16, dt)
    _go([n, 1], [n, 130], 1, 1, D, 32, dt)


@pytest.mark.parametrize("dt,D", [("f16", 128), ("bf16", 64)])
@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (14, 2), (16, 1), (40, 1)])
def test_groups(Hq, Hkv, D, dt):
    """Groups that do not divide a tile: a token's heads fall into two workgroups."""
    _go([50, 3, 23], [200, 3, 64], Hq, Hkv, D, 16, dt)


@pytest.mark.parametrize("kv", [1, 63, 64, 65, 127, 128, 129, 192, 193])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_key_edges(kv, page):
    """Lengths at the edges of the 64-key tiles and of the pages; fewer keys than new tokens leave rows empty."""
    _go([70], [kv], 2, 1, 128, page, "bf16")
    _go([70, 100], [kv, kv + 30], 1, 1, 64, page, "f16")


def test_batch():
    """150 requests of 0 to 200 new tokens: every tile finds its request."""
    qn = [(0, 1, 7, 70, 33, 0, 129, 2, 64, 65, 1, 200)[(5 * b) % 12] for b in range(150)]
    _go(qn, [n + (37 * b) % 90 for b, n in enumerate(qn)], 2, 1, 64, 16, "bf16")


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 128), (2, 2, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2500, 70)])
def test_splits(Hq, Hkv, D, window, sinks):
    """A long context for few rows: keys split over workgroups, the same bits each time."""
    import torch
    c, got = _go([90], [5000], Hq, Hkv, D, 16, "bf16", window, sinks)
    again = c.run(window, sinks)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    _go([90, 3, 140], [4500, 4000, 145], Hq, Hkv, D, 64, "f16", window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (63, 0), (64, 64), (65, 17), (100, 130), (300, 1), (4000, 4)])
@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
def test_window_and_sinks(window, sinks, dt, D):
    _go([150, 1, 70], [400, 300, 70], 2, 1, D, 16, dt, window, sinks)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), "lowest"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
@pytest.mark.parametrize("dt,D", [("f16", 128), ("bf16", 64)])
def test_hidden_places_hold_anything(value, window, sinks, dt, D):
    """Keys and values that no new token sees are not finite, pages wholly before the window are gone: nothing shows."""
    import torch
    log(f"hidden {value} {dt} window={window}")
    c = Case([100, 70], [190, 401], 2, 1, D, 16, dt)
    v = torch.finfo(c.dt).min if value == "lowest" else value
    keep = torch.zeros((c.k.shape[0], 16), dtype=torch.bool)
    for b, n in enumerate(c.kvl):
        for p in range(n - c.qn[b], n):
            for j in OA.visible(p, n, window, sinks):
                keep[int(c.table[b, j // 16]), j % 16] = True
    hide = ~keep[:, None, :, None].expand_as(c.k)
    c.k[hide], c.v[hide] = v, v
    if window:
        for b, n in enumerate(c.kvl):
            for blk in range(n // 16):
                if not keep[int(c.table[b, blk])].any():
                    c.table[b, blk] = -1
    c.check(c.run(window, sinks), window, sinks)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("window", [0, 20])
def test_values_some_rows_see(value, dt, D, window):
    """A value that is not finite reaches the rows that see it and no other row."""
    log(f"partly hidden {value} {dt} window={window}")
    c = Case([80, 65, 300], [100, 300, 300], 4, 2, D, 16, dt)
    for b, j in ((0, 37), (0, 50), (0, 99), (1, 297), (2, 100), (2, 130), (2, 250)):
        c.v[int(c.table[b, j // 16]), :, j % 16, (j * 3) % D] = value
    c.check(c.run(window, 0), window, 0)


def test_nan_keys_and_queries():
    log("nan keys and queries")
    c = Case([70, 90], [160, 300], 4, 2, 64, 16, "bf16")
    c.k[int(c.table[0, 6]), 0, 9] = float("nan")  # key 105 of request 0, KV head 0
    c.q[71, 3] = float("nan")
    c.check(c.run())


def test_bad_pages_and_narrow_table():
    """Page ids outside the cache and keys past the table's width are left out."""
    log("bad pages")
    c = Case([70, 90], [200, 330], 4, 2, 128, 16, "f16")
    c.table[0, 3], c.table[0, 12], c.table[1, 0], c.table[1, 7], c.table[1, 20] = -1, 2**31 - 1, c.k.shape[0], -2**31, 999999
    c.check(c.run())
    c.check(c.run(60, 20), 60, 20)
    c.table = c.table[:, :9].contiguous()
    c.check(c.run())


def test_offsets_outside_the_tokens():
    """The requests before a bad offset are computed; one that leaves [0, T] or ends before it begins writes nothing."""
    import torch
    log("bad offsets")
    c = Case([90, 40, 50], [100, 50, 60], 4, 2, 64, 16, "f16")
    full = c.run()[0]
    out = torch.full((180, 4, 64), 7.0, dtype=c.dt, device=require_gpu())
    c.cu = torch.tensor([0, 90, 5000, 180], dtype=torch.int32)
    c.run(out=out)
    assert torch.equal(out[:90], full[:90]) and bool((out[90:] == 7).all())


def test_strides():
    """Queries inside a fused projection, heads first, caches with gaps, a wider table."""
    import torch
    log("strides")
    dev = require_gpu()
    c = Case([80, 7, 133], [100, 60, 170], 4, 2, 64, 16, "bf16", extra_cols=3)
    T = c.q.shape[0]
    fused = torch.randn((T, 8, 72), device=dev).to(c.dt)
    q = fused[:, 1:5, :64]
    q.copy_(c.q)
    body = 2 * 16 * 64
    caches = []
    for x in (c.k, c.v):
        wide = torch.full((x.shape[0], body + 8), float("nan"), dtype=c.dt, device=dev)
        wide[:, :body] = x.reshape(-1, body).to(dev)
        caches.append(wide[:, :body].unflatten(1, (2, 16, 64)))
    wide = torch.full((3, c.table.shape[1] + 5), 1 << 30, dtype=torch.int32, device=dev)
    table = wide[:, :c.table.shape[1]]
    table.copy_(c.table)
    c.check(c.run(q=q, caches=caches, table=table))
    c.check(c.run(q=c.q.to(dev).transpose(0, 1).contiguous().transpose(0, 1)))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 20.0])
def test_scales(dt, scale):
    log(f"scale {scale} {dt}")
    c = Case([90, 65], [300, 65], 4, 2, 64, 16, dt)
    c.check(c.run(scale=scale), scale=scale)


def test_growing_scores():
    """Maxima that rise along the keys (every tile rescales) and fall (none does)."""
    import torch
    for sign in (1, -1):
        log(f"growing {sign}")
        c = Case([140], [1500], 2, 1, 64, 16, "bf16")
        for j in range(1500):
            c.k[int(c.table[0, j // 16]), 0, j % 16] = sign * j * 0.02
        c.q = (c.q.abs() + 0.5).to(torch.bfloat16)
        c.check(c.run())


def test_cache_past_32_bits():
    import torch
    dev = require_gpu()
    c = Case([70, 5], [100, 300], 8, 8, 128, 64, "bf16")
    pages = 2**31 // (8 * 64 * 128) + 20
    log(f"tiles {pages} pages of 8 x 64 x 128")
    big = [torch.empty((pages, 8, 64, 128), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    n = c.k.shape[0]
    for x, src in zip(big, (c.k, c.v)):
        x[-n:] = src.to(dev)
    table = torch.where(c.table >= 0, c.table + (pages - n), c.table).to(dev)
    c.check(c.run(caches=big, table=table))


def test_graph_of_a_mixed_step():
    """Both kernels in one captured call with one workspace: every replay equals the eager call."""
    import torch
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    log("graph")
    c = Case([1, 1, 90], [3000, 700, 5000], 8, 2, 128, 16, "bf16")
    eager = c.run()
    ws = tq.new_workspace(tq.tq_paged_attention_workspace_bytes(92, 8, 2, 128, 3, 90, 5000), dev)
    d = [t.to(dev) for t in (c.q, c.k, c.v, c.table, c.cu, c.kv)]
    out = torch.empty_like(eager[0])
    call = lambda: tq.tq_paged_attention(*d, 90, 5000, out=out, return_lse=True, workspace=ws)  # noqa: E731
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
    assert int(ws[:tq.TQ_WORKSPACE_FLAG_BYTES].count_nonzero()) == 0
