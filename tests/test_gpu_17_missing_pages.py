"""Paged attention where the first page that is not there lies inside a run of key tiles, behind tiles that every row
sees whole, against the fp64 oracle (tolerances derived in test_gpu_11_attention).

Keys of such pages count as not there whatever tile, wave or split meets the first of them: after the first tile of a
workgroup's run, on the last page alone, on pages that one wave looks up, with waves that have no rows.
"""
import pytest
import torch

import oracle.attention as OA
from gpu_common import log, require_gpu
from test_gpu_11_attention import Case

pytestmark = pytest.mark.gpu

TILE = 64  # keys


def _check(qn, kv, missing, Hq, Hkv, D, page, dt, window=0, sinks=0):
    """missing: (request, first key of the page, id in its place)."""
    log(f"missing {missing} qn={qn} kv={kv} Hq={Hq} Hkv={Hkv} D={D} page={page} {dt} window={window} sinks={sinks}")
    c = Case(qn, kv, Hq, Hkv, D, page, dt)
    for b, key, bad in missing:
        c.table[b, key // page] = bad
    c.check(c.run(window, sinks), window, sinks)
    c.check(c.run(window, sinks, workspace=None), window, sinks)


@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("tile", [2, 3, 7])
@pytest.mark.parametrize("n", [130, 128, 97, 33])
def test_first_gap_behind_whole_tiles(n, tile, dt, D):
    """A chunk over a context of twelve tiles: one page of 16 keys gone, of each wave's in turn, or a whole tile's."""
    ctx = 12 * TILE
    for w in range(4):
        _check([n], [ctx + n], [(0, tile * TILE + 16 * w, -1)], 2, 1, D, 16, dt)
    _check([n, 1], [ctx + n, 90], [(0, tile * TILE + 16 * w, -1) for w in range(4)], 1, 1, D, 16, dt)
    _check([n], [ctx + n], [(0, tile * TILE, 1 << 30), (0, (tile + 2) * TILE + 32, -5)], 2, 2, D, 64, dt)


@pytest.mark.parametrize("dt,D", [("f16", 128), ("bf16", 64)])
@pytest.mark.parametrize("key", [256, 512, 768])
def test_large_pages(key, dt, D):
    """Pages of four tiles: the second, third or fourth is gone, and the rest of the context with it."""
    _check([150], [1100], [(0, key, -1)], 2, 1, D, 256, dt)
    _check([150, 2], [1100, 700], [(0, k, -1) for k in range(key, 1100, 256)] + [(1, 512, -1)], 2, 1, D, 256, dt)


@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("rows", [1, 2, 4])
def test_waves_without_rows(rows, dt, D):
    """Decoding requests beside a chunk: three waves of their tiles have no rows; the last page, or one inside, is gone."""
    for kv, key in ((200, 192), (200, 128), (257, 256), (500, 320), (500, 400), (700, 688)):
        _check([rows, 60, rows], [kv, 90, kv + 13], [(0, key, -1)], 1, 1, D, 16, dt)
        _check([60, rows], [300, kv], [(1, key, -1)], 2, 2, D, 16, dt)


@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
def test_gap_in_a_later_split(dt, D):
    """Few rows over a long context, whose keys are split: gaps in the middle of the splits' runs."""
    for keys in ([11 * TILE], [40 * TILE + 16], [12 * TILE, 30 * TILE + 48, 62 * TILE]):
        _check([90], [4200], [(0, k, -1) for k in keys], 2, 1, D, 16, dt)


@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
def test_released_pages_behind_the_sinks(dt, D):
    """130 sinks, and the pages between them and the window gone: the third tile of the sinks has gaps."""
    n, kv, window, sinks = 100, 1500, 300, 130
    c = Case([n], [kv], 2, 1, D, 16, dt)
    seen = {j for p in range(kv - n, kv) for j in OA.visible(p, kv, window, sinks)}
    gone = [j for j in range(0, kv, 16) if not any(j + i in seen for i in range(16))]
    assert min(gone) == 144
    _check([n], [kv], [(0, j, -1) for j in gone], 2, 1, D, 16, dt, window, sinks)
    _check([n, 1, 2], [kv, 1000, 64], [(0, j, -1) for j in gone], 2, 1, D, 16, dt, window, sinks)


@pytest.mark.parametrize("dt,D", [("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("pages_left", [0, 3, 9, 20])
def test_step_that_runs_out_of_pages(pages_left, dt, D):
    """Plan, append and attention of a step whose free list ends inside a chunk: its last keys have no page."""
    import bit_weight_only_tq_amd as tq
    dev = require_gpu()
    log(f"free list of {pages_left} {dt} D={D}")
    qn, kv = [1, 300, 1], [400, 700, 333]
    c = Case(qn, kv, 2, 1, D, 16, dt)
    ctx = [b - a for a, b in zip(qn, kv)]
    free = []
    for b, (was, now) in enumerate(zip(ctx, kv)):
        for blk in range(-(-was // 16), -(-now // 16)):
            free.append(int(c.table[b, blk]))
            c.table[b, blk] = -1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    table, kc, vc = c.table.to(dev), c.k.to(dev), c.v.to(dev)
    T = sum(qn)
    plan = tq.tq_paged_plan(i32(ctx), i32(qn), table, i32(free[:pages_left]), i32([0]), T)
    assert plan.state.tolist()[0] == min(pages_left, len(free))
    assert (plan.state.tolist()[1] > 0) == (pages_left < len(free))
    g = torch.Generator().manual_seed(pages_left)
    k, v = [torch.randn((T, 1, D), generator=g).to(c.dt).to(dev) for _ in range(2)]
    tq.tq_kv_append(None, k, v, kc, vc, plan.slots)
    torch.cuda.synchronize()
    c.table, c.k, c.v = table.cpu(), kc.cpu(), vc.cpu()
    assert plan.cu_q.tolist() == c.cu.tolist() and plan.kv_lens.tolist() == kv
    c.check(c.run())
    c.check(c.run(workspace=None))
