"""Plan of a paged step and append to a paged cache, in plain loops (fp64).

The specification the GPU kernels are compared with: every request takes its
fresh pages from the free list in request order, every token is placed on its
own, and rotary positions turn each pair of dimensions by its angle.
"""

import numpy as np


def plan(ctx, new, table, free, head, tokens, page):
    """-> dict of table (a copy), cu_q, kv_lens, positions, slots, state (see tq_paged_plan)."""
    table = np.array(table, dtype=np.int64)
    width = table.shape[1]
    cu, kv, positions, slots = [0], [], [], []
    lost = 0
    for b in range(len(ctx)):
        c, n = max(int(ctx[b]), 0), max(int(new[b]), 0)
        for blk in range(-(-c // page), -(-(c + n) // page)):
            if blk >= width:
                break
            table[b, blk] = free[head] if head < len(free) else -1
            head = min(head + 1, len(free))
        for pos in range(c, c + n):
            blk = pos // page
            pg = int(table[b, blk]) if blk < width else -1
            slot = pg * page + pos % page if pg >= 0 else -1
            if len(positions) < tokens:
                positions.append(pos)
                slots.append(slot)
                lost += slot < 0
            else:
                lost += 1
        cu.append(cu[-1] + n)
        kv.append(c + n)
    pad = tokens - len(positions)
    return {"table": table, "cu_q": cu, "kv_lens": kv, "positions": positions + [0] * pad,
            "slots": slots + [-1] * pad, "state": [head, lost]}


def rotate(x, rope, positions, interleaved):
    """x [T, H, D] fp64 -> (turned, sum of |terms|): the pairs (i, i + rot/2), or (2i, 2i + 1), turned."""
    y, mag = np.array(x, dtype=np.float64), np.abs(np.array(x, dtype=np.float64))
    if rope is None:
        return y, mag
    half = rope.shape[1] // 2
    for t in range(x.shape[0]):
        p = int(positions[t])
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            if not 0 <= p < rope.shape[0]:
                y[t, :, a] = y[t, :, b] = mag[t, :, a] = mag[t, :, b] = np.nan
                continue
            c, s = float(rope[p, i]), float(rope[p, half + i])
            u, w = x[t, :, a].astype(np.float64), x[t, :, b].astype(np.float64)
            y[t, :, a], y[t, :, b] = u * c - w * s, w * c + u * s
            mag[t, :, a], mag[t, :, b] = np.abs(u * c) + np.abs(w * s), np.abs(w * c) + np.abs(u * s)
    return y, mag


def store(cache, x, slots):
    """A copy of cache [pages, H, page, D] (fp64) with x [T, H, D] in its slots."""
    out = np.array(cache, dtype=np.float64)
    pages, _, page, _ = out.shape
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            out[int(s) // page, :, int(s) % page] = x[t]
    return out
