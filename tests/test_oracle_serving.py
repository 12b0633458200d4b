"""Pins of the serving oracles against something other than themselves."""
import cmath

import numpy as np

import oracle.paged as OP


def test_plan_by_hand():
    """Three requests, pages of 4: one grows inside its page, one takes two pages, one rests."""
    table = [[7, -1, -1], [3, -1, -1], [5, 6, -1]]
    r = OP.plan([2, 4, 8], [1, 5, 0], table, [20, 21, 22, 23], 1, 8, 4)
    assert r["cu_q"] == [0, 1, 6, 6] and r["kv_lens"] == [3, 9, 8]
    assert r["positions"] == [2, 4, 5, 6, 7, 8, 0, 0]
    assert r["slots"] == [30, 84, 85, 86, 87, 88, -1, -1]
    assert r["table"].tolist() == [[7, -1, -1], [3, 21, 22], [5, 6, -1]] and r["state"] == [3, 0]


def test_plan_invariants():
    """Every token with a slot has one of its own, and no two requests share a page."""
    rng = np.random.default_rng(1)
    for page in (16, 64):
        ctx, new = rng.integers(0, 200, 20), rng.integers(0, 90, 20)
        held = -(-ctx // page)
        ids = rng.permutation(1000)
        table = np.full((20, 40), -1)
        at = 0
        for b in range(20):
            table[b, :held[b]] = ids[at:at + held[b]]
            at += held[b]
        r = OP.plan(ctx, new, table, ids[at:], 0, int(new.sum()), page)
        assert len(set(r["slots"])) == len(r["slots"]) and min(r["slots"]) >= 0 and r["state"][1] == 0
        used = r["table"][r["table"] >= 0]
        assert len(set(used.tolist())) == used.size == int((-(-(ctx + new) // page)).sum())


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(2)
    T, H, D, rot = 3, 2, 10, 6
    x = rng.standard_normal((T, H, D))
    ang = rng.uniform(-3, 3, (5, rot // 2))
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    pos = [4, 0, 2]
    for inter in (False, True):
        y, _ = OP.rotate(x, rope, pos, inter)
        for t in range(T):
            for i in range(rot // 2):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
                z = (x[t, 1, a] + 1j * x[t, 1, b]) * cmath.exp(1j * ang[pos[t], i])
                assert abs(y[t, 1, a] - z.real) < 1e-14 and abs(y[t, 1, b] - z.imag) < 1e-14
        assert np.array_equal(y[:, :, rot:], x[:, :, rot:])


def test_store_places_rows():
    cache = np.zeros((3, 2, 16, 4))
    x = np.arange(1, 17).reshape(2, 2, 4).astype(float)
    out = OP.store(cache, x, [2 * 16 + 5, -1])
    assert np.array_equal(out[2, :, 5], x[0]) and np.count_nonzero(out) == 8
