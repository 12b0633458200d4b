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


# ---------------------------------------------------------------- attention

def test_attention_equal_scores_average_the_visible_values():
    """Zero queries weigh all visible keys alike, whatever the keys hold."""
    import oracle.attention as OA
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 4, 1, 16, 8))
    table = np.array([[2, 0, 3]])
    flat = v[[2, 0, 3], 0].reshape(48, 8)
    q = np.zeros((3, 2, 8))
    for window, sinks in ((0, 0), (5, 0), (5, 2), (1, 0), (100, 3)):
        r = OA.attend(q, k, v, table, [0, 3], [40], 0.3, window, sinks)
        for i in range(3):
            p = 37 + i
            see = [j for j in range(40) if j <= p and (not window or p - j < window or j < sinks)]
            assert np.allclose(r["out"][i, 1], flat[see].mean(0), atol=1e-14)
            assert np.isclose(r["lse"][i, 0], np.log(len(see)), atol=1e-14)


def test_attention_is_a_softmax():
    """Against a dense softmax over a contiguous cache, and the gradient of lse in the scale is the mean score."""
    import oracle.attention as OA
    rng = np.random.default_rng(4)
    k, v = rng.standard_normal((2, 2, 1, 16, 8))
    q = rng.standard_normal((1, 1, 8))
    f = lambda s: OA.attend(q, k, v, np.array([[0, 1]]), [0, 1], [23], s)  # noqa: E731
    s = 0.4 * k[:, 0].reshape(32, 8)[:23] @ q[0, 0]
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(f(0.4)["out"][0, 0], w @ v[:, 0].reshape(32, 8)[:23], atol=1e-13)
    d = (f(0.4 + 1e-6)["lse"] - f(0.4 - 1e-6)["lse"]) / 2e-6
    assert np.isclose(d[0, 0], (w * s).sum() / 0.4, atol=1e-6)


def test_attention_empty_and_missing():
    """No key, rows before the first key, pages that do not exist: zeros and -inf; hidden NaN stays hidden."""
    import oracle.attention as OA
    k, v = np.ones((2, 2, 1, 16, 4))
    v = v * np.arange(1.0, 17)[:, None]
    v[1, 0, 3:] = np.nan
    q = np.ones((4, 1, 4))
    r = OA.attend(q, k, v, np.array([[-1, 1]]), [0, 4], [19], 1.0)
    assert np.array_equal(r["out"][:3], np.where(np.arange(3)[:, None, None] < 1, 0, [[[1.0]], [[1.0]], [[1.5]]]) *
                          np.ones((3, 1, 4)))
    assert np.isneginf(r["lse"][0, 0]) and np.allclose(r["out"][3], 2.0)
    r = OA.attend(q, k, v, np.array([[0]]), [0, 4], [2], 1.0)
    assert np.array_equal(np.isneginf(r["lse"][:, 0]), [True, True, False, False])


# ----------------------------------------------------------------- sampling

def test_sampling_by_hand():
    """Five tokens with weights 8, 4, 2, 1, 1 (ties at the end)."""
    import oracle.sampling as OS
    row = np.log([2.0, 8.0, 1.0, 4.0, 1.0])
    full = lambda **kw: OS.kept(row, **kw)[0].tolist()  # noqa: E731
    assert full() == [1, 3, 0, 2, 4]
    assert full(top_k=4) == [1, 3, 0, 2] and full(top_k=9) == full()
    assert full(min_p=0.2) == [1, 3, 0] and full(min_p=2.0) == [1]
    assert full(top_p=0.51) == [1, 3] and full(top_p=0.8) == [1, 3, 0] and full(top_p=0.0) == [1]
    assert full(temperature=0.0) == [1] and full(temperature=2.0, min_p=0.4) == [1, 3, 0]
    assert full(top_k=2, top_p=0.7) == [1, 3] and full(top_k=2, top_p=0.6) == [1]  # of 12, not of 16
    # index order: 2/16, 10/16, 11/16, 15/16, 16/16
    got = [OS.sample(row, u)[0] for u in (0.0, 0.12, 0.13, 0.62, 0.63, 0.68, 0.69, 0.93, 0.94, 0.999, 1.5)]
    assert got == [0, 0, 1, 1, 2, 2, 3, 3, 4, 4, 4]
    tok, lp = OS.sample(row, 0.5, top_k=2)
    assert tok == 1 and abs(lp - np.log(8 / 12)) < 1e-14
    assert OS.sample(np.full(3, -np.inf), 0.5) == (-1, -np.inf)
    assert OS.sample(np.array([np.nan, 1.0, -np.inf]), 0.9) == (1, 0.0)
    assert OS.sample(np.array([np.inf, 1.0, np.inf]), 0.6)[0] == 2


def test_sampling_frequencies_are_the_probabilities():
    import oracle.sampling as OS
    rng = np.random.default_rng(6)
    row = rng.standard_normal(7)
    n = 4000
    count = np.bincount([OS.sample(row, (i + 0.5) / n, temperature=0.7)[0] for i in range(n)], minlength=7)
    p = np.exp(row / 0.7) / np.exp(row / 0.7).sum()
    assert np.abs(count / n - p).max() <= 1.0 / n
