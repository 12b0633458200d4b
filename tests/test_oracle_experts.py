"""The fp64 definitions of the experts' and adapters' operators, pinned by hand and by other forms (CPU only)."""
import numpy as np
import pytest

import oracle.experts as OE


def test_route_by_hand():
    inf, nan = np.inf, np.nan
    x = [[0.0, 2.0, 2.0, 1.0], [nan, -inf, 3.0, -inf], [-inf, -inf, nan, -inf], [inf, 5.0, inf, 1.0]]
    e, w, off, rows, places = OE.route(x, 2)
    assert e.tolist() == [[1, 2], [2, -1], [-1, -1], [0, 2]]
    np.testing.assert_allclose(w, [[0.5, 0.5], [1, 0], [0, 0], [0.5, 0.5]])
    assert off.tolist() == [0, 1, 2, 5, 5]
    assert rows.tolist() == [6, 0, 1, 2, 7, 3, 4, 5]
    assert places.tolist() == [[1, 2], [3, -1], [-1, -1], [0, 4]]
    _, w, *_ = OE.route([[0.0, np.log(3.0)]], 1, renormalize=False)
    assert w[0, 0] == pytest.approx(0.75)


def test_route_is_a_stable_sort():
    rng = np.random.default_rng(3)
    e, w, off, rows, places = OE.route(rng.integers(0, 4, (50, 7)).astype(float), 3)
    flat = e.reshape(-1)
    assert (rows == np.argsort(flat, kind="stable")).all()
    assert (flat[rows] == np.repeat(np.arange(7), np.diff(off))).all()
    assert (rows[places.reshape(-1)] == np.arange(150)).all()
    np.testing.assert_allclose(w.sum(1), 1.0)


def test_product_combine_and_lora_against_matrices():
    rng = np.random.default_rng(4)
    T, E, N, K, k = 9, 4, 6, 8, 2
    A, W, bias = rng.normal(size=(T, K)), rng.normal(size=(E, N, K)), rng.normal(size=(E, N))
    e, w, off, rows, places = OE.route(rng.normal(size=(T, E)), k)
    C, mag = OE.product(A, W, off, rows, bias)
    whole = np.einsum("tk,enk->ten", A, W) + bias
    out = OE.combine(C, places, w, add=A[:, :N])
    want = A[:, :N] + sum(w[:, j, None] * whole[np.arange(T), e[:, j]] for j in range(k))
    np.testing.assert_allclose(out, want)
    assert (mag >= np.abs(C) - 1e-12).all()
    again, _ = OE.product(A[rows // k], W, off, None, bias)
    np.testing.assert_allclose(again, C)
    g = OE.gated(C)
    np.testing.assert_allclose(g, C[:, :3] * C[:, 3:] / (1 + np.exp(-C[:, :3])))
    LA, LB = rng.normal(size=(3, 5, K)), rng.normal(size=(3, N, 5))
    ids = np.array([0, -1, 2, 1, 3, 2, 0, 0, 1])
    got, h = OE.lora(A, A[:, :N], LA, LB, ids, [1.0, 0.5, -2.0])
    for t, l in enumerate(ids):
        want = A[t, :N] + ([1.0, 0.5, -2.0][l] * LB[l] @ LA[l] @ A[t] if 0 <= l < 3 else 0)
        np.testing.assert_allclose(got[t], want)
    assert not h[1].any()
