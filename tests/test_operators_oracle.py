"""The operators' 64-bit statements: gradients against differences, the plan's order (CPU)."""

import numpy as np
import pytest

from oracle import operators as O


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_gradient_is_the_difference_quotient(kind, renormalise):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 12))
    ids, _ = O.route(x, 4, kind, renormalise=renormalise)
    ids[1, 3] = -1
    ids[2, :] = -1
    dw = rng.standard_normal(ids.shape)
    got = O.route_grad(x, ids, dw, kind, renormalise, 2.5)
    h = 1e-5
    for t in range(5):
        for e in range(12):
            up, down = x[t].copy(), x[t].copy()
            up[e] += h
            down[e] -= h
            live = ids[t] >= 0
            d = (O.weights_of(up, ids[t], kind, renormalise, 2.5) - O.weights_of(down, ids[t], kind, renormalise, 2.5)) / (2 * h)
            # central differences: h^2 / 6 times a third derivative of order one, and 1e-16 / h of rounding
            assert abs(np.dot(d[live], dw[t][live]) - got[t, e]) < 1e-8


def test_combine_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(4)
    _, places = O.plan(np.array([[0, 2], [1, -1], [2, 0]]), 3)
    rows, w, dy = rng.standard_normal((6, 5)), rng.standard_normal((3, 2)), rng.standard_normal((3, 5))
    grad_rows, grad_w = O.combine_grad(rows, places, w, dy)
    h = 1e-6

    def loss(r, v):
        return float((O.combine(r, places, v) * dy).sum())
    for i in np.ndindex(rows.shape):
        d = np.zeros_like(rows)
        d[i] = h
        assert abs((loss(rows + d, w) - loss(rows - d, w)) / (2 * h) - grad_rows[i]) < 1e-8   # linear: rounding only
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((loss(rows, w + d) - loss(rows, w - d)) / (2 * h) - grad_w[i]) < 1e-8


def test_combine_without_weights_is_the_gradient_of_dispatch():
    rng = np.random.default_rng(5)
    _, places = O.plan(np.array([[0, 2], [1, -1], [2, 0]]), 3)
    x, drows = rng.standard_normal((3, 4)), rng.standard_normal((6, 4))
    dx = O.combine(drows, places)
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = 1.0
        assert np.isclose((O.dispatch(d, places) * drows).sum(), dx[i], rtol=1e-12, atol=1e-12)


def test_embed_gradient_is_the_transpose():
    rng = np.random.default_rng(6)
    tokens = np.array([3, 5, 3, 9, -1, 4])
    dy = rng.standard_normal((6, 2))
    got = O.embed_grad(dy, tokens, 3, first=3, scale=2.0)
    for r in range(3):
        for c in range(2):
            table = np.zeros((3, 2))
            table[r, c] = 1.0
            assert np.isclose((O.embed(table, tokens, 3, 2.0) * dy).sum(), got[r, c], rtol=1e-12)


def test_plan_packs_experts_in_order():
    offsets, places = O.plan(np.array([[2, 0], [2, 5], [0, -1]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert places.tolist() == [[2, 0], [3, ~4], [1, ~5]]


def test_route_by_hand():
    x = np.array([[0.0, 2.0, 1.0, -np.inf], [-np.inf] * 4, [1.0, 1.0, 1.0, 1.0]])
    ids, w = O.route(x, 3, renormalise=True)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [0, 1, 2]]
    e = np.exp([2.0, 1.0, 0.0])
    assert np.allclose(w[0], e / e.sum()) and np.allclose(w[1], 0) and np.allclose(w[2], 1 / 3)
    # two groups of two; the second has the best pair but not the best expert
    ids, _ = O.route(np.array([[3.0, -9.0, 2.0, 2.0]]), 1, "sigmoid", groups=2, kept_groups=1, group_best=2)
    assert ids.tolist() == [[2]]
    ids, _ = O.route(np.array([[3.0, -9.0, 2.0, 2.0]]), 1, "sigmoid", groups=2, kept_groups=1, group_best=1)
    assert ids.tolist() == [[0]]
