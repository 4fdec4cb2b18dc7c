"""Layer norm, balance and distillation in 64 bits: gradients against differences, ranges against the whole (CPU)."""

import numpy as np
import pytest

from oracle import operators as O

H = 1e-5


def difference(f, x):
    """Central differences of f at x: off by H^2 / 6 of a third derivative of order one, and 1e-16 / H of rounding."""
    out = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += H
        down[i] -= H
        out[i] = (f(up) - f(down)) / (2 * H)
    return out


def test_layer_norm_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    x, w, b, dy, dt = (rng.standard_normal(s) for s in ((3, 6), 6, 6, (3, 6), (3, 6)))
    dx, dw, db = O.layer_norm_grad(dy, x, O.layer_norm(x, w, b, 0.1)[1], w, dt)

    def loss(x=x, w=w, b=b):
        return (O.layer_norm(x, w, b, 0.1)[0] * dy).sum() + (x * dt).sum()
    assert np.allclose(difference(lambda v: loss(x=v), x), dx, rtol=0, atol=1e-8)
    assert np.allclose(difference(lambda v: loss(w=v), w), dw, rtol=0, atol=1e-8)
    assert np.allclose(difference(lambda v: loss(b=v), b), db, rtol=0, atol=1e-8)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_balance_gradient_is_the_difference_quotient(kind):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((6, 5))
    ids, _ = O.route(x, 2, kind)
    ids[1] = -1
    ids[2, 1] = 7
    _, sums, loss = O.balance(x, ids, kind, 2.5)
    got = O.balance_grad(x, ids, sums, 3.0, kind, 2.5)
    assert np.allclose(difference(lambda v: 3.0 * O.balance(v, ids, kind, 2.5)[2], x), got, rtol=0, atol=1e-8)
    assert (got[1] == 0).all() and sums[-1] == 5


def test_balance_of_experts_that_are_alike_is_the_scale():
    ids = np.stack([np.arange(8), np.roll(np.arange(8), 1)], 1)
    assert abs(O.balance(np.zeros((8, 8)), ids, scale=0.25)[2] - 0.25) < 1e-15


def distil_case(rng, T=4, V=11, K=4):
    z, t = 2 * rng.standard_normal((T, V)), 2 * rng.standard_normal((T, K))
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)])
    ids[1, 2] = -1
    ids[2, 1] = ids[2, 0]
    ids[3, :] = V
    return z, ids, t


def test_distillation_gradient_is_the_difference_quotient():
    z, ids, t = distil_case(np.random.default_rng(3))
    g = np.array([1.0, -2.0, 0.5, 3.0])

    def loss(v):
        return O.distil_join(O.distil_parts(v, ids, t, temperature=1.5)[None], 1.5, 2.0)
    got = O.distil_grad(z, ids, t, loss(z)[1], g, temperature=1.5, scale=2.0)
    assert np.allclose(difference(lambda v: (loss(v)[0] * g).sum(), z), got, rtol=0, atol=1e-8)
    assert (got[3] == 0).all() and loss(z)[0][3] == 0


def test_distillation_is_the_divergence():
    z, ids, t = distil_case(np.random.default_rng(4))
    loss = O.distil_join(O.distil_parts(z, ids, t, temperature=0.5)[None], 0.5)[0]
    log_p = z[0] / 0.5 - np.log(np.exp(z[0] / 0.5).sum())
    q = np.exp(t[0] / 0.5) / np.exp(t[0] / 0.5).sum()
    assert abs((q * (np.log(q) - log_p[ids[0]])).sum() - loss[0]) < 1e-12


@pytest.mark.parametrize("cuts", [(0, 11), (0, 4, 11), (0, 1, 1, 6, 11)])
def test_ranges_join_to_the_whole(cuts):
    z, ids, t = distil_case(np.random.default_rng(5))
    z[0, :4] = -np.inf
    ids[0] = [4, 6, 8, 10]
    want_loss, want = O.distil_join(O.distil_parts(z, ids, t)[None])
    parts = np.stack([O.distil_parts(z[:, a:b], ids, t, first=a, vocabulary=11) for a, b in zip(cuts, cuts[1:])])
    loss, stats = O.distil_join(parts)
    assert np.allclose(loss, want_loss, rtol=1e-12, atol=1e-12) and np.allclose(stats, want, rtol=1e-12)
    whole = O.distil_grad(z, ids, t, want, np.ones(4))
    for a, b in zip(cuts, cuts[1:]):
        assert np.allclose(O.distil_grad(z[:, a:b], ids, t, stats, np.ones(4), a, 11), whole[:, a:b], rtol=1e-12, atol=1e-15)
