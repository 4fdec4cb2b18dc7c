"""Layer norm, balance and distillation on the GPU, against their 64-bit statements.

Bounds as in test_gpu_operators: u is half a unit in the last place of the
output type relative to its value, e = 2^-24 one binary32 rounding.  A sum is
off by the number of additions that a term passes through times e, of the sum
of the terms' sizes; expf is within 2 ulp (4 e), ex2.approx within 2^-22 (4 e).
"""

import math

import numpy as np
import pytest
import torch

from oracle import operators as O
from collective_datapath_reduce_gb300 import purlin as P
from collective_datapath_reduce_gb300 import torch_api as purlin
from test_gpu_operators import DEV, DTYPES, E24, U, Guarded, close, floats, h, ints, make, refused, spread  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def status(h):  # noqa: F811
    return P.purlin_status_get(h.raw, torch.cuda.current_stream().cuda_stream)


# --------------------------------------------------------------- layer norm

def vector(values, dtype):
    t = floats(values).to(dtype)
    return t, t.double().cpu().numpy()


def chain(D):
    """Additions that an element of a row passes through: within a thread, lanes, warps."""
    return 16 + D // 512 + 5 + 16


def norm_bounds(t64, w64, b64, y, stats, eps, dtype):
    """Bounds of y and stats: the mean is off by dm, the distances by that and a rounding, the
    variance by twice their errors and its own sum's, the deviation's inverse by half of that."""
    n, D = chain(t64.shape[1]), t64.shape[1]
    mean, rstd = stats[:, :1], stats[:, 1:]
    dm = (n + 1) * E24 * np.abs(t64).mean(1, keepdims=True)
    off = np.abs(t64 - mean)
    dd = dm + E24 * off
    dvar = (2 * off * dd + dd * dd).mean(1, keepdims=True) + (n + 3) * E24 * (off ** 2).mean(1, keepdims=True)
    rel = 0.5 * dvar * rstd ** 2 * 1.01 + 3 * E24
    w = np.ones(D) if w64 is None else np.abs(w64)
    bound = w * rstd * (dd + off * (rel + 3 * E24)) + E24 * np.abs(y) + U[dtype] * np.abs(y) * 1.01
    return bound, np.hstack([dm, rel * rstd])


NORMS = [(1, 1, 0, 0), (3, 2, 0, 0), (1, 8, 0, 0), (7, 7, 1, 1), (5, 64, 0, 8), (9, 129, 3, 1), (130, 33, 0, 0), (33, 256, 0, 0),
         (17, 520, 8, 0), (6, 1537, 0, 0), (5, 2048, 0, 2), (4, 2056, 0, 0), (3, 4096, 0, 0), (2, 4104, 8, 8), (3, 8191, 0, 0),
         (2, 8192, 0, 0), (3, 8200, 0, 0), (2, 20001, 7, 3), (700, 160, 0, 0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wdtype", DTYPES)
@pytest.mark.parametrize("T,D,pad,off", NORMS)
def test_layer_norm(h, T, D, pad, off, wdtype, dtype):  # noqa: F811
    rng = np.random.default_rng(T * 100 + D)
    x, x64 = make(rng.standard_normal((T, D)) * 3 + 1.5, dtype, pad, off)
    r, r64 = make(rng.standard_normal((T, D)), dtype, pad, off)
    w, w64 = vector(1 + 0.3 * rng.standard_normal(D), wdtype)
    b, b64 = vector(rng.standard_normal(D), wdtype)
    for residual, weight, bias in ((None, w, b), (r, w, b), (r, None, None), (None, w, None), (r, None, b)):
        y, total, stats = Guarded(T, D, dtype, pad, off), Guarded(T, D, dtype, pad, off), Guarded(T, 2, F32)
        purlin.layer_norm(x, weight, bias, y.view, h, residual=residual, total=total.view, stats=stats.view, eps=1e-3)
        want_total = x64 + (0 if residual is None else r64)
        close(total.view, want_total, np.abs(want_total) * (U[dtype] + E24))
        t64 = total.view.double().cpu().numpy()
        args = (None if weight is None else w64, None if bias is None else b64)
        want, want_stats = O.layer_norm(t64, *args, 1e-3)
        bound, bound_stats = norm_bounds(t64, *args, want, want_stats, 1e-3, dtype)
        # a bias that cancels: the product is rounded with it, once
        close(y.view, want, bound)
        close(stats.view, want_stats, bound_stats)
        assert y.intact() and total.intact() and stats.intact()
        again = Guarded(T, D, dtype, pad, off)
        purlin.layer_norm(x, weight, bias, again.view, h, residual=residual, eps=1e-3)     # neither total nor stats
        assert torch.equal(again.view, y.view)


@pytest.mark.parametrize("D", [33, 96, 4096, 9000])
def test_layer_norm_in_place(h, D):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(1)
    x, r = (torch.randn(5, D, generator=g, device=DEV).to(BF16) for _ in range(2))
    w = torch.randn(D, generator=g, device=DEV)
    y, total = torch.empty_like(x), torch.empty_like(x)
    purlin.layer_norm(x, w, w, y, h, residual=r, total=total)
    for on_y, on_total in (("x", "r"), ("r", "x"), ("x", None), ("r", None), (None, "x"), (None, "r")):
        t = {"x": x.clone(), "r": r.clone()}
        y2, total2 = t.get(on_y, torch.empty_like(x)), t.get(on_total, torch.empty_like(x))
        purlin.layer_norm(t["x"], w, w, y2, h, residual=t["r"], total=total2)
        assert torch.equal(y2, y) and torch.equal(total2, total)
    purlin.layer_norm(x.clone(), w, None, y, h)
    x2 = x.clone()
    purlin.layer_norm(x2, w, None, x2, h)
    assert torch.equal(x2, y)


def test_layer_norm_of_rows_without_spread_and_not_finite(h):  # noqa: F811
    x = torch.full((5, 64), 3.0, device=DEV)
    x[1, 3], x[2, 5] = math.nan, math.inf
    x[3] = torch.finfo(F32).min
    b = torch.full((64,), 0.5, device=DEV)
    y, stats = torch.empty_like(x), torch.empty(5, 2, device=DEV)
    purlin.layer_norm(x, None, b, y, h, stats=stats, eps=0.25)
    assert (y[0] == 0.5).all() and (y[4] == 0.5).all() and stats[0].tolist() == [3.0, 2.0]
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()


GRADS = [(0, 8, 0, 0), (1, 1, 0, 0), (1, 4096, 0, 0), (3, 2, 0, 0), (7, 7, 1, 1), (9, 129, 3, 1), (130, 33, 0, 0), (40, 256, 0, 0),
         (17, 520, 8, 0), (700, 96, 0, 0), (6, 1537, 0, 0), (5, 2048, 0, 2), (200, 2056, 0, 0), (320, 4096, 0, 0), (3, 8191, 0, 0),
         (200, 8192, 0, 0), (3, 8200, 0, 0), (160, 9001, 7, 3), (5003, 64, 0, 0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wdtype", DTYPES)
@pytest.mark.parametrize("T,D,pad,off", GRADS)
def test_layer_norm_gradient(h, T, D, pad, off, wdtype, dtype):  # noqa: F811
    rng = np.random.default_rng(T * 100 + D)
    x, x64 = make(rng.standard_normal((T, D)) * 3 + 1.5, dtype, pad, off)
    dy, dy64 = make(rng.standard_normal((T, D)), dtype, pad, off)
    dt, dt64 = make(rng.standard_normal((T, D)), dtype, pad, off)
    w, w64 = vector(1 + 0.3 * rng.standard_normal(D), wdtype)
    stats, s64 = make(O.layer_norm(x64, eps=1e-3)[1], F32)
    for total, weight in ((None, w), (dt, w), (dt, None)):
        dx, dw, db = Guarded(T, D, dtype, pad, off), Guarded(1, D, wdtype), Guarded(1, D, wdtype)
        purlin.layer_norm_grad(dy, x, stats, weight, dx.view, dw.view[0], db.view[0], h, grad_total=total)
        want, want_w, want_b = O.layer_norm_grad(dy64, x64, s64, None if weight is None else w64,
                                                 None if total is None else dt64)
        n = chain(D)
        hat = np.abs((x64 - s64[:, :1]) * s64[:, 1:])
        g = np.abs(dy64 * (1 if weight is None else w64))
        if T:
            mean_g, mean_gh = g.mean(1, keepdims=True), (g * hat).mean(1, keepdims=True)
            bound = s64[:, 1:] * E24 * (4 * g + (n + 5) * mean_g + (n + 9) * hat * mean_gh) + E24 * np.abs(want)
            close(dx.view, want, (bound + np.abs(want) * U[dtype]) * 1.01)
        # rows of a CTA's group, groups, CTAs by warps and warps
        n = T // 152 + 16 + 152 // 8 + 8
        close(dw.view[0], want_w, np.abs(want_w) * U[wdtype] + (np.abs(dy64) * hat).sum(0) * (n + 4) * E24)
        close(db.view[0], want_b, np.abs(want_b) * U[wdtype] + np.abs(dy64).sum(0) * (n + 1) * E24)
        assert dx.intact() and dw.intact() and db.intact()
        for gw, gb in ((dw, None), (None, db), (None, None)):      # each alone, and the rows alone
            dx2, dw2, db2 = Guarded(T, D, dtype, pad, off), Guarded(1, D, wdtype), Guarded(1, D, wdtype)
            purlin.layer_norm_grad(dy, x, stats, weight, dx2.view, gw and dw2.view[0], gb and db2.view[0], h, grad_total=total)
            assert torch.equal(dx2.view, dx.view)
            assert gw is None or torch.equal(dw2.view, dw.view)
            assert gb is None or torch.equal(db2.view, db.view)


@pytest.mark.parametrize("D", [33, 96, 4096, 9000])
def test_layer_norm_gradient_in_place(h, D):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(2)
    x, dy, dt = (torch.randn(900, D, generator=g, device=DEV).to(BF16) for _ in range(3))
    w = torch.randn(D, generator=g, device=DEV)
    stats = torch.rand(900, 2, generator=g, device=DEV)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    purlin.layer_norm_grad(dy, x, stats, w, dx, dw, db, h, grad_total=dt)
    for on in range(3):
        t = [x.clone(), dy.clone(), dt.clone()]
        dw2, db2 = torch.empty_like(w), torch.empty_like(w)
        purlin.layer_norm_grad(t[1], t[0], stats, w, t[on], dw2, db2, h, grad_total=t[2])
        assert torch.equal(t[on], dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


# ------------------------------------------------------------------ balance

BALANCES = [(0, 4, 2), (1, 1, 1), (1, 8, 2), (5, 7, 7), (64, 60, 4), (65, 64, 6), (300, 33, 3), (900, 128, 8), (700, 160, 6),
            (200, 256, 8), (130, 384, 8), (70, 1000, 32), (66, 1024, 10), (5000, 16, 2)]


def balance_case(rng, T, E, k, dtype, pad=0):
    x, x64 = make(spread(rng, T, E) if T else np.zeros((0, E)), dtype, pad)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]) if T else np.zeros((0, k), dtype=np.int64)
    if T > 4:
        ids[1] = -1               # padding, whose logits may be anything
        x[1, 0] = math.nan
        x[3] = -math.inf
        ids[3] = E                # out of range: padding too
        ids[2, 0] = ids[2, -1]    # the same expert twice
        ids[4, k // 2:] = -1
        x64 = x.double().cpu().numpy()
    return x, x64, ids


def share_error(E):
    """Relative: a rounded difference of 6 at most, expf, the sum of E in lanes and warps, the division."""
    return (6 + 4 + E // 32 + 6 + 5 + 3) * E24


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", BALANCES)
def test_balance(h, T, E, k, kind, dtype):  # noqa: F811
    rng = np.random.default_rng(T + E)
    scores = purlin.Scores.SIGMOID if kind == "sigmoid" else purlin.Scores.SOFTMAX
    for pad in (0, 3):
        x, x64, ids = balance_case(rng, T, E, k, dtype, pad)
        counts, sums, loss = Guarded(1, E, torch.int32), Guarded(1, 2 * E + 1, F32), Guarded(1, 1, F32)
        purlin.balance_loss(x, ints(ids), counts.view[0], sums.view[0], loss.view[0], h, scores=scores, scale=0.5)
        with np.errstate(invalid="ignore"):
            want_c, want_s, want = O.balance(x64, ids, kind, 0.5)
        assert np.array_equal(counts.view[0].cpu().numpy(), want_c)
        assert np.array_equal(sums.view[0, :E].cpu().numpy(), want_c) and sums.view[0, 2 * E].item() == want_s[2 * E]
        n = T // 2432 + 1 + 8 + 8 + 38
        rel = share_error(E) + n * E24
        close(sums.view[0], want_s, want_s * rel)
        close(loss.view[0], want, want * (rel + (E // 256 + 5 + 8 + 8 + 8) * E24))
        joined = Guarded(1, 1, F32)
        purlin.balance_join(sums.view[0], joined.view[0], h, scale=0.5)
        close(joined.view[0], want, want * (rel + (E // 256 + 5 + 8 + 8 + 8) * E24))
        without = Guarded(1, 2 * E + 1, F32)
        purlin.balance_loss(x, ints(ids), counts.view[0], without.view[0], None, h, scores=scores)
        assert torch.equal(without.view, sums.view)
        assert counts.intact() and sums.intact() and loss.intact() and joined.intact()

        s64 = sums.view[0].double().cpu().numpy()
        base, base64 = make(rng.standard_normal((T, E)) * 1e-3, dtype, pad)
        g, g64 = make(np.array([[2.5]]), F32)
        for b, grad in ((None, None), (base, g[0])):
            out = Guarded(T, E, dtype, pad)
            purlin.balance_loss_grad(x, ints(ids), sums.view[0], grad, out.view, h, scores=scores, scale=0.5, base=b)
            f = 1.0 if grad is None else 2.5
            with np.errstate(invalid="ignore"):
                want_g = O.balance_grad(x64, ids, s64, f, kind, 0.5) + (0 if b is None else base64)
            size = np.zeros((T, E))
            for t in range(T):
                if any(0 <= e < E for e in ids[t]):
                    c = f * 0.5 * E * s64[:E] / (s64[:E].sum() * s64[2 * E])
                    p = O.shares_of(x64[t], kind)
                    size[t] = p * (c + (p * c).sum())
            # the coefficient, two shares, their products' sum, three products
            close(out.view, want_g, np.abs(want_g) * (U[dtype] + E24) + size * (2 * share_error(E) + (E // 256 + E // 32 + 40) * E24))
            assert out.intact()
        if T:
            out = base.clone() if pad == 0 else None
            if out is not None:
                purlin.balance_loss_grad(x, ints(ids), sums.view[0], g[0], out, h, scores=scores, scale=0.5, base=out)
                again = torch.empty_like(out)
                purlin.balance_loss_grad(x, ints(ids), sums.view[0], g[0], again, h, scores=scores, scale=0.5, base=base)
                assert torch.equal(out, again)


def test_balance_without_a_token_that_counts(h):  # noqa: F811
    x, ids = torch.full((70, 9), math.nan, device=DEV), ints(np.full((70, 2), -1))
    counts, sums, loss = torch.ones(9, dtype=torch.int32, device=DEV), torch.ones(19, device=DEV), torch.ones(1, device=DEV)
    grad = torch.ones(70, 9, device=DEV)
    purlin.balance_loss(x, ids, counts, sums, loss, h)
    purlin.balance_loss_grad(x, ids, sums, None, grad, h)
    assert (counts == 0).all() and (sums == 0).all() and loss.item() == 0 and (grad == 0).all()


def test_balance_of_ranks_is_that_of_all_their_tokens(h):  # noqa: F811
    rng = np.random.default_rng(6)
    x, x64, ids = balance_case(rng, 500, 24, 3, F32)
    want = O.balance(np.nan_to_num(x64), ids, scale=2.0)
    sums, outs = [torch.empty(49, device=DEV) for _ in range(2)], [torch.empty(49, device=DEV) for _ in range(2)]
    loss = torch.empty(1, device=DEV)
    for r in range(2):
        part = slice(0, 230) if r == 0 else slice(230, 500)
        purlin.balance_loss(x[part], ints(ids[part]), torch.empty(24, dtype=torch.int32, device=DEV), sums[r], None, h)
    purlin.all_reduce(sums, outs, h)
    purlin.balance_join(outs[1], loss, h, scale=2.0)
    close(loss, want[2], want[2] * (share_error(24) + 80 * E24))


# -------------------------------------------------------------- distillation

def distil_case(rng, T, R, K, dtype, first, vocabulary, tdtype, wide, pad, off):
    z, z64 = make(rng.standard_normal((T, R)) * 3, dtype, pad, off)
    t = floats(rng.standard_normal((T, K)) * 2).to(tdtype)
    ids = np.stack([(rng.integers(vocabulary) + rng.permutation(max(K, 2 * K if vocabulary >= 2 * K else K))[:K]) % vocabulary
                    for _ in range(T)])
    if R:
        ids[0, 0] = first
        ids[-1, -1] = first + R - 1
    if T > 3:
        ids[1] = -1                       # no teacher
        ids[2, K // 2:] = vocabulary + 5  # fewer picks
        ids[3, 0] = ids[3, K - 1]         # a word twice
        t[2, 0] = -math.inf
    return z, z64, t, t.double().cpu().numpy(), torch.from_numpy(ids).to(DEV, torch.int64 if wide else torch.int32), ids


def distil_bounds(z64, ids, t64, parts, first, vocabulary, tau, split=1):
    """Bounds of the parts: the sum's terms, of exponents up to `far`, rounded three times, ex2, the
    additions of a thread, its rescaled sums, lanes, warps and CTAs; q alike, with its K additions."""
    T, R = z64.shape
    K = ids.shape[1]
    bound = np.zeros((T, 4))
    for t in range(T):
        m = parts[t, 0] if parts[t, 0] > -np.inf else 0.0
        # terms far below the largest do not count: their share is beneath their error's
        far = min(88.0, np.max(np.where(z64[t] > -np.inf, m - z64[t], 0.0), initial=0.0) / tau)
        bound[t, 1] = parts[t, 1] * ((R // 256 + 20) + 4 + 3 * far + 16 * 5) * E24 + R * 2.0 ** -126
        q = O.teacher_of(ids[t], t64[t], vocabulary, tau)
        seen = np.where(np.isfinite(t64[t]) & (q > 0), t64[t], np.nan)
        reach = 0.0 if np.isnan(seen).all() else (np.nanmax(seen) - np.nanmin(seen)) / tau
        rel = (2 * reach + 4 + K // 256 + 5 + 8 + 4) * E24
        here = [(q[k], z64[t, i - first]) for k, i in enumerate(ids[t]) if first <= i < first + R and q[k] > 0]
        size = sum(a * (abs(math.log(a)) + abs(v - m) / tau + 1) for a, v in here)
        bound[t, 2] = size * (2 * rel + 8 * E24)
        bound[t, 3] = 2 * rel * parts[t, 3]
    return bound


DISTILS = [
    # tokens, words, picks, first, vocabulary, dtype, teacher's, 64-bit ids, temperature, pad, offset
    (1, 1, 1, 0, 1, F32, F32, True, 1.0, 0, 0),
    (1, 3, 2, 0, 3, BF16, F32, True, 2.0, 0, 0),
    (2, 17, 4, 5, 40, F32, BF16, False, 0.5, 0, 1),
    (5, 64, 5, 0, 64, BF16, BF16, False, 1.0, 0, 0),
    (9, 129, 16, 129, 258, BF16, F32, True, 2.0, 3, 1),
    (33, 1000, 7, 0, 1000, F32, F32, False, 1.0, 0, 0),
    (3, 2047, 300, 0, 2047, F32, F32, True, 0.75, 5, 3),
    (2, 8192, 64, 8192, 32768, BF16, F32, True, 1.0, 0, 0),
    (7, 20000, 1024, 0, 20000, BF16, BF16, True, 1.0, 0, 0),
    (4, 32003, 32, 0, 32003, BF16, F32, True, 1.0, 0, 0),
    (40, 30001, 33, 7, 40000, F32, F32, False, 3.0, 0, 0),
    (700, 513, 8, 0, 513, BF16, F32, True, 1.0, 0, 0),
    (3, 0, 4, 10, 20, F32, F32, True, 1.0, 0, 0),
]


@pytest.mark.parametrize("case", DISTILS, ids=str)
def test_distil(h, case):  # noqa: F811
    T, R, K, first, V, dtype, tdtype, wide, tau, pad, off = case
    rng = np.random.default_rng(R + K)
    z, z64, t, t64, ids, ids64 = distil_case(rng, T, R, K, dtype, first, V, tdtype, wide, pad, off)
    parts = Guarded(T, 4, F32)
    purlin.distil_parts(z, ids, t, parts.view, h, first=first, vocabulary=V, temperature=tau)
    want = O.distil_parts(z64, ids64, t64, first, V, tau)
    bound = distil_bounds(z64, ids64, t64, want, first, V, tau)
    assert np.array_equal(parts.view[:, 0].cpu().numpy(), want[:, 0])
    close(parts.view[:, 1:], want[:, 1:], bound[:, 1:])
    assert parts.intact()
    if first == 0 and V == R:
        loss, stats = Guarded(1, T, F32), Guarded(T, 2, F32)
        purlin.distil_loss(z, ids, t, loss.view[0], stats.view, h, temperature=tau, scale=1.5)
        assert torch.equal(stats.view, parts.view[:, :2]) and loss.intact() and stats.intact()
        want_loss, _ = O.distil_join(want[None], tau, 1.5)
        log_s = np.log(want[:, 1])
        of_loss = 1.5 * (bound[:, 2] + bound[:, 3] * np.abs(log_s) + want[:, 3] * (bound[:, 1] / want[:, 1] + 4 * E24 * np.abs(log_s))
                         + 3 * E24 * (np.abs(want[:, 2]) + np.abs(log_s)))
        close(loss.view[0], want_loss, of_loss)
        joined, js = torch.empty(T, device=DEV), torch.empty(T, 2, device=DEV)
        purlin.distil_join(parts.view, joined, js, h, temperature=tau, scale=1.5)
        assert torch.equal(joined, loss.view[0]) and torch.equal(js, stats.view)
    if R == 0:
        return

    # the gradient, given statistics of a vocabulary of which this is a part
    s64 = want[:, :2] * np.array([1.0, 2.5 if V > R else 1.0])
    stats, s64 = make(s64, F32)
    g, g64 = make(rng.standard_normal((1, T)), F32)
    out = Guarded(T, R, dtype, pad, off)
    purlin.distil_loss_grad(z, ids, t, stats, g[0], out.view, h, first=first, vocabulary=V, temperature=tau, scale=1.5)
    want_g = O.distil_grad(z64, ids64, t64, s64, g64[0], first, V, tau, 1.5)
    p = np.exp((z64 - s64[:, :1]) / tau) / s64[:, 1:]
    far = (s64[:, :1] - z64) / tau
    q = np.zeros((T, R))
    for i in range(T):
        qt = O.teacher_of(ids64[i], t64[i], V, tau)
        for k, w in enumerate(ids64[i]):
            if first <= w < first + R:
                q[i, w - first] += qt[k]
    G = np.abs(g64[0])[:, None] * 1.5 / tau
    reach = 2 * 6 * 2 / tau
    of_g = G * (p * (3 * np.abs(far) + 4 + 6) + q * (2 * reach + 4 + K // 256 + 40)) * E24 + G * 2.0 ** -126
    close(out.view, want_g, np.abs(want_g) * U[dtype] * 1.01 + of_g)
    assert out.intact()
    if R > 4:      # another alignment of the gradient's rows
        out2 = Guarded(T, R, dtype, pad + 1, off + 1)
        purlin.distil_loss_grad(z, ids, t, stats, g[0], out2.view, h, first=first, vocabulary=V, temperature=tau, scale=1.5)
        assert torch.equal(out2.view, out.view) and out2.intact()
    purlin.distil_loss_grad(z, ids, t, stats, g[0], z, h, first=first, vocabulary=V, temperature=tau, scale=1.5)   # in place
    assert torch.equal(z, out.view)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R", [40, 5000])
def test_distil_of_masked_and_lowest_values(h, R, dtype):  # noqa: F811
    low = torch.finfo(dtype).min
    z = torch.zeros(8, R, device=DEV, dtype=dtype)
    z[0] = -math.inf                        # nothing left
    z[1] = low                              # values like others: all alike
    z[2, 1:] = -math.inf                    # one word
    z[3, 3] = -math.inf                     # at a pick
    z[4, 7] = math.nan
    z[5, 7] = math.inf
    z[6, 1:] = low                          # differences past the type's range
    z[6, 0] = torch.finfo(dtype).max
    z[7] = math.nan                         # padding
    ids = ints([[0, 1]] * 3 + [[3, 4]] + [[0, 1]] * 3 + [[-1, R]])
    ids[2] = ints([0, 0])
    ids[6] = ints([0, -1])
    t = torch.zeros(8, 2, device=DEV)
    loss, stats, g = torch.empty(8, device=DEV), torch.empty(8, 2, device=DEV), torch.ones(8, device=DEV)
    grad = torch.empty_like(z)
    purlin.distil_loss(z, ids, t, loss, stats, h, temperature=0.5)
    purlin.distil_loss_grad(z, ids, t, stats, g, grad, h, temperature=0.5)
    got, grad = loss.tolist(), grad.float()
    assert got[0] == 0 and (grad[0] == 0).all()
    want = math.log(R) - math.log(2)
    assert abs(got[1] - want) < 16 * E24 * math.log(R) and stats[1].tolist() == [low, R]
    u = U[dtype]
    # 1 / R and q are exact or rounded once; four roundings of the difference, then the type's
    assert (grad[1, 2:] - 2 / R).abs().max().item() <= 2 / R * (4 * E24 + u) and abs(grad[1, 0].item() + 1 - 2 / R) <= 4 * E24 + u
    # a word twice: the sum of q log q over two picks of one half each
    assert abs(got[2] - math.log(0.5)) < 4 * E24 and (grad[2] == 0).all()
    assert got[3] == math.inf and torch.isfinite(grad[3]).all() and abs(grad[3, 3].item() + 1) <= u
    assert math.isnan(got[4]) and torch.isnan(grad[4]).all() and math.isnan(got[5]) and torch.isnan(grad[5]).all()
    assert got[6] == 0 and (grad[6] == 0).all() and stats[6, 1].item() == 1
    assert got[7] == 0 and (grad[7] == 0).all()
    t[:, 0] = math.nan
    purlin.distil_loss(z, ids, t, loss, stats, h)
    purlin.distil_loss_grad(z, ids, t, stats, g, grad := torch.empty_like(z), h)
    assert math.isnan(loss[1].item()) and torch.isnan(grad[1]).all() and loss[7].item() == 0
    t[:] = -math.inf
    purlin.distil_loss(z, ids, t, loss, stats, h)
    purlin.distil_loss_grad(z, ids, t, stats, g, grad, h)
    assert (loss == 0).all() and (grad == 0).all()


@pytest.mark.parametrize("cuts", [(0, 999), (0, 250, 500, 750, 999), (0, 1, 1, 600, 998, 999)])
def test_distil_by_ranges(h, cuts):  # noqa: F811
    """Parts of ranges, gathered and joined: the whole vocabulary's loss, and its gradient by columns."""
    rng = np.random.default_rng(7)
    T, V, K, tau = 11, 999, 9, 1.5
    z, z64, t, t64, ids, ids64 = distil_case(rng, T, V, K, BF16, 0, V, F32, True, 0, 0)
    z[5, :300] = -math.inf
    whole, stats = torch.empty(T, device=DEV), torch.empty(T, 2, device=DEV)
    purlin.distil_loss(z, ids, t, whole, stats, h, temperature=tau, scale=2.0)
    n = len(cuts) - 1
    parts = torch.empty(n, T, 4, device=DEV)
    ranges = [z[:, a:b].contiguous() for a, b in zip(cuts, cuts[1:])]
    for r, (a, b) in enumerate(zip(cuts, cuts[1:])):
        purlin.distil_parts(ranges[r], ids, t, parts[r], h, first=a, vocabulary=V, temperature=tau)
    loss, joined = torch.empty(T, device=DEV), torch.empty(T, 2, device=DEV)
    purlin.distil_join(parts, loss, joined, h, temperature=tau, scale=2.0)
    assert torch.equal(joined[:, 0], stats[:, 0])
    # both are off by a few roundings of sums of at most 20 terms each in a thread, of values below 20
    close(joined[:, 1], stats[:, 1].double().cpu().numpy(), 200 * E24 * stats[:, 1].double().cpu().numpy())
    close(loss, whole.double().cpu().numpy(), 2.0 * 20 * 200 * E24)
    g = torch.ones(T, device=DEV)
    grad = torch.empty_like(z)
    purlin.distil_loss_grad(z, ids, t, joined, g, grad, h, temperature=tau, scale=2.0)
    for r, (a, b) in enumerate(zip(cuts, cuts[1:])):
        out = torch.empty_like(ranges[r])
        purlin.distil_loss_grad(ranges[r], ids, t, joined, g, out, h, first=a, vocabulary=V, temperature=tau, scale=2.0)
        assert torch.equal(out, grad[:, a:b])


# ------------------------------------------------- streams, graphs, refusals

def everything(h, stream=None):  # noqa: F811
    """One call of each operator on small fixed inputs; returns the outputs."""
    g = torch.Generator(device=DEV).manual_seed(9)
    T, E, k, D, V, K = 700, 40, 4, 136, 1001, 12
    x, r, dy = (torch.randn(T, D, generator=g, device=DEV).to(BF16) for _ in range(3))
    w, b = torch.randn(D, generator=g, device=DEV), torch.randn(D, generator=g, device=DEV)
    logits, z = torch.randn(T, E, generator=g, device=DEV), torch.randn(T, V, generator=g, device=DEV)
    ids, words = (torch.rand(T, n, generator=g, device=DEV).topk(m, 1).indices.to(torch.int32) for n, m in ((E, k), (V, K)))
    t, dl = torch.randn(T, K, generator=g, device=DEV), torch.randn(T, generator=g, device=DEV)
    f = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    o = dict(y=torch.empty_like(x), total=torch.empty_like(x), stats=f(T, 2), dx=torch.empty_like(x), dw=f(D), db=f(D),
             counts=torch.empty(E, dtype=torch.int32, device=DEV), sums=f(2 * E + 1), loss=f(1), joined=f(1), dlogits=f(T, E),
             kl=f(T), ks=f(T, 2), parts=f(T, 4), kl2=f(T), ks2=f(T, 2), dz=f(T, V))

    def call():
        purlin.layer_norm(x, w, b, o["y"], h, residual=r, total=o["total"], stats=o["stats"], stream=stream)
        purlin.layer_norm_grad(dy, o["total"], o["stats"], w, o["dx"], o["dw"], o["db"], h, grad_total=r, stream=stream)
        purlin.balance_loss(logits, ids, o["counts"], o["sums"], o["loss"], h, stream=stream)
        purlin.balance_join(o["sums"], o["joined"], h, stream=stream)
        purlin.balance_loss_grad(logits, ids, o["sums"], o["joined"], o["dlogits"], h, stream=stream)
        purlin.distil_loss(z, words, t, o["kl"], o["ks"], h, stream=stream)
        purlin.distil_parts(z, words, t, o["parts"], h, stream=stream)
        purlin.distil_join(o["parts"], o["kl2"], o["ks2"], h, stream=stream)
        purlin.distil_loss_grad(z, words, t, o["ks2"], dl, o["dz"], h, stream=stream)
    return call, o


def test_other_streams_and_graphs_give_the_same(h):  # noqa: F811
    call, want = everything(h)
    call()
    torch.cuda.synchronize()
    assert status(h) == (P.PL_OK, P.PL_OK)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        call, got = everything(h, stream)
        side.wait_stream(torch.cuda.current_stream())
        call()
        side.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), name
    with torch.cuda.stream(side):
        call, got = everything(h)
        call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
        for t in got.values():
            t.zero_()
        graph.replay()
        graph.replay()
        side.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name


def test_two_streams_of_one_handle_need_no_order(h):  # noqa: F811
    call, want = everything(h)
    call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = [everything(h, s) for s in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for call, _ in jobs:
            call()
    torch.cuda.synchronize()
    for _, got in jobs:
        for name in want:
            assert torch.equal(got[name], want[name]), name


def test_refusals_on_the_gpu(h):  # noqa: F811
    f = lambda *s, dtype=F32: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    x, w = f(8, 16), f(16)
    refused(purlin.layer_norm, x, w, w, f(8, 16), h, eps=-1.0)
    refused(purlin.layer_norm, x, w, w, f(8, 16), h, eps=math.nan)
    refused(purlin.layer_norm, x[:4], w, w, x[2:6], h)                                  # part of itself
    refused(purlin.layer_norm, x, w, w, x, h, total=x)                                  # both on it
    refused(purlin.layer_norm, x, x[0], None, x, h)                                     # its weight is written
    refused(purlin.layer_norm, x, w, w, f(8, 16), h, stats=x.view(-1)[:16].view(8, 2))
    big = f(8, 32)
    refused(purlin.layer_norm, big[:, :16], w, w, big[:, 16:], h)                       # columns of one matrix
    refused(purlin.layer_norm_grad, x, f(8, 16), f(8, 2), w, f(8, 16), w, f(16), h)     # grad_weight on weight
    refused(purlin.layer_norm_grad, x, x, f(8, 2), w, f(8, 16), f(16), x[0], h)
    refused(purlin.layer_norm_grad, x[:4], f(4, 16), f(4, 2), w, x[1:5], f(16), f(16), h)
    refused(purlin.balance_loss, f(4, 1025), i(4, 2), i(1025), f(2051), f(1), h)
    refused(purlin.balance_loss, f(4, 64), i(4, 33), i(64), f(129), f(1), h)
    refused(purlin.balance_loss, f(4, 2), i(4, 3), i(2), f(5), f(1), h)
    refused(purlin.balance_loss, f(4, 8), i(4, 2), i(8), f(17), f(1), h, scale=math.inf)
    refused(purlin.balance_loss, f(4, 8), i(4, 2), i(8), f(17), f(1), h, scores=2)
    sums = f(17)
    refused(purlin.balance_loss, f(4, 8), i(4, 2), i(8), sums, sums[:1], h)
    refused(purlin.balance_join, sums, sums[3:4], h)
    refused(purlin.balance_loss_grad, x[:4], i(4, 2), f(33), None, x[2:6], h)
    refused(purlin.balance_loss_grad, x, i(8, 2), f(33), None, x, h)                    # in place of the logits
    flat = f(200)
    refused(purlin.balance_loss_grad, f(4, 16), i(4, 2), f(33), None, flat[:64].view(4, 16), h, base=flat[16:80].view(4, 16))
    refused(purlin.distil_loss, f(4, 16), i(4, 1025), f(4, 1025), f(4), f(4, 2), h)
    for tau in (0.0, -1.0, math.nan, math.inf, 1e-31):
        refused(purlin.distil_loss, f(4, 16), i(4, 2), f(4, 2), f(4), f(4, 2), h, temperature=tau)
    refused(purlin.distil_loss, f(4, 16), i(4, 2), f(4, 2), f(4), f(4, 2), h, scale=math.nan)
    refused(purlin.distil_parts, f(4, 16), i(4, 2), f(4, 2), f(4, 4), h, first=5, vocabulary=20)
    refused(purlin.distil_parts, f(4, 16), i(4, 2), f(4, 2), f(4, 4), h, first=-1)
    refused(purlin.distil_parts, f(4, 16), i(4, 2), f(4, 2), f(17)[1:].view(4, 4), h)   # not at 8 bytes
    refused(purlin.distil_loss_grad, x[:4], i(4, 2), f(4, 2), f(4, 2), f(4), x[1:5], h)
    refused(purlin.distil_loss_grad, f(4, 16), i(4, 2), f(4, 2), flat[:8].view(4, 2), f(4), flat[:64].view(4, 16), h)
    s = torch.cuda.current_stream().cuda_stream
    assert P.purlin_layer_norm_grad(h.raw, x, 16, f(8, 16), 16, f(8, 2), 8, 16, P.PL_F32, w, P.PL_F32, None, 0, f(8, 16), 16,
                                    f(16), f(16), None, 0, s) == P.PL_ERR_WORKSPACE
    assert P.purlin_balance_loss(h.raw, f(900, 8), 8, P.PL_F32, i(900, 2), 900, 2, 8, 0, 1.0, i(8), f(17), f(1), None, 0,
                                 s) == P.PL_ERR_WORKSPACE
    assert P.purlin_layer_norm(h.raw, x.data_ptr() + 2, 16, None, 0, 4, 16, P.PL_F32, w, w, P.PL_F32, 1e-5, f(4, 16), 16, None, 0,
                               None, s) == P.PL_ERR_ALIGNMENT
    assert P.purlin_layer_norm(h.raw, x, 15, None, 0, 4, 16, P.PL_F32, w, w, P.PL_F32, 1e-5, f(4, 16), 16, None, 0, None,
                               s) == P.PL_ERR_INVALID_ARG
    assert P.purlin_layer_norm(h.raw, x, 16, None, 0, 4, 16, P.PL_U8, w, w, P.PL_F32, 1e-5, f(4, 16), 16, None, 0, None,
                               s) == P.PL_ERR_UNSUPPORTED
    d = P.make_distillation(16, 0, 17, 2, 4, P.PL_F32)
    assert P.purlin_distil_loss(h.raw, x, 16, P.PL_F32, 8, d, i(8, 2), f(8, 2), f(8), f(8, 2), s) == P.PL_ERR_INVALID_ARG
    assert status(h) == (P.PL_OK, P.PL_OK)


def test_no_tokens(h):  # noqa: F811
    f = lambda *s: torch.full(s, 5.0, device=DEV)  # noqa: E731
    i = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    purlin.layer_norm(f(0, 8), None, None, f(0, 8), h)
    dw, counts, sums, loss = f(8), torch.ones(8, dtype=torch.int32, device=DEV), f(17), f(1)
    purlin.layer_norm_grad(f(0, 8), f(0, 8), f(0, 2), None, f(0, 8), dw, None, h)
    purlin.balance_loss(f(0, 8), i, counts, sums, loss, h)
    purlin.balance_loss_grad(f(0, 8), i, sums, None, f(0, 8), h)
    purlin.distil_loss(f(0, 8), i, f(0, 2), f(0), f(0, 2), h)
    purlin.distil_join(f(2, 0, 4), f(0), f(0, 2), h)
    purlin.distil_loss_grad(f(0, 8), i, f(0, 2), f(0, 2), f(0), f(0, 8), h)
    assert (dw == 0).all() and (counts == 0).all() and (sums == 0).all() and loss.item() == 0
