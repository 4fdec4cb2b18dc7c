"""The operators around the collectives on the GPU, against their 64-bit statements.

Bounds, all derived from the formats: u is half a unit in the last place of the
output type relative to its value (2^-24 binary32, 2^-8 bf16), e = 2^-24 one
binary32 rounding.  A sum of n terms in binary32 is off by at most n e times
the sum of the terms' sizes, in any order.  CUDA's expf is within 2 ulp, a
division or addition within half an ulp.
"""

import math

import numpy as np
import pytest
import torch

from oracle import operators as O
from collective_datapath_reduce_gb300 import purlin as P
from collective_datapath_reduce_gb300 import torch_api as purlin

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.bfloat16]
DEV = "cuda:0"
GUARD = 64


@pytest.fixture(scope="module")
def h():
    handle = purlin.initialize(2, DEV)
    yield handle
    purlin.finalize(handle)


class Guarded:
    """A rows x width matrix inside a larger buffer of a fixed pattern: `pad`
    elements between rows, `off` elements past an aligned address."""

    def __init__(self, rows, width, dtype, pad=0, off=0):
        self.rows, self.width, self.ld, self.off = rows, width, width + pad, off
        self.raw = torch.full((GUARD + off + rows * self.ld + GUARD,), -77.0 if dtype.is_floating_point else -77,
                              dtype=dtype, device=DEV)
        self.view = self.raw[GUARD + off:].as_strided((rows, width), (self.ld, 1))

    def intact(self):
        copy = self.raw.clone()
        copy[GUARD + self.off:].as_strided((self.rows, self.width), (self.ld, 1)).fill_(-77)
        return bool((copy == -77).all())


def make(values, dtype, pad=0, off=0):
    """A device matrix of the values rounded to dtype, and those values in 64 bits."""
    g = Guarded(values.shape[0], values.shape[1], dtype, pad, off)
    g.view.copy_(torch.from_numpy(np.ascontiguousarray(values, dtype=np.float32)))
    return g.view, g.view.double().cpu().numpy()


def close(got, want, bound):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3])


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def floats(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV)


# ------------------------------------------------------------------ routing

def spread(rng, T, E, low=-3.0, high=3.0):
    """Logits whose scores are far apart against binary32 rounding: a permuted grid per token."""
    grid = np.linspace(low, high, E)
    return np.stack([rng.permutation(grid) for _ in range(T)])


def run_route(h, x, k, dtype, pad=0, off=0, stream=None, **kw):
    bias = kw.pop("bias", None)
    xs, x64 = make(x, dtype, pad, off)
    ids, w = Guarded(x.shape[0], k, torch.int32), Guarded(x.shape[0], k, torch.float32)
    kind = kw.pop("scores", "softmax")
    purlin.route_experts(xs, ids.view, w.view, h, bias=None if bias is None else floats(bias),
                         scores=purlin.Scores.SIGMOID if kind == "sigmoid" else purlin.Scores.SOFTMAX, stream=stream, **kw)
    assert ids.intact() and w.intact()
    return ids.view.cpu().numpy(), w.view, x64


ROUTES = [
    # tokens, experts, k, scores, bias, groups, kept, group_best, renormalise, scale
    (1, 8, 2, "softmax", False, 1, 1, 1, True, 1.0),
    (5, 1, 1, "softmax", False, 1, 1, 1, False, 1.0),
    (33, 7, 7, "sigmoid", False, 1, 1, 1, True, 2.5),
    (17, 33, 3, "softmax", False, 1, 1, 1, False, 1.0),
    (9, 60, 4, "softmax", False, 1, 1, 1, True, 1.0),
    (64, 64, 6, "softmax", True, 1, 1, 1, True, 16.0),
    (31, 64, 6, "softmax", False, 8, 3, 1, False, 16.0),
    (20, 160, 6, "softmax", False, 8, 3, 2, True, 1.0),
    (41, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
    (13, 256, 8, "sigmoid", False, 8, 4, 2, True, 2.5),
    (13, 96, 5, "sigmoid", True, 32, 7, 1, True, 1.0),
    (13, 32, 5, "sigmoid", False, 32, 9, 2, True, 1.0),
    (6, 384, 8, "sigmoid", True, 1, 1, 1, True, 1.0),
    (4, 1000, 32, "softmax", False, 5, 2, 1, True, 1.0),
    (4, 1024, 10, "softmax", False, 1, 1, 1, True, 1.0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", ROUTES, ids=str)
def test_route(h, case, dtype):
    T, E, k, kind, biased, groups, kept, best, renorm, scale = case
    rng = np.random.default_rng(E + k)
    x = spread(rng, T, E, -1.0, 1.0) if biased else spread(rng, T, E)
    # tiers, so that scores of different experts stay apart after the bias is added
    bias = rng.integers(0, 3, E) * 1.0 if biased else None
    for pad, off in ((0, 0), (3, 1), (8, 8)):
        ids, w, x64 = run_route(h, x, k, dtype, pad, off, scores=kind, bias=bias, groups=groups, kept_groups=kept,
                                group_best=best, renormalise=renorm, scale=scale)
        margin = []
        want, want_w = O.route(x64, k, kind, bias, groups, kept, best, renorm, scale, margin)
        # a decision lies this far from the next: keys of size 6 at most, off by a few roundings each
        assert not margin or min(margin) > 6 * 6 * E24
        assert np.array_equal(ids, want)
        # expf of a rounded difference of size 6, the sum of E terms, divisions, the picks' sum, the scale
        close(w, want_w, np.abs(want_w) * (2 * 6 + 2 * 4 + E + k + 8) * E24 + 1e-30)


@pytest.mark.parametrize("dtype", DTYPES)
def test_route_ties_fall_to_the_lowest_expert(h, dtype):
    ids, w, _ = run_route(h, np.zeros((3, 100)), 5, dtype)
    assert (ids == np.arange(5)).all()
    close(w, 0.2, 8 * E24)
    x = np.tile(np.array([0.0, -0.0, 1.0, 1.0, -0.0, 0.0]), (2, 1))
    for kind in ("softmax", "sigmoid"):
        ids, _, _ = run_route(h, x, 6, dtype, scores=kind)
        assert (ids == [2, 3, 0, 1, 4, 5]).all()
    # sigmoids that round to 1: without a bias the logits still order them
    ids, _, _ = run_route(h, np.array([[40.0, 50.0, 30.0, 60.0]]), 4, dtype, scores="sigmoid")
    assert (ids == [3, 1, 0, 2]).all()
    # equal groups: the first ones are kept
    ids, _, _ = run_route(h, np.zeros((2, 64)), 4, dtype, groups=16, kept_groups=1)
    assert (ids == np.arange(4)).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_with_experts_switched_off(h, kind):
    rng = np.random.default_rng(0)
    x = spread(rng, 6, 24)
    x[0] = -np.inf
    x[1, 3:] = -np.inf
    x[2, :8] = -np.inf           # a whole group
    x[3, 1:8] = -np.inf          # one expert of a group
    x[4] = np.where(np.arange(24) % 2, np.finfo(np.float32).min, x[4])   # the lowest value is a value
    for kw in ({}, dict(groups=3, kept_groups=2, group_best=2), dict(groups=3, kept_groups=2, group_best=1)):
        ids, w, x64 = run_route(h, x, 8, torch.float32, scores=kind, **kw)
        want, want_w = O.route(x64, 8, kind, **kw)
        assert np.array_equal(ids, want)
        close(w, want_w, np.abs(want_w) * 64 * E24 + 1e-30)
        assert (ids[0] == -1).all() and (w[0] == 0).all()
    # a bias of -inf switches an expert off for every token
    bias = np.zeros(24)
    bias[:20] = -np.inf
    ids, w, x64 = run_route(h, spread(rng, 3, 24), 6, torch.float32, scores=kind, bias=bias)
    assert np.array_equal(ids, O.route(x64, 6, kind, bias)[0]) and (ids[:, 4:] == -1).all() and (ids[:, :4] >= 20).all()


def test_route_nan_and_infinity(h):
    x = np.zeros((4, 10))
    x[:, 4] = 1.0
    x[0, 2] = np.nan
    x[1] = np.nan
    x[2, 7] = np.inf
    ids, w, _ = run_route(h, x, 3, torch.float32)
    assert ids.tolist() == [[4, 0, 1], [-1, -1, -1], [7, 4, 0], [4, 0, 1]]
    w = w.cpu().numpy()
    assert np.isnan(w[0]).all() and (w[1] == 0).all() and np.isnan(w[2]).all() and np.isfinite(w[3]).all()
    ids, w, _ = run_route(h, x, 3, torch.float32, scores="sigmoid", renormalise=False)
    assert ids.tolist() == [[4, 0, 1], [-1, -1, -1], [7, 4, 0], [4, 0, 1]]
    assert np.isfinite(w.cpu().numpy()).all() and w[2, 0] == 1.0


def test_route_scores_too_small_to_renormalise(h):
    # a bias makes the token pick experts whose probabilities round to 0
    x = np.zeros((1, 8))
    x[0, 0] = 200.0
    bias = np.where(np.arange(8) < 4, -10.0, 10.0)
    ids, w, _ = run_route(h, x, 2, torch.float32, bias=bias)
    assert ids.tolist() == [[4, 5]] and (w == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("T,E,k,pad", [(1, 1, 1, 0), (3, 8, 2, 0), (65, 60, 4, 5), (7, 256, 8, 0), (2, 1000, 32, 0)])
def test_route_gradient(h, T, E, k, pad, kind, renormalise, dtype):
    rng = np.random.default_rng(E)
    xs, x64 = make(rng.standard_normal((T, E)) * 2, dtype, pad)
    ids, _ = O.route(x64, k, kind)
    ids[T // 2, k // 2:] = -1            # fewer picks, and below no picks, and an id out of range
    if T > 2:
        ids[1, :] = -1
        ids[2, 0] = E
    dw = rng.standard_normal((T, k))
    dws, dw64 = make(dw, torch.float32)
    out = Guarded(T, E, dtype, pad)
    purlin.route_experts_grad(xs, ints(ids), dws, out.view, h, scores=purlin.Scores.SIGMOID if kind == "sigmoid"
                              else purlin.Scores.SOFTMAX, renormalise=renormalise, scale=2.5)
    want = O.route_grad(x64, np.where(ids < E, ids, -1), dw64, kind, renormalise, 2.5)
    # the terms that cancel: picks' gradients over the picks' sum, times scores and their mean
    s = np.stack([O.scores_of(r, kind) for r in x64])
    live = (ids >= 0) & (ids < E)
    total = (np.take_along_axis(s, np.where(live, ids, 0), 1) * live).sum(1, keepdims=True) if renormalise else np.ones((T, 1))
    size = 2 * s * 2.5 * (np.abs(dw64) * live).sum(1, keepdims=True) / np.maximum(total, 1e-20)
    close(out.view, want, np.abs(want) * U[dtype] + size * (E + 4 * k + 40) * E24)
    assert out.intact()


# ------------------------------------------------------------------ exchange

@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 32, 1024), (5, 3, 2), (17, 8, 128), (1000, 8, 7),
                                   (1024, 8, 256), (8193, 1, 64), (1025, 8, 1024), (20000, 8, 256), (200003, 6, 33),
                                   (2048, 1, 16), (2049, 1, 16), (4097, 1, 1024), (32768, 2, 100), (65537, 1, 100),
                                   (3000, 8, 1024), (16384, 1, 7), (16385, 1, 1024)])
def test_plan(h, T, k, E):
    rng = np.random.default_rng(T + k)
    ids = rng.integers(-1, E + 2, (T, k)) if E > 1 else rng.integers(0, 2, (T, k))
    if T > 8:
        ids[: T // 4] = 1          # a run of one expert
    offsets, places = Guarded(1, E + 1, torch.int32), Guarded(max(T, 1), k, torch.int32)
    purlin.expert_plan(ints(ids), offsets.view[0], places.view[:T], h)
    want_o, want_p = O.plan(ids, E)
    assert np.array_equal(offsets.view[0].cpu().numpy(), want_o)
    assert np.array_equal(places.view[:T].cpu().numpy(), want_p)
    assert offsets.intact() and places.intact()


def exchange(rng, T, k, E, dropped=True):
    ids = np.stack([rng.permutation(max(E, k))[:k] for _ in range(T)])
    ids[ids >= E] = -1
    if dropped and T > 2:
        ids[1] = -1
        ids[2, 0] = -1
    return O.plan(ids, E)[1]


ROWS = [(1, 1, 1, 0, 0), (2, 1, 8, 0, 0), (5, 2, 7, 0, 0), (3, 8, 129, 3, 1), (19, 8, 64, 0, 8), (9, 6, 1537, 0, 0),
        (33, 4, 1000, 24, 0), (4, 32, 256, 0, 2), (40, 8, 4096, 0, 0), (7, 3, 5000, 0, 4)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,D,pad,off", ROWS)
def test_dispatch_and_combine(h, T, k, D, pad, off, dtype):
    rng = np.random.default_rng(D)
    places = exchange(rng, T, k, 64)
    x, x64 = make(rng.standard_normal((T, D)), dtype, pad, off)
    rows = Guarded(T * k, D, dtype, pad, off)
    purlin.dispatch_rows(x, ints(places), rows.view, h)
    assert np.array_equal(rows.view.double().cpu().numpy(), O.dispatch(x64, places)) and rows.intact()

    r, r64 = make(rng.standard_normal((T * k, D)), dtype, pad, off)
    r64[~places[places < 0]] = 5.0
    r.copy_(torch.from_numpy(r64))
    r[torch.from_numpy(~places[places < 0])] = float("nan")       # rows of dropped picks are not read
    w, w64 = make(rng.standard_normal((T, k)), torch.float32)
    for weights, weights64 in ((w, w64), (None, None)):
        y = Guarded(T, D, dtype, pad, off)
        purlin.combine_rows(r, ints(places), weights, y.view, h)
        want = O.combine(r64, places, weights64)
        size = O.combine(np.abs(r64), places, None if weights is None else np.abs(weights64))
        close(y.view, want, np.abs(want) * U[dtype] + size * (k + 2) * E24)
        assert y.intact()

    dy, dy64 = make(rng.standard_normal((T, D)), dtype, pad, off)
    dr, dw = Guarded(T * k, D, dtype, pad, off), Guarded(T, k, torch.float32)
    r.copy_(torch.from_numpy(r64))
    purlin.combine_rows_grad(r, ints(places), w, dy, dr.view, dw.view, h)
    want_r, want_w = O.combine_grad(r64, places, w64, dy64)
    close(dr.view, want_r, np.abs(want_r) * (U[dtype] + 2 * E24))
    size = O.combine_grad(np.abs(r64), places, np.abs(w64), np.abs(dy64))[1]
    close(dw.view, want_w, size * (D + 2) * E24)
    assert dr.intact() and dw.intact()


@pytest.mark.parametrize("D", [64, 67])
def test_dispatch_copies_every_bit_pattern(h, D):
    bits = torch.randint(-2**15, 2**15, (9, D), dtype=torch.int32, device=DEV).to(torch.int16)   # NaN payloads among them
    places = O.plan(np.tile(np.arange(3), (9, 1)), 3)[1]
    rows = torch.empty(27, D, dtype=torch.bfloat16, device=DEV)
    purlin.dispatch_rows(bits.view(torch.bfloat16), ints(places), rows, h)
    want = O.dispatch(bits.cpu().numpy(), places)
    assert np.array_equal(rows.view(torch.int16).cpu().numpy(), want)


def test_combine_with_a_weight_of_infinity_stays_in_its_row(h):
    places = ints(O.plan(np.array([[0], [1], [2]]), 3)[1])
    rows = torch.ones(3, 8, device=DEV)
    w = torch.tensor([[1.0], [math.inf], [math.nan]], device=DEV)
    y = torch.empty(3, 8, device=DEV)
    purlin.combine_rows(rows, places, w, y, h)
    assert (y[0] == 1).all() and torch.isinf(y[1]).all() and torch.isnan(y[2]).all()


def test_places_outside_the_rows_are_skipped_and_reported(h):
    x = torch.ones(2, 16, device=DEV)
    rows = Guarded(4, 16, torch.float32)
    places = ints([[0, 4], [-9, 1]])
    purlin.dispatch_rows(x, places, rows.view, h)
    st, dev = P.purlin_status_get(h.raw, torch.cuda.current_stream().cuda_stream)
    assert (st, dev) == (P.PL_OK, P.PL_ERR_BOUNDS) and rows.intact()
    assert (rows.view[:2] == 1).all() and (rows.view[2:] == -77).all()
    y = Guarded(2, 16, torch.float32)
    purlin.combine_rows(x.repeat(2, 1), places, None, y.view, h)
    st, dev = P.purlin_status_get(h.raw, torch.cuda.current_stream().cuda_stream)
    assert dev == P.PL_ERR_BOUNDS and (y.view == 1).all()
    dr, dw = Guarded(4, 16, torch.float32), Guarded(2, 2, torch.float32)
    purlin.combine_rows_grad(x.repeat(2, 1), places, torch.ones(2, 2, device=DEV), x, dr.view, dw.view, h)
    st, dev = P.purlin_status_get(h.raw, torch.cuda.current_stream().cuda_stream)
    assert dev == P.PL_ERR_BOUNDS and dr.intact() and dw.view.tolist() == [[16.0, 0.0], [0.0, 16.0]]
    st, dev = P.purlin_status_get(h.raw, torch.cuda.current_stream().cuda_stream)
    assert dev == P.PL_OK


def test_exchange_past_32_bit_offsets(h):
    """Rows of 2.3 Gi elements: every row checked on the GPU."""
    T, k, D, E = 70001, 8, 4096, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(T, D, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, 1).indices.to(torch.int32)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    places = torch.empty(T, k, dtype=torch.int32, device=DEV)
    rows = torch.empty(T * k, D, dtype=torch.bfloat16, device=DEV)
    purlin.expert_plan(ids, offsets, places, h)
    purlin.dispatch_rows(x, places, rows, h)
    order = ids.flatten().sort(stable=True).indices
    for a in range(0, T * k, 1 << 17):
        part = order[a:a + (1 << 17)]
        assert torch.equal(rows[a:a + (1 << 17)], x[part // k])
    y = torch.empty_like(x)
    purlin.combine_rows(rows, places, torch.full((T, k), 0.125, device=DEV), y, h)
    assert torch.equal(y, x)                       # eight eighths of one value are exact
    grad_rows, grad_w = torch.empty_like(rows), torch.empty(T, k, device=DEV)
    purlin.combine_rows_grad(rows, places, torch.full((T, k), 0.5, device=DEV), x, grad_rows, grad_w, h)
    for a in range(0, T * k, 1 << 17):
        assert torch.equal(grad_rows[a:a + (1 << 17)], rows[a:a + (1 << 17)] * 0.5)    # halves are exact
    # every pick's product is the token's with itself: D squares near 1, in binary32
    assert ((grad_w - x.float().square().sum(1, keepdim=True)).abs() <= 2 * D * D * E24 * 2).all()
    assert torch.equal(grad_w, grad_w[:, :1].expand(-1, k))
    assert P.purlin_status_get(h.raw)[1] == P.PL_OK


def test_route_past_32_bit_offsets(h):
    """2.1 Gi logits: the last tokens are routed as they are alone."""
    T, E, k = 2100007, 1024, 4
    x = torch.empty(T, E, dtype=torch.bfloat16, device=DEV)
    x[:-100].fill_(0.0)
    x[-100:].normal_(generator=torch.Generator(device=DEV).manual_seed(3))
    ids, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    purlin.route_experts(x, ids, w, h)
    ids1, w1 = torch.empty(100, k, dtype=torch.int32, device=DEV), torch.empty(100, k, device=DEV)
    purlin.route_experts(x[-100:].clone(), ids1, w1, h)
    assert torch.equal(ids[-100:], ids1) and torch.equal(w[-100:], w1)
    assert (ids[:-100] == torch.arange(k, device=DEV, dtype=torch.int32)).all() and (w[:-100] == 0.25).all()
    grad, grad1 = torch.empty_like(x), torch.empty(100, E, dtype=torch.bfloat16, device=DEV)
    dw = torch.ones(T, k, device=DEV)
    dw[:, 0] = 2.0
    purlin.route_experts_grad(x, ids, dw, grad, h)
    purlin.route_experts_grad(x[-100:].clone(), ids1, dw[:100], grad1, h)
    assert torch.equal(grad[-100:], grad1) and torch.equal(grad[0], grad[T // 2])


# ----------------------------------------------------------------- embedding

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("n,R,D,pad,off,first", [(1, 1, 1, 0, 0, 0), (5, 100, 7, 0, 0, 0), (300, 50, 64, 0, 0, 25),
                                                 (33, 10, 1537, 0, 0, -3), (9, 64, 4096, 0, 0, 1 << 20), (70, 9, 40, 5, 3, 0)])
def test_embed(h, n, R, D, pad, off, first, wide, dtype):
    rng = np.random.default_rng(n)
    table, t64 = make(rng.standard_normal((R, D)), dtype, pad, off)
    tokens = rng.integers(first - 3, first + R + 3, n)
    tokens[0] = -100
    dev = torch.from_numpy(tokens).to(DEV).to(torch.int64 if wide else torch.int32)
    for scale in (1.0, 8.3125):
        out = Guarded(n, D, dtype, pad, off)
        purlin.embed(table, dev, out.view, h, first=first, scale=scale)
        want = O.embed(t64, tokens, first, scale)
        close(out.view, want, np.abs(want) * (U[dtype] + E24) if scale != 1.0 else 0.0)
        assert out.intact()


def test_embed_far_tokens(h):
    """Tokens at the ends of 64 bits are outside the range, not wrapped into it."""
    table = torch.ones(4, 8, device=DEV)
    tokens = torch.tensor([-2**63, 2**63 - 1, 2**32, 2**32 + 1, 3, -1], device=DEV)
    out = torch.empty(6, 8, device=DEV)
    purlin.embed(table, tokens, out, h)
    assert out.sum(1).tolist() == [0, 0, 0, 0, 8, 0]
    grad = torch.empty(4, 8, device=DEV)
    purlin.embed_grad(out.fill_(1.0), tokens, grad, h)
    assert grad.sum(1).tolist() == [0, 0, 0, 8]


GRADS = [
    # tokens, rows, width, pad, off, first, how the tokens fall
    (1, 1, 1, 0, 0, 0, "any"), (3, 5, 9, 0, 0, 0, "any"), (32, 7, 8, 0, 0, 0, "one"), (33, 7, 8, 0, 0, 0, "one"),
    (64, 40, 64, 0, 0, 5, "any"), (100, 1000, 129, 3, 1, 0, "any"), (1000, 50, 40, 0, 0, 0, "hot"),
    (4097, 3000, 16, 0, 0, -7, "hot"), (8192, 100, 8, 0, 0, 0, "any"), (8193, 100, 8, 0, 0, 0, "any"),
    (9000, 2, 24, 0, 0, 0, "one"), (20000, 70000, 8, 0, 0, 0, "hot"), (8200, 1300000, 2, 0, 0, 0, "any"),
    (300, 1100000, 4, 0, 0, 0, "any"), (200, 64, 1100, 0, 0, 0, "outside"), (170000, 900, 4, 0, 0, 0, "hot"),
    (2048, 3000, 4, 0, 0, 0, "any"), (2049, 3000, 4, 0, 0, 0, "hot"), (65536, 700, 4, 0, 0, 0, "hot"),
    (65537, 70000, 4, 0, 0, 0, "hot"), (40, 600000, 3, 1, 0, 0, "any"), (0, 100, 48, 0, 0, 0, "any"),
]


@pytest.mark.parametrize("dtypes", [(x, t) for x in DTYPES for t in DTYPES], ids=str)
@pytest.mark.parametrize("case", GRADS, ids=str)
def test_embed_gradient(h, case, dtypes):
    n, R, D, pad, off, first, fall = case
    rng = np.random.default_rng(n)
    tokens = rng.integers(first - 2, first + R + 2, n)
    if fall == "one":
        tokens[:] = first + R // 2
    elif fall == "hot":
        tokens[rng.random(n) < 0.4] = first + R // 3
    elif fall == "outside":
        tokens[:] = first + R
    dy, dy64 = make(rng.standard_normal((n, D)), dtypes[0], pad, off)
    dev = torch.from_numpy(tokens).to(DEV)
    at = tokens - first
    inside = (at >= 0) & (at < R)
    total, size, count = np.zeros((R, D)), np.zeros((R, D)), np.zeros((R, 1))
    np.add.at(total, at[inside], dy64[inside])          # 64 bits
    np.add.at(size, at[inside], np.abs(dy64[inside]))
    np.add.at(count, at[inside], 1.0)
    first_base, b64 = make(rng.standard_normal((R, D)), dtypes[1], pad, off)
    for base in ("none", "other", "same"):
        out = Guarded(R, D, dtypes[1], pad, off)
        if base == "same":
            out.view.copy_(first_base)
        purlin.embed_grad(dy, dev, out.view, h, first=first, scale=1.5,
                          base={"none": None, "other": first_base, "same": out.view}[base])
        want = 1.5 * total + (0.0 if base == "none" else b64)
        bound = np.abs(want) * (U[dtypes[1]] + E24) + 1.5 * size * (count + 2) * E24
        close(out.view, want, bound)
        assert out.intact()


def test_embed_past_32_bit_offsets(h):
    """A table of 2.2 Gi elements: lookups near its end, and the gradient's rows."""
    R, D = 530001, 4096
    table = torch.empty(R, D, dtype=torch.bfloat16, device=DEV)
    tokens = torch.tensor([R - 1, 0, R // 2, R - 1, R, 524288], device=DEV)
    table[tokens[[0, 1, 2, 5]]] = torch.arange(1, 5, device=DEV, dtype=torch.bfloat16)[:, None].expand(-1, D)
    out = torch.empty(6, D, dtype=torch.bfloat16, device=DEV)
    purlin.embed(table, tokens, out, h)
    assert (out == torch.tensor([1, 2, 3, 1, 0, 4], device=DEV)[:, None]).all()
    table.fill_(9.0)
    purlin.embed_grad(out, tokens, table, h)
    want = torch.zeros(R, device=DEV)
    want[tokens[[0, 1, 2, 5]]] = torch.tensor([2.0, 2, 3, 4], device=DEV)
    for a in range(0, R, 1 << 16):
        assert (table[a:a + (1 << 16)].float() == want[a:a + (1 << 16), None]).all()


def test_embed_gradient_of_a_long_narrow_table(h):
    """So many rows that a CTA marks its share in several pieces."""
    R = 90000001
    tokens = torch.tensor([0, R - 1, 45000000, 262144, 262143, R - 1], device=DEV)
    grad = torch.full((R, 1), 7.0, dtype=torch.bfloat16, device=DEV)
    purlin.embed_grad(torch.ones(6, 1, dtype=torch.bfloat16, device=DEV), tokens, grad, h)
    at = grad[:, 0].nonzero()[:, 0]
    assert at.tolist() == [0, 262143, 262144, 45000000, R - 1] and grad[at, 0].tolist() == [1, 1, 1, 1, 2]


def test_embed_gradient_repeats_bit_for_bit(h):
    g = torch.Generator(device=DEV).manual_seed(2)
    dy = torch.randn(30000, 264, generator=g, device=DEV)
    tokens = (torch.rand(30000, generator=g, device=DEV) ** 6 * 5000).to(torch.int64)
    outs = [torch.empty(5000, 264, device=DEV) for _ in range(3)]
    for o in outs:
        purlin.embed_grad(dy, tokens, o, h)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ---------------------------------------------------------------------- clip

def clip_inputs(rng, sizes, dtype, offs):
    tensors, values = [], []
    for i, n in enumerate(sizes):
        v = rng.standard_normal(n) * 10.0 ** rng.integers(-3, 1)
        t, v64 = make(v[None, :], dtype, 0, offs[i % len(offs)])
        tensors.append(t[0])
        values.append(v64[0])
    return tensors, values


SIZES = {"one": [1], "small": [3, 1, 8, 16, 17, 1000], "chunks": [16384, 16385, 40000, 5], "empty": [0, 7, 0],
         "many": [5 + i % 7 for i in range(65)], "very many": [1 + i % 5 for i in range(1100)], "large": [3000001, 70]}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("max_norm,scale", [(0.25, 1.0), (1e9, 0.125), (math.inf, -2.0), (0.0, 1.0)])
def test_clip(h, sizes, dtype, max_norm, scale):
    rng = np.random.default_rng(7)
    grads, values = clip_inputs(rng, SIZES[sizes], dtype, (0, 1, 8, 3))
    outs = [Guarded(1, g.numel(), dtype, 0, (0, 1, 8, 2)[i % 4]) for i, g in enumerate(grads)]
    norm = torch.empty(1, device=DEV)
    purlin.clip_grad_norm(grads, [o.view[0] for o in outs], max_norm, norm, h, scale=scale)
    want, want_norm = O.clip(values, max_norm, scale)
    # 32 squares at most are added in binary32 by one thread, the rest in 64 bits; then one rounding
    assert abs(norm.item() - want_norm) <= want_norm * (32 + 4) * E24
    for o, w in zip(outs, want):
        close(o.view[0], w, np.abs(w) * (U[dtype] + (36 + 8) * E24))
        assert o.intact()
    alone = torch.empty(1, device=DEV)
    purlin.clip_grad_norm(grads, None, max_norm, alone, h, scale=scale)
    assert torch.equal(alone, norm)
    purlin.clip_grad_norm(grads, grads, max_norm, alone, h, scale=scale)        # in place
    assert torch.equal(alone, norm)
    for g, o in zip(grads, outs):
        assert torch.equal(g, o.view[0])


def test_clip_of_nothing(h):
    norm = torch.full((1,), 7.0, device=DEV)
    purlin.clip_grad_norm([], [], 1.0, norm, h)
    assert norm.item() == 0.0
    z = [torch.zeros(100, device=DEV)]
    purlin.clip_grad_norm(z, z, 1.0, norm, h)
    assert norm.item() == 0.0 and (z[0] == 0).all()


def test_clip_past_32_bit_offsets(h):
    n = 2200000003
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device=DEV)
    norm = torch.empty(1, device=DEV)
    purlin.clip_grad_norm([g], [g], 0.25 * math.sqrt(n), norm, h)     # half of the norm
    assert abs(norm.item() - 0.5 * math.sqrt(n)) <= 0.5 * math.sqrt(n) * 4 * E24     # all partial sums are exact
    assert (g == 0.25).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_clip_of_values_whose_squares_overflow(h, dtype):
    """The squares pass binary32, the norm does not."""
    rng = np.random.default_rng(1)
    for n in (100, 200000):
        g, v = make(rng.standard_normal((1, n)) * 1e30, dtype)
        norm, out = torch.empty(1, device=DEV), Guarded(1, n, dtype)
        purlin.clip_grad_norm([g[0]], [out.view[0]], 1.0, norm, h)
        want, want_norm = O.clip([v[0]], 1.0)
        assert abs(norm.item() - want_norm) <= want_norm * 4 * E24     # all in 64 bits, rounded to 32
        # the factor is 1 / norm, near 1e-33, and a product near 1e-3 rounds like any
        close(out.view[0], want[0], np.abs(want[0]) * (U[dtype] + 12 * E24))


def test_clip_with_values_that_are_not_finite(h):
    norm = torch.empty(1, device=DEV)
    g = [torch.ones(100, device=DEV), torch.ones(5, device=DEV)]
    o = [torch.empty_like(t) for t in g]
    g[1][2] = math.inf
    purlin.clip_grad_norm(g, o, 1.0, norm, h)
    assert math.isinf(norm.item()) and (o[0] == 0).all() and math.isnan(o[1][2].item()) and o[1][0].item() == 0
    g[1][2] = math.nan
    purlin.clip_grad_norm(g, o, 1.0, norm, h)
    assert math.isnan(norm.item()) and torch.isnan(o[0]).all() and torch.isnan(o[1]).all()
    purlin.clip_grad_norm(g, o, math.inf, norm, h, scale=0.5)      # never clips
    assert math.isnan(norm.item()) and (o[0] == 0.5).all()


# ----------------------------------------------- streams, graphs, refusals

def everything(h, stream=None):
    """One call of each operator on small fixed inputs; returns the outputs."""
    g = torch.Generator(device=DEV).manual_seed(9)
    T, k, E, D, R = 300, 4, 32, 48, 500
    logits = torch.randn(T, E, generator=g, device=DEV)
    x = torch.randn(T, D, generator=g, device=DEV)
    tokens = torch.randint(0, R, (9000,), generator=g, device=DEV)
    dy = torch.randn(9000, D, generator=g, device=DEV)
    table = torch.randn(R, D, generator=g, device=DEV)
    o = dict(ids=torch.empty(T, k, dtype=torch.int32, device=DEV), w=torch.empty(T, k, device=DEV),
             dl=torch.empty(T, E, device=DEV), offsets=torch.empty(E + 1, dtype=torch.int32, device=DEV),
             places=torch.empty(T, k, dtype=torch.int32, device=DEV), rows=torch.empty(T * k, D, device=DEV),
             y=torch.empty(T, D, device=DEV), dr=torch.empty(T * k, D, device=DEV), dw=torch.empty(T, k, device=DEV),
             emb=torch.empty(9000, D, device=DEV), dt=torch.empty(R, D, device=DEV), clipped=torch.empty(R, D, device=DEV),
             norm=torch.empty(1, device=DEV))

    def call():
        purlin.route_experts(logits, o["ids"], o["w"], h, stream=stream)
        purlin.expert_plan(o["ids"], o["offsets"], o["places"], h, stream=stream)
        purlin.dispatch_rows(x, o["places"], o["rows"], h, stream=stream)
        purlin.combine_rows(o["rows"], o["places"], o["w"], o["y"], h, stream=stream)
        purlin.combine_rows_grad(o["rows"], o["places"], o["w"], x, o["dr"], o["dw"], h, stream=stream)
        purlin.route_experts_grad(logits, o["ids"], o["dw"], o["dl"], h, stream=stream)
        purlin.embed(table, tokens, o["emb"], h, stream=stream)
        purlin.embed_grad(dy, tokens, o["dt"], h, stream=stream)
        purlin.clip_grad_norm([o["dt"]], [o["clipped"]], 1.0, o["norm"], h, stream=stream)
    return call, o


def test_other_streams_and_graphs_give_the_same(h):
    call, want = everything(h)
    call()
    torch.cuda.synchronize()
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


def test_streams_of_one_handle_need_no_order(h):
    """The same handle on two streams at once: each has its workspace."""
    g = torch.Generator(device=DEV).manual_seed(5)
    jobs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for n in (30000, 50000):
        tokens = (torch.rand(n, generator=g, device=DEV) ** 4 * 3000).to(torch.int64)
        dy = torch.randn(n, 128, generator=g, device=DEV)
        ids = torch.randint(0, 64, (n, 4), generator=g, device=DEV, dtype=torch.int32)
        jobs.append((tokens, dy, ids))

    def run(job, stream):
        tokens, dy, ids = job
        grad, offsets, places = torch.empty(3000, 128, device=DEV), torch.empty(65, dtype=torch.int32, device=DEV), torch.empty_like(ids)
        clipped, norm = torch.empty_like(dy), torch.empty(1, device=DEV)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            purlin.embed_grad(dy, tokens, grad, h, stream=stream)
            purlin.expert_plan(ids, offsets, places, h, stream=stream)
            purlin.clip_grad_norm([dy], [clipped], 1.0, norm, h, stream=stream)
        return grad, offsets, places, clipped, norm
    want = [run(j, None) for j in jobs]
    torch.cuda.synchronize()
    got = [run(j, s) for j, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        for a, b in zip(w, o):
            assert torch.equal(a, b)


def test_renormalised_weights_sum_to_one(h):
    call, o = everything(h)
    call()
    torch.cuda.synchronize()
    assert P.purlin_status_get(h.raw)[1] == P.PL_OK
    assert (o["w"].double().sum(1) - 1).abs().max().item() < 8 * E24


def refused(fn, *args, **kw):
    with pytest.raises((ValueError, P.PurlinError)):
        fn(*args, **kw)


def test_refusals_on_the_gpu(h):
    f = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device=DEV)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    refused(purlin.route_experts, f(4, 1025), i(4, 2), f(4, 2), h)                       # too many experts
    refused(purlin.route_experts, f(4, 64), i(4, 33), f(4, 33), h)                       # too many picks
    refused(purlin.route_experts, f(4, 2), i(4, 3), f(4, 3), h)                          # more picks than experts
    refused(purlin.route_experts, f(4, 10), i(4, 2), f(4, 2), h, groups=3)               # groups do not divide
    refused(purlin.route_experts, f(4, 12), i(4, 4), f(4, 4), h, groups=4, kept_groups=1)  # kept groups too small
    refused(purlin.route_experts, f(4, 12), i(4, 2), f(4, 2), h, groups=4, kept_groups=5)
    refused(purlin.route_experts, f(4, 12), i(4, 2), f(4, 2), h, groups=4, kept_groups=2, group_best=3)
    refused(purlin.route_experts, f(4, 12), i(4, 2), f(4, 2), h, scale=math.inf)
    refused(purlin.route_experts, f(4, 12), i(4, 2), f(4, 2), h, scores=2)
    buf = f(64)
    refused(purlin.route_experts, buf[:48].view(4, 12), i(4, 2), buf[40:48].view(4, 2), h)   # output inside the logits
    refused(purlin.expert_plan, i(4, 2), i(1026), i(4, 2), h)
    same = i(4, 2)
    refused(purlin.expert_plan, same, i(9), same, h)
    x = f(8, 16)
    refused(purlin.dispatch_rows, x[:4], i(4, 2), x, h)
    refused(purlin.combine_rows, x, i(4, 2), None, x[4:], h)
    refused(purlin.combine_rows_grad, x, i(4, 2), f(4, 2), f(4, 16), x, f(4, 2), h)
    refused(purlin.embed, x, i(8), x, h)
    refused(purlin.embed_grad, x, i(8), x, h)
    refused(purlin.embed_grad, f(8, 16), i(8), x[1:], h, base=x[:7])                      # base overlaps, not the same
    refused(purlin.clip_grad_norm, [x], [x], -1.0, f(1), h)
    refused(purlin.clip_grad_norm, [x], [x], math.nan, f(1), h)
    refused(purlin.clip_grad_norm, [x], [x], 1.0, f(1), h, scale=math.nan)
    flat = f(100)
    refused(purlin.clip_grad_norm, [flat[:50], flat[40:90]], [flat[:50], flat[40:90]], 1.0, f(1), h)
    refused(purlin.clip_grad_norm, [flat[:50], flat[:50]], [flat[:50], f(50)], 1.0, f(1), h)
    refused(purlin.clip_grad_norm, [flat[:50]], [flat[1:51]], 1.0, f(1), h)
    refused(purlin.clip_grad_norm, [flat[:50], f(50)], [f(50), flat[:50]], 1.0, f(1), h)
    refused(purlin.clip_grad_norm, [flat], None, 1.0, flat[:1], h)
    purlin.clip_grad_norm([flat[:50], flat[:50]], [f(50), f(50)], 1.0, f(1), h)            # reads may share
    s = torch.cuda.current_stream().cuda_stream
    # workspaces too small, misaligned pointers, unknown handle
    assert P.purlin_expert_plan_bytes(90000, 1, 8) > 0
    assert P.purlin_expert_plan(h.raw, i(90000, 1), 90000, 1, 8, i(9), i(90000, 1), None, 0, s) == P.PL_ERR_WORKSPACE
    assert P.purlin_embed_grad(h.raw, x, 16, P.PL_F32, i(8), 4, 8, 16, 1.0, None, 0, f(8, 16), 16, P.PL_F32, 8, 0, None, 0,
                               s) == P.PL_ERR_WORKSPACE
    assert P.purlin_clip_grad_norm(h.raw, [x], None, [8], P.PL_F32, 1.0, 1.0, f(1), None, 0, s) == P.PL_ERR_WORKSPACE
    assert P.purlin_embed(h.raw, x.data_ptr() + 2, 16, 4, 0, i(4), 4, 4, 16, 1.0, P.PL_F32, f(4, 16), 16, s) == P.PL_ERR_ALIGNMENT
    assert P.purlin_embed(h.raw, x, 15, 8, 0, i(4), 4, 4, 16, 1.0, P.PL_F32, f(4, 16), 16, s) == P.PL_ERR_INVALID_ARG
    assert P.purlin_embed(h.raw, x, 16, 8, 0, i(4), 2, 4, 16, 1.0, P.PL_F32, f(4, 16), 16, s) == P.PL_ERR_UNSUPPORTED
    assert P.purlin_embed(h.raw, x, 16, 8, 0, i(4), 4, 4, 16, 1.0, P.PL_U8, f(4, 16), 16, s) == P.PL_ERR_UNSUPPORTED
    assert P.purlin_embed(h.raw, None, 16, 8, 0, i(4), 4, 4, 16, 1.0, P.PL_F32, f(4, 16), 16, s) == P.PL_ERR_INVALID_ARG
    assert P.purlin_embed(None, x, 16, 8, 0, i(4), 4, 4, 16, 1.0, P.PL_F32, f(4, 16), 16, s) == P.PL_ERR_INVALID_ARG
    host = torch.zeros(8, 16)
    assert P.purlin_embed(h.raw, host, 16, 8, 0, i(4), 4, 4, 16, 1.0, P.PL_F32, f(4, 16), 16, s) == P.PL_ERR_INVALID_ARG
    assert P.purlin_status_get(h.raw, s) == (P.PL_OK, P.PL_OK)


def test_tables_in_pinned_host_memory(h):
    table = torch.randn(50, 32).pin_memory()
    tokens = torch.tensor([3, 49, 50, 0, 3], device=DEV)
    out = torch.empty(5, 32, device=DEV)
    purlin.embed(table, tokens, out, h)
    assert torch.equal(out.cpu(), torch.cat([table[[3, 49]], torch.zeros(1, 32), table[[0, 3]]]))


@pytest.mark.parametrize("D", [64, 801])
def test_rows_in_pinned_host_memory(h, D):
    places = O.plan(np.tile(np.arange(4), (20, 1)), 4)[1]
    x = torch.randn(20, D)
    rows, y = torch.empty(80, D).pin_memory(), torch.empty(20, D).pin_memory()
    purlin.dispatch_rows(x.pin_memory(), ints(places), rows, h)
    torch.cuda.synchronize()
    assert np.array_equal(rows.numpy(), O.dispatch(x.numpy(), places))
    purlin.combine_rows(rows, ints(places), torch.full((20, 4), 0.25, device=DEV), y, h)
    torch.cuda.synchronize()
    assert torch.equal(y, x)            # four quarters of one value are exact


@pytest.mark.parametrize("n", [100, 30000])
def test_embed_gradient_of_32_bit_tokens(h, n):
    g = torch.Generator(device=DEV).manual_seed(8)
    tokens = torch.randint(-5, 205, (n,), generator=g, device=DEV)
    dy = torch.randn(n, 40, generator=g, device=DEV)
    wide, narrow = torch.empty(200, 40, device=DEV), torch.empty(200, 40, device=DEV)
    purlin.embed_grad(dy, tokens, wide, h)
    purlin.embed_grad(dy, tokens.to(torch.int32), narrow, h)
    assert torch.equal(wide, narrow)
