"""Kernel variants that are chosen by size, each at sizes that choose it, against the 64-bit statements.

Bounds as in test_gpu_operators.py.  The sizes follow the launch rules: several
tokens a group from 304 CTAs on, several column tiles past 256 vectors of a
sum's row and past 40 KiB of a token's unaligned pieces, running sums in shared
memory past 8 picks."""

import numpy as np
import pytest
import torch

from oracle import operators as O
from collective_datapath_reduce_gb300 import purlin as P
from collective_datapath_reduce_gb300 import torch_api as purlin
from test_gpu_operators import DEV, DTYPES, E24, U, Guarded, close, exchange, h, ints, make  # noqa: F401 (h: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,D", [(12001, 40), (3001, 1024)])
def test_embed_of_many_tokens(h, n, D, dtype):
    rng = np.random.default_rng(n)
    R = 700
    table, t64 = make(rng.standard_normal((R, D)), dtype)
    tokens = rng.integers(-5, R + 5, n)
    for scale in (1.0, 8.3125):
        out = Guarded(n, D, dtype)
        purlin.embed(table, torch.from_numpy(tokens).to(DEV), out.view, h, scale=scale)
        want = O.embed(t64, tokens, 0, scale)
        close(out.view, want, np.abs(want) * (U[dtype] + E24) if scale != 1.0 else 0.0)
        assert out.intact()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,D", [(2601, 1, 1024), (10001, 1, 40), (1303, 2, 1024), (1303, 3, 1024), (5001, 4, 64)])
def test_exchange_of_many_tokens_with_few_picks(h, T, k, D, dtype):
    rng = np.random.default_rng(T)
    places = exchange(rng, T, k, 16)
    x, x64 = make(rng.standard_normal((T, D)), dtype)
    rows = Guarded(T * k, D, dtype)
    purlin.dispatch_rows(x, ints(places), rows.view, h)
    assert np.array_equal(rows.view.double().cpu().numpy(), O.dispatch(x64, places)) and rows.intact()
    w, w64 = make(rng.standard_normal((T, k)), torch.float32)
    r64 = O.dispatch(x64, places) + 0.0
    for weights, weights64 in ((w, w64), (None, None)):
        y = Guarded(T, D, dtype)
        purlin.combine_rows(rows.view, ints(places), weights, y.view, h)
        want = O.combine(r64, places, weights64)
        size = O.combine(np.abs(r64), places, None if weights is None else np.abs(weights64))
        close(y.view, want, np.abs(want) * U[dtype] + size * (k + 2) * E24)
        assert y.intact()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,D", [(5, 12, 1537), (3, 32, 1001), (4, 8, 5001), (3, 9, 4099), (2, 17, 12289)])
def test_combine_of_unaligned_rows_in_tiles_and_with_many_picks(h, T, k, D, dtype):
    rng = np.random.default_rng(D)
    places = exchange(rng, T, k, 64)
    r, r64 = make(rng.standard_normal((T * k, D)), dtype)
    r64[~places[places < 0]] = 0.0
    r[torch.from_numpy(~places[places < 0]).to(DEV)] = float("nan")       # rows of dropped picks are not read
    w, w64 = make(rng.standard_normal((T, k)), torch.float32)
    for weights, weights64 in ((w, w64), (None, None)):
        y = Guarded(T, D, dtype)
        purlin.combine_rows(r, ints(places), weights, y.view, h)
        want = O.combine(r64, places, weights64)
        size = O.combine(np.abs(r64), places, None if weights is None else np.abs(weights64))
        close(y.view, want, np.abs(want) * U[dtype] + size * (k + 2) * E24)
        assert y.intact()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [67, 801])
def test_places_outside_unaligned_rows_are_skipped_and_reported(h, D, dtype):
    s = torch.cuda.current_stream().cuda_stream
    x, x64 = make(np.random.default_rng(D).standard_normal((2, D)), dtype)
    rows = Guarded(4, D, dtype)
    places = ints([[0, 4], [-9, 1]])
    purlin.dispatch_rows(x, places, rows.view, h)
    assert P.purlin_status_get(h.raw, s) == (P.PL_OK, P.PL_ERR_BOUNDS) and rows.intact()
    assert torch.equal(rows.view[:2], x) and (rows.view[2:] == -77).all()
    y = Guarded(2, D, dtype)
    r = torch.cat([x, x])
    purlin.combine_rows(r, places, None, y.view, h)
    assert P.purlin_status_get(h.raw, s) == (P.PL_OK, P.PL_ERR_BOUNDS) and torch.equal(y.view, x) and y.intact()
    dr, dw = Guarded(4, D, dtype), Guarded(2, 2, torch.float32)
    purlin.combine_rows_grad(r, places, torch.ones(2, 2, device=DEV), x, dr.view, dw.view, h)
    assert P.purlin_status_get(h.raw, s) == (P.PL_OK, P.PL_ERR_BOUNDS) and dr.intact() and dw.intact()
    assert torch.equal(dr.view[:2], x) and (dr.view[2:] == -77).all()
    assert dw.view[0, 1] == 0 and dw.view[1, 0] == 0
    size = (x64 ** 2).sum(1)
    close(torch.stack([dw.view[0, 0], dw.view[1, 1]]), size, size * (D + 2) * E24)
    assert P.purlin_status_get(h.raw, s) == (P.PL_OK, P.PL_OK)


@pytest.mark.parametrize("dtypes", [(x, t) for x in DTYPES for t in DTYPES], ids=str)
@pytest.mark.parametrize("n,R,D,hot", [(300, 50, 4096, True), (300, 50, 4096, False), (700, 3, 2304, True), (90, 40, 1111, True)])
def test_embed_gradient_in_column_tiles(h, n, R, D, hot, dtypes):
    rng = np.random.default_rng(n + D)
    tokens = rng.integers(-2, R + 2, n)
    if hot:
        tokens[rng.random(n) < 0.5] = R // 3
    dy, dy64 = make(rng.standard_normal((n, D)), dtypes[0])
    inside = (tokens >= 0) & (tokens < R)
    total, size, count = np.zeros((R, D)), np.zeros((R, D)), np.zeros((R, 1))
    np.add.at(total, tokens[inside], dy64[inside])
    np.add.at(size, tokens[inside], np.abs(dy64[inside]))
    np.add.at(count, tokens[inside], 1.0)
    base, b64 = make(rng.standard_normal((R, D)), dtypes[1])
    for kind in ("none", "other", "same"):
        out = Guarded(R, D, dtypes[1])
        if kind == "same":
            out.view.copy_(base)
        purlin.embed_grad(dy, torch.from_numpy(tokens).to(DEV), out.view, h, scale=1.5,
                          base={"none": None, "other": base, "same": out.view}[kind])
        want = 1.5 * total + (0.0 if kind == "none" else b64)
        close(out.view, want, np.abs(want) * (U[dtypes[1]] + E24) + 1.5 * size * (count + 2) * E24)
        assert out.intact()
