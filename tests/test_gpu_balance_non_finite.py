"""The balance of tokens that count and whose logits are not all finite, for both kinds of scores."""

import math

import numpy as np
import pytest
import torch

from oracle import operators as O
from collective_datapath_reduce_gb300 import torch_api as purlin
from test_gpu_operators import DTYPES, E24, U, Guarded, close, h, ints, make, spread  # noqa: F401 (h: a fixture)
from test_gpu_row_operators import F32, share_error

pytestmark = pytest.mark.gpu


def same(got, want, bound):
    """NaN where the definition has NaN, and only there; elsewhere within the bound."""
    got, nan = got.double().cpu(), np.isnan(want)
    assert np.array_equal(torch.isnan(got).numpy(), nan)
    keep = ~nan
    close(got[torch.from_numpy(keep)], want[keep], bound[keep])


WHAT = {
    "a NaN": lambda x, t: x.__setitem__((t, x.shape[1] // 2), math.nan),
    "all NaN": lambda x, t: x.__setitem__(t, math.nan),
    "a +inf": lambda x, t: x.__setitem__((t, 0), math.inf),
    "a NaN and a +inf": lambda x, t: (x.__setitem__((t, 0), math.inf), x.__setitem__((t, x.shape[1] - 1), math.nan)),
    "nothing but -inf": lambda x, t: x.__setitem__(t, -math.inf),
    "some -inf": lambda x, t: x.__setitem__((t, slice(None, None, 2)), -math.inf),
}


# one cluster and two launches, each with a token fetched ahead and (past 512 experts) without
@pytest.mark.parametrize("T,E,k", [(1, 2, 1), (70, 60, 4), (2100, 64, 6), (600, 600, 8), (700, 1000, 8)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("what", WHAT)
def test_logits_that_are_not_finite(h, what, dtype, kind, T, E, k):  # noqa: F811
    rng = np.random.default_rng(T + E)
    scores = purlin.Scores.SIGMOID if kind == "sigmoid" else purlin.Scores.SOFTMAX
    x, x64 = make(spread(rng, T, E), dtype)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    if T > 4:
        ids[3] = -1
    clean = O.balance(x64, ids, kind)[1]
    rows = sorted({T // 2, T - 1})
    for t in rows:
        WHAT[what](x, t)
    x64 = x.double().cpu().numpy()
    counts, sums, loss = Guarded(1, E, torch.int32), Guarded(1, 2 * E + 1, F32), Guarded(1, 1, F32)
    purlin.balance_loss(x, ints(ids), counts.view[0], sums.view[0], loss.view[0], h, scores=scores, scale=0.5)
    with np.errstate(invalid="ignore"):
        want_c, want_s, want = O.balance(x64, ids, kind, 0.5)
    assert ("NaN" in what or (kind == "softmax" and "+inf" in what)) == bool(np.isnan(want))
    assert np.array_equal(counts.view[0].cpu().numpy(), want_c)
    # the shares', then the tokens of a warp, its CTA's warps and the CTAs' sums; the loss adds the experts' products
    rel = share_error(E) + (T // 2432 + 1 + 8 + 8 + 38) * E24
    same(sums.view[0], want_s, np.abs(want_s) * rel)
    of_loss = rel + (E // 256 + 5 + 8 + 8 + 8) * E24
    same(loss.view[0], np.array([want]), np.abs(np.array([want])) * of_loss)
    joined = Guarded(1, 1, F32)
    purlin.balance_join(sums.view[0], joined.view[0], h, scale=0.5)
    same(joined.view[0], np.array([want]), np.abs(np.array([want])) * of_loss)
    assert counts.intact() and sums.intact() and loss.intact()

    # the gradient of finite sums: NaN stays in its own token
    given, s64 = make(clean[None], F32)
    base, base64 = make(rng.standard_normal((T, E)) * 1e-3, dtype)
    for b in (None, base):
        out = Guarded(T, E, dtype)
        purlin.balance_loss_grad(x, ints(ids), given[0], None, out.view, h, scores=scores, scale=0.5, base=b)
        with np.errstate(invalid="ignore"):
            want_g = O.balance_grad(x64, ids, s64[0], 1.0, kind, 0.5) + (0 if b is None else base64)
        size = np.zeros((T, E))
        for t in range(T):
            if any(0 <= e < E for e in ids[t]):
                c = 0.5 * E * s64[0, :E] / (s64[0, :E].sum() * s64[0, 2 * E])
                with np.errstate(invalid="ignore"):
                    p = O.shares_of(x64[t], kind)
                size[t] = p * (c + (p * c).sum())
        # the coefficient, two shares, their products' sum, three products
        same(out.view, want_g, np.abs(want_g) * (U[dtype] + E24) + size * (2 * share_error(E) + (E // 256 + E // 32 + 40) * E24))
        assert out.intact()
