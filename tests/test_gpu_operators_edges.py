"""Values, handles and buffers at the edges of what the operators' header allows.

Bounds as in test_gpu_operators.py."""

import math

import numpy as np
import pytest
import torch

from oracle import operators as O
from collective_datapath_reduce_gb300 import purlin as P
from collective_datapath_reduce_gb300 import torch_api as purlin
from test_gpu_operators import DEV, DTYPES, E24, U, Guarded, close, h, ints, make  # noqa: F401 (h: a fixture)

pytestmark = pytest.mark.gpu


# widths of whole vectors at aligned addresses, and odd ones
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,k", [(64, 3), (2048, 12), (67, 3), (801, 12)])
def test_combine_gradient_of_a_dropped_pick_is_zero_whatever_the_token_holds(h, D, k, dtype):
    rng = np.random.default_rng(D)
    T = 5
    ids = np.stack([rng.permutation(16)[:k] for _ in range(T)])
    ids[1, 0] = ids[1, k - 1] = ids[3, 1] = -1
    ids[4] = -1
    places = O.plan(ids, 16)[1]
    r, r64 = make(rng.standard_normal((T * k, D)), dtype)
    w, w64 = make(rng.standard_normal((T, k)), torch.float32)
    dy, dy64 = make(rng.standard_normal((T, D)), dtype)
    dy[1, D // 2], dy[3, 0], dy[4, D - 1] = math.inf, math.nan, -math.inf
    dr, dw = Guarded(T * k, D, dtype), Guarded(T, k, torch.float32)
    purlin.combine_rows_grad(r, ints(places), w, dy, dr.view, dw.view, h)
    dropped = torch.from_numpy(places < 0).to(DEV)
    assert (dw.view[dropped] == 0).all()
    assert (dr.view[torch.from_numpy(~places[places < 0]).to(DEV)] == 0).all()
    assert not torch.isfinite(dw.view[[1, 3]][~dropped[[1, 3]]]).any()      # picks that are not dropped follow the formula
    want_r, want_w = O.combine_grad(r64, places, w64, dy64)
    size = O.combine_grad(np.abs(r64), places, np.abs(w64), np.abs(dy64))[1]
    close(dw.view[[0, 2]], want_w[[0, 2]], size[[0, 2]] * (D + 2) * E24)
    at = places[[0, 2]].ravel()
    close(dr.view[torch.from_numpy(at).to(DEV)], want_r[at], np.abs(want_r[at]) * (U[dtype] + 2 * E24))
    assert dr.intact() and dw.intact()


@pytest.mark.parametrize("n", [100, 300000])
def test_clip_of_a_norm_that_only_its_scale_brings_into_range(h, n):
    """The gradients' own norm is past binary32, scale times it is not."""
    g, v = make(np.random.default_rng(2).uniform(-1.0, 1.0, (1, n)) * 3e38, torch.float32)
    assert float(np.linalg.norm(v)) > 3.5e38
    norm, out = torch.empty(1, device=DEV), Guarded(1, n, torch.float32)
    purlin.clip_grad_norm([g[0]], [out.view[0]], 1e3, norm, h, scale=2.0 ** -10)
    want, want_norm = O.clip([v[0]], 1e3, 2.0 ** -10)
    assert abs(norm.item() - want_norm) <= want_norm * 4 * E24          # all in 64 bits, rounded to 32
    # the factor is 1000 / the norm times the scale, above 1e-37: a binary32 value like any
    close(out.view[0], want[0], np.abs(want[0]) * (U[torch.float32] + 12 * E24))
    purlin.clip_grad_norm([g[0]], None, 1e3, norm, h, scale=0.0)
    assert norm.item() == 0.0


@pytest.mark.parametrize("dtypes", [(x, t) for x in DTYPES for t in DTYPES], ids=str)
@pytest.mark.parametrize("n,D", [(300, 2304), (9000, 64)])
def test_embed_gradient_with_a_workspace_that_is_just_16_byte_aligned(h, n, D, dtypes):
    """What the header asks of the workspace; several runs, so that parts of sums go through it."""
    R, s = 40, torch.cuda.current_stream().cuda_stream
    g = torch.Generator(device=DEV).manual_seed(n)
    dy = torch.randn(n, D, generator=g, device=DEV).to(dtypes[0])
    tokens = torch.randint(0, R, (n,), generator=g, device=DEV)
    tokens[::2] = 7
    kinds = [P.PL_F32 if t is torch.float32 else P.PL_BF16 for t in dtypes]
    need = P.purlin_embed_grad_bytes(n, R, D)
    raw = torch.full((need + 128,), 0xA5, dtype=torch.uint8, device=DEV)
    assert raw.data_ptr() % 32 == 0
    outs = []
    for off in (32, 48):
        out = Guarded(R, D, dtypes[1])
        ws = raw[off:off + need]
        assert P.purlin_embed_grad(h.raw, dy, D, kinds[0], tokens, 8, n, D, 1.0, None, 0, out.view, D, kinds[1], R, 0, ws,
                                   need, s) == P.PL_OK
        assert out.intact() and (raw[:off] == 0xA5).all() and (raw[off + need:] == 0xA5).all()
        raw.fill_(0xA5)
        outs.append(out.view)
    assert torch.equal(outs[0], outs[1])
    want = O.embed_grad(dy.double().cpu().numpy(), tokens.cpu().numpy(), R)
    size = O.embed_grad(dy.double().abs().cpu().numpy(), tokens.cpu().numpy(), R)
    close(outs[1], want, np.abs(want) * (U[dtypes[1]] + E24) + size * (n + 2) * E24)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", [(5, 1, 300), (4001, 1025, 7, 16384), (40000, 3)])
def test_clip_in_place_again_and_again(h, sizes, dtype):
    """Each call reads what the one before wrote to the same place; elsewhere it gives the same bits."""
    g = torch.Generator(device=DEV).manual_seed(sum(sizes))
    flat = torch.randn(sum(sizes) + 64 * len(sizes), generator=g, device=DEV).to(dtype)
    starts = [sum(sizes[:i]) + 3 * i for i in range(len(sizes))]      # any alignment
    here = [flat[a:a + n] for a, n in zip(starts, sizes)]
    there = [t.clone() for t in here]
    norm, same = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    for _ in range(12):
        purlin.clip_grad_norm(here, here, 0.5, norm, h, scale=1.5)
        new = [torch.empty_like(t) for t in there]
        before = sum(float((t.double() ** 2).sum()) for t in there) ** 0.5 * 1.5
        purlin.clip_grad_norm(there, new, 0.5, same, h, scale=1.5)
        there = new
        # 32 squares at most are added in binary32 by one thread, the rest in 64 bits
        assert abs(same.item() - before) <= before * (32 + 4) * E24
        # the tensors lie at other addresses modulo 16 here, so their threads' shares differ
        assert abs(norm.item() - same.item()) <= before * 2 * (32 + 4) * E24
        for t, u in zip(here, there):
            assert ((t.double() - u.double()).abs() <= u.double().abs() * (4 * U[dtype] + 200 * E24)).all()
        there = [t.clone() for t in here]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,groups,kept", [(32, 4, 4), (32, 4, 2), (60, 3, 3), (60, 3, 1), (256, 8, 8), (256, 8, 3), (1000, 5, 1),
                                            (256, 32, 32), (256, 32, 5)])
def test_route_keeps_the_group_of_an_infinite_logit(h, E, groups, kept, dtype):
    """Without groups the expert is the first pick; its group counts as infinite, not as nothing."""
    x = np.stack([np.random.default_rng(E + t).permutation(np.linspace(-3.0, 3.0, E)) for t in range(5)])
    x[0, E // 2] = x[1, E - 1] = x[2, 0] = x[2, E // 3] = x[3, 5] = np.inf
    xs, x64 = make(x, dtype)
    for kind, scores in (("softmax", purlin.Scores.SOFTMAX), ("sigmoid", purlin.Scores.SIGMOID)):
        for best in (1, 2):
            ids, w = Guarded(5, 4, torch.int32), Guarded(5, 4, torch.float32)
            purlin.route_experts(xs, ids.view, w.view, h, scores=scores, groups=groups, kept_groups=kept, group_best=best)
            assert ids.intact() and w.intact()
            want = O.route(x64, 4, kind, None, groups, kept, best)[0]
            got = ids.view.cpu().numpy()
            if kind == "softmax" or kept == groups or best == 1:
                assert got[:, 0].tolist() == [E // 2, E - 1, 0, 5, int(np.argmax(x64[4])) if best == 1 or kept == groups else got[4, 0]]
            assert np.array_equal(got, want), (kind, best)
            assert torch.isnan(w.view[:4, 0]).all() == (kind == "softmax") and torch.isfinite(w.view[4]).all()
