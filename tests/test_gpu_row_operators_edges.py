"""Layer norm, balance and distillation at odd addresses of every buffer, in host memory, past 32-bit offsets, by threads."""

import math
import threading

import numpy as np
import pytest
import torch

from oracle import operators as O
from collective_datapath_reduce_gb300 import purlin as P
from collective_datapath_reduce_gb300 import torch_api as purlin
from test_gpu_operators import DEV, E24, Guarded, h  # noqa: F401 (h: a fixture)
from test_gpu_row_operators import BF16, F32, everything, status

pytestmark = pytest.mark.gpu


def at(t, off):
    """A copy of t that starts `off` elements past a 256-byte boundary."""
    flat = torch.empty(t.numel() + off, dtype=t.dtype, device=t.device)
    out = flat[off:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_every_buffer_at_the_alignment_of_its_elements(h, dtype, off):  # noqa: F811
    """Results are those of aligned buffers: exactly where the arithmetic does not go by vectors."""
    g = torch.Generator(device=DEV).manual_seed(off)
    T, D, E, k, V, K = 37, 264, 40, 4, 1032, 12
    r = lambda *s, t=dtype: torch.randn(s, generator=g, device=DEV).to(t)  # noqa: E731
    x, dy, dt, w, b = r(T, D), r(T, D), r(T, D), r(D), r(D)
    logits, z, teacher, dl = r(T, E), r(T, V), r(T, K, t=F32), r(T, t=F32)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, 1).indices.to(torch.int32)
    words = torch.rand(T, V, generator=g, device=DEV).topk(K, 1).indices.to(torch.int32)

    def run(a):
        n = lambda *s, t=dtype: a(torch.zeros(s, dtype=t, device=DEV))  # noqa: E731
        o = dict(y=n(T, D), total=n(T, D), stats=n(T, 2, t=F32), dx=n(T, D), dw=n(D), db=n(D), counts=n(E, t=torch.int32),
                 sums=n(2 * E + 1, t=F32), loss=n(1, t=F32), dlogits=n(T, E), kl=n(T, t=F32), ks=n(T, 2, t=F32), dz=n(T, V))
        purlin.layer_norm(a(x), a(w), a(b), o["y"], h, residual=a(dt), total=o["total"], stats=o["stats"])
        purlin.layer_norm_grad(a(dy), o["total"], o["stats"], a(w), o["dx"], o["dw"], o["db"], h, grad_total=a(dt))
        purlin.balance_loss(a(logits), a(ids), o["counts"], o["sums"], o["loss"], h)
        purlin.balance_loss_grad(a(logits), a(ids), o["sums"], o["loss"], o["dlogits"], h, base=a(logits))
        purlin.distil_loss(a(z), a(words), a(teacher), o["kl"], o["ks"], h)
        purlin.distil_loss_grad(a(z), a(words), a(teacher), o["ks"], a(dl), o["dz"], h)
        return o
    want, got = run(lambda t: t), run(lambda t: at(t, off))
    for name in want:
        a, b_ = want[name].double(), got[name].double()
        # other orders of sums of 1032 terms at most, and the output's rounding
        step = 2.0 ** -7 if want[name].dtype is BF16 else 0.0
        bound = step * a.abs() + 2 * 1032 * E24 * a.abs().mean() * 16
        assert ((a - b_).abs() <= bound).all(), name
    assert torch.equal(want["counts"], got["counts"])


def test_rows_in_pinned_host_memory(h):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(1)
    for D in (96, 101):
        x = torch.randn(9, D, generator=g, device=DEV)
        y, dx = torch.empty_like(x), torch.empty_like(x)
        w, stats, dw = torch.randn(D, generator=g, device=DEV), torch.empty(9, 2, device=DEV), torch.empty(D, device=DEV)
        hx, hy, hdx = x.cpu().pin_memory(), torch.empty(9, D).pin_memory(), torch.empty(9, D).pin_memory()
        purlin.layer_norm(x, w, None, y, h, stats=stats)
        purlin.layer_norm(hx, w, None, hy, h)
        purlin.layer_norm_grad(y, x, stats, w, dx, dw, None, h)
        purlin.layer_norm_grad(y, hx, stats, w, hdx, dw, None, h)
        z = torch.randn(4, 5 * D, generator=g, device=DEV)
        ids, t = torch.arange(8, device=DEV).view(4, 2), torch.zeros(4, 2, device=DEV)
        loss, other, s = torch.empty(4, device=DEV), torch.empty(4, device=DEV), torch.empty(4, 2, device=DEV)
        purlin.distil_loss(z, ids, t, loss, s, h)
        purlin.distil_loss(z.cpu().pin_memory(), ids, t, other, s, h)
        counts, sums, sums2 = torch.empty(D, dtype=torch.int32, device=DEV), torch.empty(2 * D + 1, device=DEV), torch.empty(2 * D + 1, device=DEV)
        picks = torch.zeros(9, 1, dtype=torch.int32, device=DEV)
        purlin.balance_loss(x, picks, counts, sums, None, h)
        purlin.balance_loss(hx, picks, counts, sums2, None, h)
        torch.cuda.synchronize()
        assert torch.equal(hy, y.cpu()) and torch.equal(hdx, dx.cpu()) and torch.equal(loss, other) and torch.equal(sums, sums2)


def test_rows_past_32_bit_offsets(h):  # noqa: F811
    """2.3 Gi elements: the last rows as the first."""
    T, D = 70001, 33000
    x = torch.empty(T, D, dtype=BF16, device=DEV)
    row = torch.randn(3, D, device=DEV).to(BF16)
    for part in x.split(9999):
        part.copy_(row[0])
    x[-2:] = row[1:]
    small = torch.cat([row[:1], row[1:]])
    ids, t = torch.tensor([[5, D - 1]], device=DEV), torch.tensor([[1.0, 0.5]], device=DEV)
    loss, stats = torch.empty(T, device=DEV), torch.empty(T, 2, device=DEV)
    want, s = torch.empty(3, device=DEV), torch.empty(3, 2, device=DEV)
    purlin.distil_loss(x, ids.expand(T, 2).contiguous(), t.expand(T, 2).contiguous(), loss, stats, h)
    purlin.distil_loss(small, ids.expand(3, 2).contiguous(), t.expand(3, 2).contiguous(), want, s, h)
    # the few rows are cut into CTAs, whose sums join in another order
    assert ((loss[-2:] - want[1:]).abs() <= 600 * E24 * want[1:].abs()).all() and (loss[:-2] == loss[0]).all()
    grad = torch.ones(T, device=DEV)
    purlin.distil_loss_grad(x, ids.expand(T, 2).contiguous(), t.expand(T, 2).contiguous(), stats, grad, x, h)
    out = torch.empty_like(small)
    purlin.distil_loss_grad(small, ids.expand(3, 2).contiguous(), t.expand(3, 2).contiguous(), stats[-3:].contiguous(), grad[:3], out, h)
    assert torch.equal(x[-3:], out) and torch.equal(x[0], x[-3])
    del x
    T, D = 300001, 8192
    x = torch.empty(T, D, dtype=BF16, device=DEV)
    for part in x.split(9999):
        part.copy_(row[0, :D])
    x[-2:] = row[1:, :D]
    stats, dw = torch.empty(T, 2, device=DEV), torch.empty(D, device=DEV)
    purlin.layer_norm(x, None, None, x, h, stats=stats)
    y, s3 = torch.empty(3, D, dtype=BF16, device=DEV), torch.empty(3, 2, device=DEV)
    purlin.layer_norm(small[:, :D], None, None, y, h, stats=s3)
    assert torch.equal(x[-2:], y[1:]) and torch.equal(stats[-2:], s3[1:]) and torch.equal(x[0], y[0]) and torch.equal(x[T // 2], y[0])
    purlin.layer_norm_grad(x, x, stats, None, x, None, dw, h)
    want = (T - 2) * y[0].double() + y[1].double() + y[2].double()
    size = (T - 2) * y[0].double().abs() + y[1].double().abs() + y[2].double().abs()
    assert ((dw.double() - want).abs() <= size * (T // 152 + 16 + 152 // 8 + 8 + 1) * E24).all()
    assert torch.equal(x[0], x[T // 2])


def test_threads_and_graphs_on_one_handle(h):  # noqa: F811
    call, want = everything(h)
    call()
    torch.cuda.synchronize()
    jobs, failures = [everything(h) for _ in range(4)], []
    start = threading.Barrier(len(jobs))

    def work(call):
        try:
            start.wait()
            for _ in range(5):
                call()
        except Exception as e:  # told to the main thread
            failures.append(e)
    threads = [threading.Thread(target=work, args=(c,)) for c, _ in jobs]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not failures
    # two graphs, replayed at once on two streams, beside the handle's own blocks
    sides, graphs = [torch.cuda.Stream() for _ in range(2)], []
    more = [everything(h) for _ in sides]
    torch.cuda.synchronize()
    for (call, _), side in zip(more, sides):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            call()
            call()
    for _ in range(3):
        for graph, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                graph.replay()
        jobs[0][0]()
    torch.cuda.synchronize()
    for _, got in jobs + more:
        for name in want:
            assert torch.equal(got[name], want[name]), name
    assert status(h) == (0, 0)


def test_rows_behind_the_last_stay_as_they_were(h):  # noqa: F811
    """Outputs with room for more rows than there are tokens: a slice is written, nothing behind it."""
    x = torch.randn(64, 80, device=DEV)
    y, stats = Guarded(64, 80, F32), Guarded(64, 2, F32)
    purlin.layer_norm(x[:5], None, None, y.view[:5], h, stats=stats.view[:5])
    assert (y.view[5:] == -77).all() and (stats.view[5:] == -77).all() and y.intact() and stats.intact()
    want = O.layer_norm(x[:5].double().cpu().numpy())[0]
    assert np.abs(y.view[:5].double().cpu().numpy() - want).max() < 200 * E24 * 4


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,D", [(20003, 16), (20003, 9), (9729, 128), (2433, 65), (305, 1280), (153, 4096), (3, 5120), (5000, 24),
                                 (300, 8200), (5, 12288), (5, 12296), (8, 8192), (20, 8192), (33, 8192)])
def test_rows_that_share_a_warp_or_do_not_fill_the_last_round(h, T, D, dtype):  # noqa: F811
    """Against torch in 64 bits on the GPU: the lanes of a warp run out of rows at different times."""
    g = torch.Generator(device=DEV).manual_seed(D)
    x, dy, dt = (torch.randn(T, D, generator=g, device=DEV).to(dtype) for _ in range(3))
    w = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
    y, dx = Guarded(T, D, dtype), Guarded(T, D, dtype)
    stats, dw, db = Guarded(T, 2, F32), Guarded(1, D, F32), Guarded(1, D, F32)
    purlin.layer_norm(x, w, w, y.view, h, stats=stats.view)
    purlin.layer_norm_grad(dy, x, stats.view, w, dx.view, dw.view[0], db.view[0], h, grad_total=dt)
    x64, dy64, w64 = x.double(), dy.double(), w.double()
    mean = x64.mean(1, keepdim=True)
    rstd = ((x64 - mean).square().mean(1, keepdim=True) + 1e-5).rsqrt()
    want = (x64 - mean) * rstd * w64 + w64
    u, n = (2.0 ** -8 if dtype is BF16 else E24), 64 + D // 512
    # distances from the mean of values below 6, and their deviation (where it is not small): a few sums of n additions
    tol = u * want.abs() + 8 * n * E24 * (1 + rstd) * (1 + want.abs())
    assert ((y.view.double() - want).abs() <= tol).all()
    mean, rstd = stats.view[:, :1].double(), stats.view[:, 1:].double()
    hat, gw = (x64 - mean) * rstd, dy64 * w64
    want = rstd * (gw - gw.mean(1, keepdim=True) - hat * (gw * hat).mean(1, keepdim=True)) + dt.double()
    size = rstd * (gw.abs() + gw.abs().mean(1, keepdim=True) + hat.abs() * (gw * hat).abs().mean(1, keepdim=True)) + dt.double().abs()
    assert ((dx.view.double() - want).abs() <= u * want.abs() + 2 * n * E24 * size).all()
    n = T // 152 + 64 + 152
    assert ((dw.view[0].double() - (dy64 * hat).sum(0)).abs() <= (n + 4) * E24 * (dy64 * hat).abs().sum(0)).all()
    assert ((db.view[0].double() - dy64.sum(0)).abs() <= n * E24 * dy64.abs().sum(0)).all()
    assert all(t.intact() for t in (y, dx, stats, dw, db))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E", [(3000, 96), (3000, 97), (700, 500), (40000, 8), (513, 1000), (512, 1024)])
def test_balance_of_every_lie_of_the_logits(h, T, E, dtype):  # noqa: F811
    """Against torch in 64 bits: experts in vectors and one by one, tokens for one launch and for two."""
    g = torch.Generator(device=DEV).manual_seed(E)
    x = torch.randn(T, E, generator=g, device=DEV).to(dtype)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(4, 1).indices.to(torch.int32)
    ids[::7] = -1
    counts, sums, loss = torch.empty(E, dtype=torch.int32, device=DEV), torch.empty(2 * E + 1, device=DEV), torch.empty(1, device=DEV)
    grad = Guarded(T, E, dtype)
    purlin.balance_loss(x, ids, counts, sums, loss, h)
    purlin.balance_loss_grad(x, ids, sums, None, grad.view, h)
    live = (ids >= 0).any(1)
    p = torch.softmax(x.double(), 1) * live[:, None]
    want_c = torch.bincount(ids[ids >= 0].long(), minlength=E)
    assert torch.equal(counts.long(), want_c) and sums[2 * E].item() == live.sum().item()
    # a difference of 12 at most, ex2, E in lanes and warps, the reciprocal; then the tokens of a warp, warps and CTAs
    rel = (3 * 12 + 4 + E // 32 + 6 + 3 + T // 2432 + 64) * E24
    assert ((sums[E:2 * E].double() - p.sum(0)).abs() <= rel * p.sum(0)).all()
    of = want_c.double() / want_c.sum()
    want = E * (of * p.sum(0) / live.sum()).sum()
    assert abs(loss.item() - want.item()) <= (rel + 64 * E24) * want.item()
    c = E * of / live.sum()
    dx = p * (c - (p * c).sum(1, keepdim=True))
    u = 2.0 ** -8 if dtype is BF16 else E24
    size = p * (c + (p * c).sum(1, keepdim=True))
    assert ((grad.view.double() - dx).abs() <= u * dx.abs() + (2 * rel + 40 * E24) * size).all() and grad.intact()


def test_one_row_with_a_stride_past_64_bits_of_bytes(h):  # noqa: F811
    """The distance to a row that is not there does not matter, whatever it wraps to."""
    x, res, y, y2, stats = (torch.randn(1, 64, device=DEV) for _ in range(5))
    stats = torch.empty(1, 2, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    purlin.layer_norm(x, None, None, y, h, residual=res)
    huge = 1 << 61
    assert P.purlin_layer_norm(h.raw, x, huge, res, huge, 1, 64, P.PL_F32, None, None, P.PL_F32, 1e-5, y2, huge, None, 0, stats,
                               s) == P.PL_OK
    assert torch.equal(y, y2)
    dx, dx2, dw, dw2 = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device=DEV), torch.empty(64, device=DEV)
    purlin.layer_norm_grad(res, x, stats, None, dx, dw, None, h, grad_total=y)
    ws = torch.empty(P.purlin_layer_norm_grad_bytes(1, 64), dtype=torch.uint8, device=DEV)
    assert P.purlin_layer_norm_grad(h.raw, res, huge, x, huge, stats, 1, 64, P.PL_F32, None, P.PL_F32, y, huge, dx2, huge, dw2, None,
                                    ws, ws.numel(), s) == P.PL_OK
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("D", [520, 1544, 5120, 8192])
def test_rows_of_nan_leave_nothing_for_the_rows_behind_them(h, D):  # noqa: F811
    """Every row is its own: whatever a call before, or the row before, left on the chip."""
    g = torch.Generator(device=DEV).manual_seed(D)
    for dtype in (F32, BF16):
        x = torch.randn(4096, D, generator=g, device=DEV).to(dtype)
        bad = torch.full_like(x, math.nan)
        mixed = x.clone()
        mixed[::2] = math.nan
        y, dx, junk, stats, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(4096, 2, device=DEV), torch.empty(D, device=DEV)
        for _ in range(20):
            purlin.layer_norm(bad, None, None, junk, h, residual=bad)
            purlin.layer_norm(x, None, None, y, h, stats=stats)
            purlin.layer_norm_grad(bad, bad, stats, None, junk, None, None, h, grad_total=bad)
            purlin.layer_norm_grad(x, x, stats, None, dx, dw, None, h)
            assert torch.isfinite(y).all() and torch.isfinite(stats).all() and torch.isfinite(dx).all() and torch.isfinite(dw).all()
            purlin.layer_norm(mixed, None, None, junk, h)
            assert torch.equal(junk[1::2], y[1::2]) and torch.isnan(junk[::2]).all()
            purlin.layer_norm_grad(mixed, mixed, stats, None, junk, None, None, h)
            assert torch.equal(junk[1::2], dx[1::2])
