"""The distilling training step against the same model in 64 bits with torch's autograd."""

import pytest
import torch

from collective_datapath_reduce_gb300 import distil_step

pytestmark = pytest.mark.gpu


def reference(model, tokens, words, teacher):
    """Loss, picks and gradients of one step, without ranks, in float64."""
    s = model.shape
    params = [p.detach().double().cpu().requires_grad_() for p in model.parameters()]
    W = s.world
    table, router = torch.cat(params[:W]), params[W]
    up, down = torch.cat(params[W + 1:2 * W + 1]), torch.cat(params[2 * W + 1:3 * W + 1])
    norms = params[3 * W + 1:]

    def norm(x, w, b):
        mean = x.mean(1, keepdim=True)
        return (x - mean) / ((x - mean).square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b
    x = table[torch.cat(tokens).cpu()] * s.scale
    n = norm(x, *norms[:2])
    p = torch.softmax(n @ router.t(), 1)
    ids = p.sort(dim=1, descending=True, stable=True).indices[:, :s.top_k]
    w = p.gather(1, ids)
    w = w / (w.sum(1, keepdim=True) + 1e-20)
    every = torch.einsum("teh,ehd->ted", torch.relu(torch.einsum("td,edh->teh", n, up)), down)
    y = (every.gather(1, ids[:, :, None].expand(-1, -1, s.width)) * w[:, :, None]).sum(1)
    picks = torch.bincount(ids.flatten(), minlength=s.experts).double()
    balance = s.balance * s.experts * (picks / picks.sum() * p.mean(0)).sum()
    z = norm(x + y, *norms[2:]) @ table.t()
    q = torch.softmax(torch.cat(teacher).double().cpu() / s.temperature, 1)
    log_p = torch.log_softmax(z / s.temperature, 1).gather(1, torch.cat(words).cpu())
    loss = s.temperature ** 2 * (q * (q.log() - log_p)).sum(1).mean() + balance
    loss.backward()
    return loss.item(), ids, [v.grad for v in params]


@pytest.mark.parametrize("shape,picks", [
    (distil_step.Shape(world=4, tokens=37, vocabulary=64, width=64, hidden=96, experts=8, top_k=3, max_norm=1e9), 5),
    (distil_step.Shape(world=2, tokens=1, vocabulary=2, width=8, hidden=8, experts=2, top_k=1, max_norm=1e9), 1),
    (distil_step.Shape(world=8, tokens=50, vocabulary=256, width=128, hidden=64, experts=64, top_k=6, max_norm=0.01,
                       balance=2.0), 16),
], ids=str)
def test_step_matches_autograd(shape, picks):
    model = distil_step.DistilStep(shape, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    W, T, V = shape.world, shape.tokens, shape.vocabulary
    tokens = [torch.randint(0, V, (T,), generator=g, device="cuda") for _ in range(W)]
    words = [torch.rand(T, V, generator=g, device="cuda").topk(picks, 1).indices for _ in range(W)]
    teacher = [torch.randn(T, picks, generator=g, device="cuda") for _ in range(W)]
    want_loss, want_ids, want = reference(model, tokens, words, teacher)
    loss, saved = model.forward(tokens, words, teacher)
    assert torch.equal(torch.cat(saved["ids"]).cpu().long(), want_ids)
    before = [p.clone() for p in model.parameters()]
    loss, norm = model.step(tokens, words, teacher)
    # ten products, norms and softmaxes in a row, of sums of at most 256 terms, in binary32: 10 x 256 x 2^-24 of the
    # sums of the terms' sizes, which exceed the sums by about the root of 256
    bound = 10 * 256 * 2.0 ** -24 * 256 ** 0.5
    assert abs(loss.item() - want_loss) <= bound * abs(want_loss)
    want_norm = float(sum((q ** 2).sum() for q in want)) ** 0.5
    assert abs(norm.item() - want_norm) <= bound * want_norm
    factor = min(1.0, shape.max_norm / (want_norm + 1e-6))
    for p, b, q in zip(model.parameters(), before, want):
        moved = (b - p).double().cpu() / shape.rate
        # the update p - rate x g rounds p once
        rounding = 2.0 ** -24 * b.double().cpu().norm() / shape.rate
        assert (moved - factor * q).norm() <= 2 * bound * factor * want_norm + rounding
    model.close()


def test_the_command_runs(capsys):
    distil_step.main()
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 10 and all("nan" not in line for line in lines)
