"""The expert-parallel training step against the same model in 64 bits with torch's autograd."""

import pytest
import torch

from collective_datapath_reduce_gb300 import expert_step

pytestmark = pytest.mark.gpu


def reference(model, tokens, targets):
    """Loss, picks and gradients of one step, without ranks, in float64."""
    s = model.shape
    params = [p.detach().double().cpu().requires_grad_() for p in model.parameters()]
    W = s.world
    table, router = torch.cat(params[:W]), params[W]
    up, down = torch.cat(params[W + 1:2 * W + 1]), torch.cat(params[2 * W + 1:])
    x = table[torch.cat(tokens).cpu()] * s.scale
    p = torch.softmax(x @ router.t(), 1)
    ids = p.sort(dim=1, descending=True, stable=True).indices[:, :s.top_k]
    w = p.gather(1, ids)
    w = w / (w.sum(1, keepdim=True) + 1e-20)
    every = torch.einsum("teh,ehd->ted", torch.relu(torch.einsum("td,edh->teh", x, up)), down)
    y = (every.gather(1, ids[:, :, None].expand(-1, -1, s.width)) * w[:, :, None]).sum(1)
    loss = ((y - torch.cat(targets).double().cpu()) ** 2).sum() / (2 * y.shape[0])
    loss.backward()
    return loss.item(), ids, [q.grad for q in params]


@pytest.mark.parametrize("shape", [
    expert_step.Shape(world=4, tokens=37, vocabulary=64, width=64, hidden=96, experts=8, top_k=3, max_norm=1e9),
    expert_step.Shape(world=2, tokens=1, vocabulary=2, width=8, hidden=8, experts=2, top_k=1, max_norm=1e9),
    expert_step.Shape(world=8, tokens=130, vocabulary=4096, width=128, hidden=64, experts=64, top_k=6, max_norm=0.01),
], ids=str)
def test_step_matches_autograd(shape):
    model = expert_step.ExpertStep(shape, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    tokens = [torch.randint(0, shape.vocabulary, (shape.tokens,), generator=g, device="cuda") for _ in range(shape.world)]
    targets = [torch.randn(shape.tokens, shape.width, generator=g, device="cuda") for _ in range(shape.world)]
    want_loss, want_ids, want = reference(model, tokens, targets)
    y, saved = model.forward(tokens)
    assert torch.equal(torch.cat(saved["ids"]).cpu().long(), want_ids)
    before = [p.clone() for p in model.parameters()]
    loss, norm = model.step(tokens, targets)
    # five products in a row of at most 128 terms each, in binary32: 5 x 128 x 2^-24
    # of the sums of the terms' sizes, which exceed the sums by about the root of 128
    bound = 5 * 128 * 2.0 ** -24 * 128 ** 0.5
    assert abs(loss.item() - want_loss) <= bound * want_loss
    want_norm = float(sum((q ** 2).sum() for q in want)) ** 0.5
    assert abs(norm.item() - want_norm) <= bound * want_norm
    factor = min(1.0, shape.max_norm / (want_norm + 1e-6))
    for p, b, q in zip(model.parameters(), before, want):
        moved = (b - p).double().cpu() / shape.rate
        # the update p - rate x g rounds p once
        rounding = 2.0 ** -24 * b.double().cpu().norm() / shape.rate
        assert (moved - factor * q).norm() <= 2 * bound * factor * q.norm() + rounding
    model.close()


def test_steps_reduce_the_loss():
    shape = expert_step.Shape(world=4, tokens=64, vocabulary=512, width=64, hidden=128, experts=8, top_k=2, rate=0.2)
    model = expert_step.ExpertStep(shape)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = [torch.randint(0, shape.vocabulary, (shape.tokens,), generator=g, device="cuda") for _ in range(4)]
    targets = [torch.randn(shape.tokens, shape.width, generator=g, device="cuda") for _ in range(4)]
    losses = [model.step(tokens, targets)[0].item() for _ in range(30)]
    assert losses[-1] < losses[0] and all(l == l for l in losses)
    model.close()
