"""A step's backward pass, asked for twice."""

import pytest
import torch

from collective_datapath_reduce_gb300 import distil_step, expert_step

pytestmark = pytest.mark.gpu


def test_distilling_step():
    """Its logits become gradients in place, so there is no second time."""
    shape = distil_step.Shape(world=2, tokens=9, vocabulary=32, width=16, hidden=24, experts=4, top_k=2)
    model = distil_step.DistilStep(shape, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    tokens = [torch.randint(0, 32, (9,), generator=g, device="cuda") for _ in range(2)]
    words = [torch.rand(9, 32, generator=g, device="cuda").topk(5, 1).indices for _ in range(2)]
    teacher = [torch.randn(9, 5, generator=g, device="cuda") for _ in range(2)]
    _, saved = model.forward(tokens, words, teacher)
    _, again = model.forward(tokens, words, teacher)
    grads = model.backward(saved)
    with pytest.raises(RuntimeError, match="forward"):
        model.backward(saved)
    for a, b in zip(grads, model.backward(again), strict=True):
        assert torch.equal(a, b)
    model.close()


def test_expert_step():
    shape = expert_step.Shape(world=2, tokens=9, vocabulary=32, width=16, hidden=24, experts=4, top_k=2)
    model = expert_step.ExpertStep(shape, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    tokens = [torch.randint(0, 32, (9,), generator=g, device="cuda") for _ in range(2)]
    y, saved = model.forward(tokens)
    grad_y = [torch.randn(t.shape, generator=g, device="cuda") for t in y]
    for a, b in zip(model.backward(grad_y, saved), model.backward(grad_y, saved), strict=True):
        assert torch.equal(a, b)
    model.close()
