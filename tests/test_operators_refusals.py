"""The operators' torch front end refuses wrong shapes, types and layouts before any library call (CPU)."""

import pytest
import torch

from collective_datapath_reduce_gb300 import purlin as P
from collective_datapath_reduce_gb300 import torch_api as purlin

F, I = torch.float32, torch.int32


@pytest.fixture
def h(monkeypatch):
    """A handle without a library behind it: any call into the library fails
    the test.  Host tensors stand in for the GPU's."""
    def boom(*a, **k):
        raise AssertionError("the library was called")
    for name in P._SIGNATURES:
        if hasattr(P, name):
            monkeypatch.setattr(P, name, boom)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    return purlin.Handle(raw=None, world=2, device=torch.device("cuda", 0))


def z(*shape, dtype=F):
    return torch.zeros(shape, dtype=dtype)


def _bad(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_routing(h):
    _bad("two dimensions", purlin.route_experts, z(8), z(4, 2, dtype=I), z(4, 2), h)
    _bad("float32 or bfloat16", purlin.route_experts, z(4, 8, dtype=torch.float16), z(4, 2, dtype=I), z(4, 2), h)
    _bad("ids must have dtype", purlin.route_experts, z(4, 8), z(4, 2, dtype=torch.int64), z(4, 2), h)
    _bad("ids must have shape", purlin.route_experts, z(4, 8), z(5, 2, dtype=I), z(4, 2), h)
    _bad("weights must have shape", purlin.route_experts, z(4, 8), z(4, 2, dtype=I), z(4, 3), h)
    _bad("bias must have shape", purlin.route_experts, z(4, 8), z(4, 2, dtype=I), z(4, 2), h, bias=z(7))
    _bad("packed rows", purlin.route_experts, z(8, 4).t(), z(4, 2, dtype=I), z(4, 2), h)
    _bad("contiguous", purlin.route_experts, z(4, 8), z(4, 4, dtype=I)[:, :2], z(4, 2), h)
    _bad("grad_logits must have dtype", purlin.route_experts_grad, z(4, 8), z(4, 2, dtype=I), z(4, 2),
         z(4, 8, dtype=torch.bfloat16), h)
    _bad("grad_weights must have shape", purlin.route_experts_grad, z(4, 8), z(4, 2, dtype=I), z(2, 2), z(4, 8), h)


def test_exchange(h):
    p = z(4, 2, dtype=I)
    _bad("experts \\+ 1", purlin.expert_plan, p, z(1, dtype=I), z(4, 2, dtype=I), h)
    _bad("places must have shape", purlin.expert_plan, p, z(9, dtype=I), z(4, 3, dtype=I), h)
    _bad("offsets must have dtype", purlin.expert_plan, p, z(9), z(4, 2, dtype=I), h)
    _bad("rows must be 8 x 16", purlin.dispatch_rows, z(4, 16), p, z(7, 16), h)
    _bad("rows must have dtype", purlin.dispatch_rows, z(4, 16), p, z(8, 16, dtype=torch.bfloat16), h)
    _bad("places must have shape", purlin.dispatch_rows, z(5, 16), p, z(10, 16), h)
    _bad("rows must be 8 x 16", purlin.combine_rows, z(8, 17), p, None, z(4, 16), h)
    _bad("weights must have shape", purlin.combine_rows, z(8, 16), p, z(8), z(4, 16), h)
    _bad("y must be 4 x 16", purlin.combine_rows, z(8, 16), p, None, z(5, 16), h)
    _bad("grad_rows must be 8 x 16", purlin.combine_rows_grad, z(8, 16), p, z(4, 2), z(4, 16), z(8, 15), z(4, 2), h)
    _bad("grad_weights must have dtype", purlin.combine_rows_grad, z(8, 16), p, z(4, 2), z(4, 16), z(8, 16), p, h)


def test_embedding(h):
    _bad("int32 or int64", purlin.embed, z(8, 16), z(4), z(4, 16), h)
    _bad("out must be 4 x 16", purlin.embed, z(8, 16), z(4, dtype=I), z(4, 15), h)
    _bad("out must have dtype", purlin.embed, z(8, 16), z(4, dtype=I), z(4, 16, dtype=torch.bfloat16), h)
    _bad("contiguous", purlin.embed, z(8, 16), z(8, dtype=I)[::2], z(4, 16), h)
    _bad("grad_out must be 4 x 16", purlin.embed_grad, z(4, 8), z(4, dtype=I), z(8, 16), h)
    _bad("base must have dtype", purlin.embed_grad, z(4, 16), z(4, dtype=I), z(8, 16), h, base=z(8, 16, dtype=torch.bfloat16))


def test_clip(h):
    _bad("norm must have shape", purlin.clip_grad_norm, [z(4)], None, 1.0, z(2), h)
    _bad("expected 1 outputs", purlin.clip_grad_norm, [z(4)], [], 1.0, z(1), h)
    _bad("one dtype", purlin.clip_grad_norm, [z(4), z(4, dtype=torch.bfloat16)], None, 1.0, z(1), h)
    _bad("gradient's size", purlin.clip_grad_norm, [z(4)], [z(5)], 1.0, z(1), h)
    _bad("contiguous", purlin.clip_grad_norm, [z(4, 4).t()], None, 1.0, z(1), h)


def test_host_tensors_that_are_not_pinned():
    h = purlin.Handle(raw=None, world=2, device=torch.device("cuda", 0))
    _bad("pinned", purlin.embed, z(8, 16), z(4, dtype=I), z(4, 16), h)
    _bad("pinned", purlin.clip_grad_norm, [z(4)], None, 1.0, z(1), h)


def test_null_handles_and_sizes_without_a_gpu():
    lib = P.load()
    assert lib.purlin_embed(None, None, 0, 0, 0, None, 4, 0, 0, 1.0, P.PL_F32, None, 0, None) == P.PL_ERR_INVALID_ARG
    assert lib.purlin_dispatch_rows(None, None, 0, None, 0, 1, 0, P.PL_F32, None, 0, None) == P.PL_ERR_INVALID_ARG
    assert P.purlin_expert_plan_bytes(16, 8, 256) == 0                  # one CTA needs no counts
    assert P.purlin_expert_plan_bytes(16384, 8, 256) > 0
    assert P.purlin_expert_plan_bytes(16384, 33, 256) == 0              # refused by the call
    assert P.purlin_embed_grad_bytes(100, 1000, 64) < P.purlin_embed_grad_bytes(100000, 1000, 64)
    assert P.purlin_clip_grad_norm_bytes() >= 8
