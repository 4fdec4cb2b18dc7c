"""Layer norm, balance and distillation refuse wrong shapes, types and layouts before any library call (CPU)."""

import pytest
import torch

from collective_datapath_reduce_gb300 import purlin as P
from collective_datapath_reduce_gb300 import torch_api as purlin
from test_operators_refusals import _bad, h, z  # noqa: F401 (h: a fixture)

B, F, I, L = torch.bfloat16, torch.float32, torch.int32, torch.int64


def test_layer_norm(h):  # noqa: F811
    x, w = z(4, 16), z(16)
    _bad("two dimensions", purlin.layer_norm, z(16), w, w, z(16), h)
    _bad("float32 or bfloat16", purlin.layer_norm, z(4, 16, dtype=torch.float16), w, w, x, h)
    _bad("y must be 4 x 16", purlin.layer_norm, x, w, w, z(4, 15), h)
    _bad("y must have dtype", purlin.layer_norm, x, w, w, z(4, 16, dtype=B), h)
    _bad("packed rows", purlin.layer_norm, z(16, 4).t(), w, w, x, h)
    _bad("weight must have shape", purlin.layer_norm, x, z(15), w, z(4, 16), h)
    _bad("weight must have shape", purlin.layer_norm, x, z(1, 16), w, z(4, 16), h)
    _bad("bias must have dtype", purlin.layer_norm, x, w, z(16, dtype=B), z(4, 16), h)
    _bad("float32 or bfloat16", purlin.layer_norm, x, z(16, dtype=torch.float64), None, z(4, 16), h)
    _bad("bias must be contiguous", purlin.layer_norm, x, w, z(32)[::2], z(4, 16), h)
    _bad("residual must have dtype", purlin.layer_norm, x, w, w, z(4, 16), h, residual=z(4, 16, dtype=B))
    _bad("total must be 4 x 16", purlin.layer_norm, x, w, w, z(4, 16), h, total=z(5, 16))
    _bad("stats must have shape", purlin.layer_norm, x, w, w, z(4, 16), h, stats=z(4))
    _bad("stats must have dtype", purlin.layer_norm, x, w, w, z(4, 16), h, stats=z(4, 2, dtype=B))
    g = (z(4, 16), z(4, 16), z(4, 2), w, z(4, 16), z(16), z(16))
    for i, bad, match in ((1, z(4, 15), "x must be 4 x 16"), (2, z(4, 1), "stats must have shape"), (3, z(8), "weight must have"),
                          (4, z(4, 16, dtype=B), "grad_x must have dtype"), (5, z(16, dtype=B), "grad_weight must have dtype"),
                          (6, z(17), "grad_bias must have shape")):
        _bad(match, purlin.layer_norm_grad, *g[:i], bad, *g[i + 1:], h)
    _bad("grad_total must be 4 x 16", purlin.layer_norm_grad, *g, h, grad_total=z(3, 16))


def test_balance(h):  # noqa: F811
    good = (z(4, 8), z(4, 2, dtype=I), z(8, dtype=I), z(17), z(1))
    for i, bad, match in ((0, z(8), "two dimensions"), (0, z(4, 8, dtype=torch.float16), "float32 or bfloat16"),
                          (1, z(4, 2), "ids must have dtype"), (1, z(3, 2, dtype=I), "ids must have shape"),
                          (2, z(8), "counts must have dtype"), (2, z(9, dtype=I), "counts must have shape"),
                          (3, z(16), "sums must have shape"), (3, z(17, dtype=B), "sums must have dtype"),
                          (4, z(2), "loss must have shape")):
        _bad(match, purlin.balance_loss, *good[:i], bad, *good[i + 1:], h)
    _bad("2 x experts \\+ 1", purlin.balance_join, z(16), z(1), h)
    _bad("2 x experts \\+ 1", purlin.balance_join, z(1), z(1), h)
    _bad("loss must have dtype", purlin.balance_join, z(17), z(1, dtype=B), h)
    grad = (z(4, 8), z(4, 2, dtype=I), z(17), z(1), z(4, 8))
    for i, bad, match in ((2, z(15), "sums must have shape"), (3, z(4), "grad_loss must have shape"),
                          (4, z(4, 8, dtype=B), "grad_logits must have dtype")):
        _bad(match, purlin.balance_loss_grad, *grad[:i], bad, *grad[i + 1:], h)
    _bad("base must be 4 x 8", purlin.balance_loss_grad, *grad, h, base=z(4, 9))


def test_distillation(h):  # noqa: F811
    good = (z(4, 8), z(4, 2, dtype=I), z(4, 2))
    out = (z(4), z(4, 2))
    for i, bad, match in ((0, z(8), "two dimensions"), (0, z(4, 8, dtype=torch.float16), "float32 or bfloat16"),
                          (1, z(4, 2), "int32 or int64"), (1, z(5, 2, dtype=L), "ids must have shape"),
                          (2, z(4, 3), "teacher must have shape"), (2, z(4, 2, dtype=torch.float16), "float32 or bfloat16")):
        for fn, rest in ((purlin.distil_loss, out), (purlin.distil_parts, (z(4, 4),)),
                         (purlin.distil_loss_grad, (z(4, 2), z(4), z(4, 8)))):
            _bad(match, fn, *good[:i], bad, *good[i + 1:], *rest, h)
    _bad("loss must have shape", purlin.distil_loss, *good, z(5), out[1], h)
    _bad("stats must have dtype", purlin.distil_loss, *good, out[0], z(4, 2, dtype=B), h)
    _bad("parts must have shape", purlin.distil_parts, *good, z(4, 3), h)
    _bad("ranges x 4 x 4", purlin.distil_join, z(3, 4), *out, h)
    _bad("ranges x 4 x 4", purlin.distil_join, z(2, 4, 3), *out, h)
    _bad("ranges x 4 x 4", purlin.distil_join, z(0, 4, 4), *out, h)
    _bad("grad_loss must have shape", purlin.distil_loss_grad, *good, z(4, 2), z(4, 1), z(4, 8), h)
    _bad("grad_logits must be 4 x 8", purlin.distil_loss_grad, *good, z(4, 2), z(4), z(4, 9), h)


def test_null_handles_and_workspaces_without_a_gpu():
    d = P.make_distillation(8, 0, 8, 2, 4, P.PL_F32)
    assert P.purlin_layer_norm(None, None, 0, None, 0, 0, 0, P.PL_F32, None, None, P.PL_F32, 1e-5, None, 0, None, 0,
                               None) == P.PL_ERR_INVALID_ARG
    assert P.purlin_balance_join(None, None, 4, 1.0, None) == P.PL_ERR_INVALID_ARG
    assert P.purlin_distil_loss(None, None, 8, P.PL_F32, 0, d, None, None, None, None) == P.PL_ERR_INVALID_ARG
    assert P.purlin_layer_norm_grad_bytes(100000, 4096) >= 2 * 4096 * 4
    assert P.purlin_layer_norm_grad_bytes(0, 4096) == 0
    assert P.purlin_balance_loss_bytes(1, 64) == 0 and P.purlin_balance_loss_bytes(100000, 64) > 0
    assert P.purlin_balance_loss_bytes(100000, 1025) == 0                # refused by the call
    assert P.make_distillation(8, 0, 8, 2, 4, P.PL_F32) is d             # one struct for all such calls
    with pytest.raises(TypeError):
        P.make_distillation(8, 0.5, 8, 2, 4, P.PL_F32)
