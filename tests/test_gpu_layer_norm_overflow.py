"""Layer norm of rows whose squares, or whose sums, pass binary32's range."""

import math

import pytest
import torch

from collective_datapath_reduce_gb300 import torch_api as purlin
from test_gpu_operators import DEV, DTYPES, h  # noqa: F401 (h: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [2, 64, 65, 520, 4096, 4097, 8200, 12296])
def test_rows_whose_squares_overflow_are_the_bias(h, D, dtype):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(D)
    x = torch.randn(5, D, generator=g, device=DEV).to(dtype)
    x[1] = 1e25                             # distances of 1e25 from a mean of about 0, whose squares are 1e50
    x[1, ::2] = -1e25
    x[3] = torch.finfo(dtype).min           # two such values add up to -inf
    w, b = torch.randn(D, generator=g, device=DEV), torch.randn(D, generator=g, device=DEV)
    y, plain, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(5, 2, device=DEV)
    purlin.layer_norm(x, w, b, y, h, stats=stats)
    purlin.layer_norm(x, w, None, plain, h)
    assert torch.equal(y[1], b.to(dtype)) and (plain[1] == 0).all()
    assert math.isfinite(stats[1, 0].item()) and stats[1, 1].item() == 0
    assert torch.isnan(y[3]).all() and torch.isnan(plain[3]).all() and stats[3, 0].item() == -math.inf
    for t in (0, 2, 4):                     # the rows beside them
        assert torch.isfinite(y[t]).all() and torch.isfinite(stats[t]).all()
