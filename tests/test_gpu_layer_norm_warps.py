"""Layer norm and its gradient at the widths whose ring of three matrices holds fewer groups of threads than a block."""

import pytest
import torch

import test_gpu_row_operators_edges as edges
from test_gpu_operators import h  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


# 8 threads a row and 16, few rows (the sums join in one cluster) and many
@pytest.mark.parametrize("D", [136, 144, 160, 268, 292, 316])
@pytest.mark.parametrize("T", [1, 5, 53, 1700, 20003])
def test_blocks_of_whole_warps(h, T, D):  # noqa: F811
    edges.test_rows_that_share_a_warp_or_do_not_fill_the_last_round(h, T, D, torch.float32)
