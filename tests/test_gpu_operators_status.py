"""What an operator finds wrong on the device is its own: the collectives of the handle go on."""

import pytest
import torch

from collective_datapath_reduce_gb300 import purlin as P
from collective_datapath_reduce_gb300 import torch_api as purlin

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def bad_dispatch(h, x, rows):
    purlin.dispatch_rows(x, torch.tensor([[0, 4], [-9, 1]], dtype=torch.int32, device=DEV), rows, h)


def report(h):
    st, dev = P.purlin_status_get(h.raw, torch.cuda.current_stream().cuda_stream)
    assert st == P.PL_OK
    return dev


@pytest.mark.parametrize("layout", [P.PL_LAYOUT_ONE_SHOT, P.PL_LAYOUT_TWO_SHOT, P.PL_LAYOUT_RING])
def test_a_bad_place_does_not_stop_the_collectives(layout):
    h = purlin.initialize(4, DEV)
    n = 1 << 16
    xs = [torch.arange(n, device=DEV, dtype=torch.float32) % 257 + r for r in range(4)]
    outs = [torch.full_like(x, -7.0) for x in xs]
    x, rows = torch.ones(2, 16, device=DEV), torch.empty(4, 16, device=DEV)
    P.check(P.purlin_tune_override(h.raw, {"layout": layout}))
    bad_dispatch(h, x, rows)
    purlin.all_reduce(xs, outs, h)
    want = xs[0] + xs[1] + xs[2] + xs[3]           # whole numbers: exact
    for o in outs:
        assert torch.equal(o, want)
    assert report(h) == P.PL_ERR_BOUNDS and report(h) == P.PL_OK
    purlin.finalize(h)


def test_finalize_reports_a_bad_place():
    h = purlin.initialize(2, DEV)
    bad_dispatch(h, torch.ones(2, 16, device=DEV), torch.empty(4, 16, device=DEV))
    with pytest.raises(P.PurlinError) as e:
        purlin.finalize(h)
    assert e.value.status == P.PL_ERR_BOUNDS


def test_a_captured_operator_outlives_a_grown_workspace():
    """The collectives' workspace moves when it grows; what a graph's operators report still arrives."""
    h = purlin.initialize(16, DEV)
    x, rows = torch.ones(2, 16, device=DEV), torch.empty(4, 16, device=DEV)
    places = torch.tensor([[0, 4], [-9, 1]], dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        purlin.dispatch_rows(x, places, rows, h)
    # ring tiles of 1 KiB: more flags than the default workspace holds
    xs = [torch.full((40 << 20,), r, dtype=torch.bfloat16, device=DEV) for r in range(16)]
    P.check(P.purlin_tune_override(h.raw, {"layout": P.PL_LAYOUT_RING, "chunk_bytes": 1024}))
    purlin.all_reduce(xs, xs, h)
    assert P.purlin_workspace_query(h.raw)[2] == 1 and report(h) == P.PL_OK
    assert all((t == 120).all() for t in xs)
    graph.replay()
    assert report(h) == P.PL_ERR_BOUNDS and report(h) == P.PL_OK
    assert (rows[:2] == 1).all()
    purlin.finalize(h)
