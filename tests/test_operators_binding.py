"""What the operators' Python binding makes of its arguments (CPU)."""

import numpy as np
import pytest
import torch

from collective_datapath_reduce_gb300 import purlin as P


def test_routing_follows_a_tensor_that_changes_in_place():
    scale, groups = torch.tensor(2.0), torch.tensor(2)
    first = P.make_routing(8, 2, scale=scale, groups=groups)
    assert (first.scale, first.groups) == (2.0, 2)
    scale.mul_(3)
    groups.mul_(2)
    second = P.make_routing(8, 2, scale=scale, groups=groups)
    assert (second.scale, second.groups) == (6.0, 4) and (first.scale, first.groups) == (2.0, 2)


def test_routing_takes_each_kind_of_number():
    want = P.make_routing(64, 4, P.PL_SCORES_SIGMOID, 8, 4, 2, True, 2.0)
    for kind in (int, np.int64, torch.tensor):
        got = P.make_routing(kind(64), kind(4), kind(P.PL_SCORES_SIGMOID), kind(8), kind(4), kind(2), kind(1), kind(2))
        assert bytes(got) == bytes(want)
    assert want.renormalise == 1 and P.make_routing(64, 4, renormalise=False).renormalise == 0


@pytest.mark.parametrize("kw", [dict(groups=2.0), dict(kept_groups="1"), dict(group_best=None), dict(scale="x")])
def test_routing_refuses_what_is_no_such_number(kw):
    with pytest.raises((TypeError, ValueError)):
        P.make_routing(8, 2, **kw)


class Buffer:
    """An object with data_ptr() that is not a tensor's."""

    def __init__(self, address):
        self.address = address

    def data_ptr(self):
        return self.address


@pytest.mark.parametrize("kind", [int, np.int64, np.uint64])
def test_addresses_of_any_kind_of_whole_number(kind):
    at = [Buffer(kind(4096 * (i + 1))) for i in range(2)]
    assert list(P._ptr_array(at)) == [4096, 8192]
    assert P._addr(at[0]) == 4096 and type(P._addr(at[0])) is int
    # on its way to the library, which is told of no handle
    assert P.purlin_all_reduce(None, at, at, 16, P.PL_F32) == P.PL_ERR_INVALID_ARG
    assert P.purlin_atom_copy(None, at[0], at[1:], 16) == P.PL_ERR_INVALID_ARG
