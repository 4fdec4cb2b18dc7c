"""Which block of memory an operator's call works in: by its own stream, whatever stream is current (CPU)."""

import contextlib
import threading
import time
import types

import pytest
import torch

from collective_datapath_reduce_gb300 import torch_api as purlin


class Cuda:
    """torch.cuda's streams without a GPU: a current stream, and those that a graph captures."""

    def __init__(self):
        self.current, self.capturing, self.blocks = 1, set(), []

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s.cuda_stream
        yield
        self.current = before

    def empty(self, nbytes, dtype, device):
        block = real_empty(nbytes, dtype=dtype)
        self.blocks.append((block, self.current))
        return block

    def allocated_on(self, block):
        return next(s for b, s in self.blocks if b is block)


real_empty = torch.empty


@pytest.fixture
def cuda(monkeypatch):
    c = Cuda()
    monkeypatch.setattr(torch.cuda, "stream", c.stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device=None: types.SimpleNamespace(cuda_stream=raw))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: c.current in c.capturing)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: c.current, raising=False)
    monkeypatch.setattr(torch, "empty", c.empty)
    return c


@pytest.fixture
def h():
    return purlin.Handle(raw=None, world=2, device=torch.device("cuda", 0))


@pytest.mark.parametrize("current", [1, 2])
@pytest.mark.parametrize("form", [int, "object"])
def test_a_call_on_a_captured_stream_gets_a_block_of_that_stream_and_nothing_is_kept(cuda, h, current, form):
    stream = 2 if form is int else types.SimpleNamespace(cuda_stream=2)
    cuda.current, cuda.capturing = current, {1, 2}
    block = purlin._workspace(100, stream, h)
    assert block.numel() >= 100 and cuda.allocated_on(block) == 2 and not h.workspaces
    assert purlin._workspace(100, stream, h) is not block and cuda.current == current


def test_the_calls_own_stream_decides_about_the_capture(cuda, h):
    kept = purlin._workspace(100, 2, h)
    assert cuda.allocated_on(kept) == 2 and purlin._workspace(50, 2, h) is kept
    cuda.capturing = {2}
    assert purlin._workspace(100, 2, h) is not kept          # current: 1, not captured
    cuda.capturing = {1}
    assert purlin._workspace(100, 2, h) is kept              # current: 1, captured
    own = purlin._workspace(100, None, h)
    assert cuda.allocated_on(own) == 1 and own is not kept and purlin._workspace(100, None, h) is not own


def test_one_block_for_each_stream_that_grows(cuda, h):
    assert purlin._workspace(0, None, h) is None
    a, b = purlin._workspace(100, None, h), purlin._workspace(100, 2, h)
    assert a is not b and purlin._workspace(100, 1, h) is a
    c = purlin._workspace(101, 1, h)
    assert c is not a and cuda.allocated_on(c) == 1 and purlin._workspace(100, None, h) is c
    assert purlin._workspace(100, 2, h) is b


def test_threads_on_one_stream_do_not_share_a_block_in_the_middle_of_a_call(cuda, h, monkeypatch):
    """A call is several launches: another thread's between them may not use the same block."""
    busy, clashes, calls = set(), [], []

    def plan(raw, ids, tokens, top_k, experts, offsets, places, ws, nbytes, stream):
        if id(ws) in busy:
            clashes.append(threading.get_ident())
        busy.add(id(ws))
        time.sleep(0.02)                  # as the library does, without the interpreter's lock
        busy.discard(id(ws))
        calls.append(stream)
        return 0

    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(purlin.P, "purlin_expert_plan_bytes", lambda *a: 64)
    monkeypatch.setattr(purlin.P, "purlin_expert_plan", plan)
    ids, offsets, places = (torch.zeros(s, dtype=torch.int32) for s in ((8, 2), 5, (8, 2)))
    start = threading.Barrier(4)

    def work():
        start.wait()
        for _ in range(3):
            purlin.expert_plan(ids, offsets, places, h)
    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(calls) == 12 and not clashes
