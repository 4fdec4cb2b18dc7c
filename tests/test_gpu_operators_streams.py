"""Operators with workspaces on streams that the caller names, captured and eager, against the same calls in order."""

import threading

import pytest
import torch

from collective_datapath_reduce_gb300 import torch_api as purlin
from test_gpu_operators import DEV, h  # noqa: F401 (h: a fixture)

pytestmark = pytest.mark.gpu


class Job:
    """An embedding gradient, a plan and a clip of one size, each with a workspace."""

    def __init__(self, n, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.tokens = (torch.rand(n, generator=g, device=DEV) ** 4 * 3000).to(torch.int64)
        self.dy = torch.randn(n, 128, generator=g, device=DEV)
        self.ids = torch.randint(0, 64, (n, 4), generator=g, device=DEV, dtype=torch.int32)
        self.out = dict(grad=torch.zeros(3000, 128, device=DEV), offsets=torch.zeros(65, dtype=torch.int32, device=DEV),
                        places=torch.zeros(n, 4, dtype=torch.int32, device=DEV), clipped=torch.zeros_like(self.dy),
                        norm=torch.zeros(1, device=DEV))

    def run(self, h, stream=None):
        o = self.out
        purlin.embed_grad(self.dy, self.tokens, o["grad"], h, stream=stream)
        purlin.expert_plan(self.ids, o["offsets"], o["places"], h, stream=stream)
        purlin.clip_grad_norm([self.dy], [o["clipped"]], 1.0, o["norm"], h, stream=stream)

    def taken(self):
        """The outputs, which are cleared for the next run."""
        torch.cuda.synchronize()
        got = {name: t.clone() for name, t in self.out.items()}
        for t in self.out.values():
            t.zero_()
        torch.cuda.synchronize()
        return got


def same(a, b):
    for name in a:
        assert torch.equal(a[name], b[name]), name


def test_branches_of_a_graph_on_named_streams(h):
    jobs = [Job(n, n) for n in (30000, 50000, 40000)]
    wants = []
    for j in jobs:
        j.run(h)
        wants.append(j.taken())
    main, sides = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        for s in sides:
            s.wait_stream(main)
        for _ in range(2):
            for j, s in zip(jobs, (sides[0], sides[1].cuda_stream, None)):
                j.run(h, s)
        for s in sides:
            main.wait_stream(s)
    later = Job(90000, 4)
    later.run(h)              # blocks that the handle keeps grow; the graph has its own
    for _ in range(3):
        graph.replay()
        for j, want in zip(jobs, wants):
            same(j.taken(), want)


def test_a_captured_stream_that_is_not_current(h):
    job = Job(30000, 5)
    side = torch.cuda.Stream()
    job.run(h, side)
    want = job.taken()
    graph = torch.cuda.CUDAGraph()
    main = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(main):         # not captured
            job.run(h, side)
    Job(90000, 6).run(h, side)                # on the handle's block for that stream
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
        same(job.taken(), want)


def test_threads_on_one_stream(h):
    jobs = [Job(n, n) for n in (30000, 50000, 40000, 60000)]
    wants = []
    for j in jobs:
        j.run(h)
        wants.append(j.taken())
    start, failures = threading.Barrier(len(jobs)), []

    def work(job):
        try:
            start.wait()
            for _ in range(10):
                job.run(h)
        except Exception as e:  # told to the main thread
            failures.append(e)
    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failures
    torch.cuda.synchronize()
    got = [j.taken() for j in jobs]
    for g, want in zip(got, wants):
        same(g, want)
