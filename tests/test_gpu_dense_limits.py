"""The full-attention layer's calls at the edges of their ranges."""
import importlib.util
import os
import threading

import pytest
import torch

from block_sparse_attention_07_gb300 import msa

from test_gpu_build_step import Step

pytestmark = pytest.mark.gpu


def test_step_metadata_from_several_host_threads():
    """Batches of different sizes built by threads of one process, each on its own stream and buffers."""
    sizes = (4096, 2100, 3000, 2600)
    steps = [Step([5] * B, [1] * B, NB=2, seed=B) for B in sizes]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    calls = [s.run(stream=st, prepare=True) for s, st in zip(steps, streams)]
    failed, start = [], threading.Barrier(len(sizes))

    def work(i):
        start.wait()
        try:
            for _ in range(4000):
                calls[i]()
        except msa.MSAError as e:
            failed.append((sizes[i], str(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for s in steps:
        s.check()


def test_measured_calls_follow_the_current_stream(monkeypatch):
    """A pass of perf/operators.py under another stream than the first one's, and captured on its stream, is ordered with
    that stream's work."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("measured_operators", path)
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    ops.own = True
    case = ops._gqa("small", 3, 100, 900, kv="fp8")
    s = ops.prepare(case, 1)
    out, lse = (t.clone() for t in ops.run(s))
    torch.cuda.synchronize()
    q = s["q"].clone()

    def late(fn):
        s["q"].zero_()
        s["out"].zero_()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)                  # the queries arrive some 10 ms later, on this stream
        s["q"].copy_(q)
        fn()

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        late(lambda: ops.run(s))
    side.synchronize()
    assert torch.equal(s["out"], out) and torch.equal(s["lse"], lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ops.run(s)
    with torch.cuda.stream(side):
        late(graph.replay)
    side.synchronize()
    assert torch.equal(s["out"], out) and torch.equal(s["lse"], lse) and int(s["flags"].item()) == 0
