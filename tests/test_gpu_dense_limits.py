"""The full-attention layer's calls at the edges of their ranges."""
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
