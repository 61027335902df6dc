"""msa_add_norm_quant from several host threads at one time, each on a stream of its own."""
import threading

import pytest
import torch

from block_sparse_attention_07_gb300 import msa

pytestmark = pytest.mark.gpu


def test_widths_with_rings_of_unequal_size():
    """Calls whose copies ahead take unequal amounts of shared memory: none is refused for another's sake."""
    failed, done = [], []

    def work(width):
        try:
            T = 2 ** 23 // width + 9
            gen = torch.Generator(device="cuda")
            gen.manual_seed(width)
            x, r = (torch.randn((T, width), generator=gen, device="cuda").bfloat16() for _ in range(2))
            out, w, stream = torch.empty_like(x), torch.ones(width, device="cuda"), torch.cuda.Stream()
            torch.cuda.synchronize()
            call = msa.add_norm_quant(x, w, residual=r, out=out, stream=stream, prepare=True)
            for i in range(6000):
                call()
                if i % 500 == 0:
                    stream.synchronize()
            stream.synchronize()
            assert "ring" in msa.last_dispatch()
            first = out.clone()
            call()
            stream.synchronize()
            done.append(torch.equal(first, out))
        except Exception as e:      # noqa: BLE001 (reported by the main thread)
            failed.append((width, repr(e)))

    threads = [threading.Thread(target=work, args=(n,)) for n in (4352, 5120, 6144, 8192)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and done == [True] * 4, failed
