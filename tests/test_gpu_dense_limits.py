"""The full-attention layer's calls at the edges of their ranges."""
import importlib.util
import os
import threading

import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa, synth
from oracle import quant as Qz

from paged import FP4_G, FP8_S, Case
from test_gpu_build_step import Step
from test_gpu_mrope import Rope, _bits

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


@pytest.mark.parametrize("T", [3000, 10000])
@pytest.mark.parametrize("kv,idx", [("bf16", None), ("fp8", "fp8"), ("nvfp4", "nvfp4"), ("nvfp4", "fp8")])
def test_rotary_of_long_batches(T, kv, idx):
    """Two warps per token (3,000) and one (10,000), with the index branch, against fp64; caches byte for byte. One KV
    head: what chooses the warps is the number of tokens."""
    ref = Rope(T, 1, 8, seed=13)
    ref.run()
    assert f"warps_per_token={1 if T == 10000 else 2} " in msa.last_dispatch()
    ref.close(_bits(ref.q_out), "q")
    at = ref.slots[ref.slots >= 0]
    kc = ref.tok(ref.cache.k.view(torch.int16)).view(np.uint16)[at]
    dead = ref.slots < 0
    live = Rope.__new__(Rope)
    live.__dict__.update(ref.__dict__, bits={"k": ref.bits["k"][~dead]}, pos=ref.pos[:, ~dead])
    live.close(kc, "k")
    r = Rope(T, 1, 8, kv=kv, idx=idx, seed=13)
    r.run()
    assert int(r.flags.item()) == 0 and f"warps_per_token={1 if T == 10000 else 2} " in msa.last_dispatch()
    assert torch.equal(r.q_out.view(torch.int16), ref.q_out.view(torch.int16))
    kf, vf = synth.bf16_bits_to_f32(kc), synth.bf16_bits_to_f32(ref.bits["v"])[~dead]
    if kv == "bf16":
        assert np.array_equal(r.tok(r.cache.v.view(torch.int16)).view(np.uint16)[at], ref.bits["v"][~dead])
    elif kv == "fp8":
        assert np.array_equal(r.tok(r.cache.k)[at], Qz.quant_kv_fp8(kf, np.float32(FP8_S)))
        assert np.array_equal(r.tok(r.cache.v)[at], Qz.quant_kv_fp8(vf, np.float32(FP8_S)))
    else:
        for got, gs, x in ((r.cache.k, r.cache.k_scale, kf), (r.cache.v, r.cache.v_scale, vf)):
            codes, scales = Qz.quant_nvfp4(x, np.float32(FP4_G))
            assert np.array_equal(r.tok(got)[at], codes) and np.array_equal(r.tok(gs)[at], scales)
    if idx:
        # the index branch is fed the first query head and the keys
        assert torch.equal(r.iq_out.view(torch.int16), r.q_out[:, :1].contiguous().view(torch.int16))
    if idx == "fp8":
        codes, scale = Qz.quant_index_keys_fp8(kf)
        assert np.array_equal(r.tok(r.ic.keys)[at], codes)
        assert np.array_equal(r.tok(r.ic.scale)[at].view(np.uint32), scale.view(np.uint32))
    elif idx == "nvfp4":
        codes, scales = Qz.quant_nvfp4(kf, np.float32(FP4_G))
        assert np.array_equal(r.tok(r.ic.keys)[at], codes) and np.array_equal(r.tok(r.ic.block_scale)[at], scales)


@pytest.mark.parametrize("group,Q", [(16, 1), (16, 2), (16, 4)])
def test_nvfp4_offsets_past_32_bits(group, Q):
    """The last pages of an NVFP4 cache whose codes and scales lie past 4 GiB (2^29 rows of 64 + 8 bytes, K and V)."""
    c = Case([400, 129], "nvfp4", 4, group, Q, seed=17)
    P = 2 ** 32 // (4 * 128 * 8) + c.P + 8
    assert P * 4 * 128 < 2 ** 31
    for name in ("k", "v", "k_scale", "v_scale"):
        t = getattr(c.cache, name)
        x = torch.empty((P,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda")
        x[P - c.P:] = t
        setattr(c.cache, name, x)
    c.table_d = torch.where(c.table_d >= 0, c.table_d + (P - c.P), c.table_d)
    c.dims.num_pages = P
    c.run()
    c.check()
    c.cache = None
    torch.cuda.empty_cache()
