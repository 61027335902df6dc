"""Calls of one kernel that take unequal amounts of shared memory, from several host threads at one time, each on a stream of
its own: none is refused for another's sake."""
import threading

import pytest
import torch

from block_sparse_attention_07_gb300 import msa

pytestmark = pytest.mark.gpu

D = 128


def score_call(B, kind, stream):
    G, NB, P = 4, 2, 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(B)
    table = torch.randint(0, P, (B, NB), generator=gen, device="cuda").int()
    lens = torch.randint(1, 2 * 128 + 1, (B,), generator=gen, device="cuda").int()
    if kind == "f32":
        q = torch.randn((B, 1, G, D), generator=gen, device="cuda")
        cache = msa.IndexCache(msa.F32, torch.randn((P, G, 128, D), generator=gen, device="cuda"))
    else:
        q = torch.randn((B, 1, G, D), generator=gen, device="cuda").bfloat16()
        keys = torch.randn((P, G, 128, D), generator=gen, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        cache = msa.IndexCache(msa.FP8_E4M3, keys, torch.rand((P, G, 128), generator=gen, device="cuda"))
    scores, flags = torch.zeros((B, 1, G, NB), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dims = msa.make_dims(B, 1, 16 * G, G, G, max_blocks_per_seq=NB, num_pages=P)
    call = msa.index_score(dims, q, msa.F32 if kind == "f32" else msa.BF16, cache, table, lens, scores, flags, stream=stream, prepare=True)
    return call, scores, flags, (q, cache, table, lens)


def attend_call(NB, kind, stream):
    B, Q, G, P = 4, 2, 4, 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(NB)
    table = torch.randint(0, P, (B, NB), generator=gen, device="cuda").int()
    lens = torch.full((B,), 200, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((P, G, 128, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((B, Q, 16 * G, D), generator=gen, device="cuda").bfloat16()
    sel = torch.full((B, Q, G, 16), -1, dtype=torch.int32, device="cuda")
    sel[..., 0], sel[..., 1] = 0, 1
    out, lse = torch.zeros_like(q), torch.zeros((B, Q, 16 * G), device="cuda")
    dims = msa.make_dims(B, Q, 16 * G, G, G, max_blocks_per_seq=NB, num_pages=P)
    cache = msa.KVCache(msa.BF16, k, v)
    ws = torch.zeros(max(256, msa.sparse_gqa_workspace_size(dims, msa.BF16)), dtype=torch.uint8, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = msa.sparse_gqa_decode(dims, q, cache, table, lens, sel, out, lse, ws, flags, stream=stream, prepare=True)
    return call, out, flags, (q, cache, table, lens, sel, lse, ws)


CASES = [(score_call, "fp8", (3, 400, 2000, 4000), ""), (score_call, "f32", (3, 400, 2000, 4000), ""),
         (attend_call, "union", (16, 1024, 4096, 8192), "union_of_positions"),
         (attend_call, "union_mma", (16, 1024, 4096, 8192), "union_of_positions")]


@pytest.mark.parametrize("make,kind,sizes,name", CASES, ids=["index fp8", "index f32", "union", "union mma"])
def test_sizes_at_one_time(monkeypatch, make, kind, sizes, name):
    if kind.startswith("union"):
        monkeypatch.setenv("MSA_MULTIPOS_ATTENTION", kind)
    streams = [torch.cuda.Stream() for _ in sizes]
    calls = [make(n, kind, s) for n, s in zip(sizes, streams)]
    torch.cuda.synchronize()
    want = []
    for call, out, _, _ in calls:
        call()
        torch.cuda.synchronize()
        assert name in msa.last_dispatch(), msa.last_dispatch()
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            for n in range(4000):
                calls[i][0]()
                if n % 8 == 7:                           # (the index call's queue holds 64 calls that run at one time)
                    streams[i].synchronize()
            streams[i].synchronize()
        except Exception as e:      # noqa: BLE001 (reported by the main thread)
            failed.append((sizes[i], repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert all(torch.equal(w, c[1]) and int(c[2].item()) == 0 for w, c in zip(want, calls))
