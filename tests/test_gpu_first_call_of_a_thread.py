"""A host thread whose first use of CUDA is one of the library's calls: the tensor-map encoder needs a context of the thread,
which the launch has to make current first."""
import threading

import pytest
import torch

from block_sparse_attention_07_gb300 import msa

pytestmark = pytest.mark.gpu

D = 128


def linear(T):
    a, w = (torch.randn((n, 256), device="cuda").to(torch.float8_e4m3fn).view(torch.uint8) for n in (T, 300))
    sa, sw = torch.rand((T, 2), device="cuda"), torch.rand((3, 2), device="cuda")
    out, flags = torch.zeros((T, 300), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    return lambda s: msa.fp8_linear(a, sa, w, sw, out, flags, stream=s, prepare=True), out, flags


def attention(kind, Q, sparse):
    G, P, B = 2, 6, 3
    dims = msa.make_dims(B, Q, 16 * G, G, G, max_blocks_per_seq=2, num_pages=P)
    q = torch.randn((B, Q, 16 * G, D), device="cuda").bfloat16()
    if kind == "bf16":
        cache = msa.KVCache(msa.BF16, *(torch.randn((P, G, 128, D), device="cuda").bfloat16() for _ in range(2)))
    else:
        cache = msa.KVCache(msa.FP8_E4M3, *(torch.randn((P, G, 128, D), device="cuda").to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)),
                            None, None, 1.0, 1.0)
    table, lens = torch.arange(6, device="cuda").int().view(3, 2), torch.full((B,), 200, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((B, Q, 16 * G), device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    size = msa.sparse_gqa_workspace_size if sparse else msa.paged_gqa_workspace_size
    ws = torch.zeros(max(256, size(dims, cache.dtype)), dtype=torch.uint8, device="cuda")
    sel = torch.full((B, Q, G, 16), -1, dtype=torch.int32, device="cuda")
    sel[..., 0], sel[..., 1] = 0, 1
    keep = (q, cache, table, lens, lse, ws, sel)
    if sparse:
        return lambda s: (msa.sparse_gqa_decode(dims, q, cache, table, lens, sel, out, lse, ws, flags, stream=s, prepare=True), keep)[0], out, flags
    return lambda s: (msa.paged_gqa_decode(dims, q, cache, table, lens, out, lse, ws, flags, stream=s, prepare=True), keep)[0], out, flags


CASES = {"linear rows": (lambda: linear(20), {"MSA_LINEAR_FORM": "rows"}), "linear rows 128": (lambda: linear(130), {"MSA_LINEAR_FORM": "rows"}),
         "linear pairs": (lambda: linear(300), {"MSA_LINEAR_FORM": "pairs"}),
         "paged fp8": (lambda: attention("fp8", 1, False), {}), "paged fp8, 8 positions": (lambda: attention("fp8", 8, False), {}),
         "paged bf16, 8 positions": (lambda: attention("bf16", 8, False), {}),
         "sparse bf16": (lambda: attention("bf16", 1, True), {}), "sparse fp8": (lambda: attention("fp8", 1, True), {}),
         "sparse union": (lambda: attention("bf16", 4, True), {"MSA_MULTIPOS_ATTENTION": "union"}),
         "sparse union mma": (lambda: attention("bf16", 4, True), {"MSA_MULTIPOS_ATTENTION": "union_mma"})}


@pytest.mark.parametrize("case", list(CASES))
def test_first_call(monkeypatch, case):
    make, env = CASES[case]
    for n, v in env.items():
        monkeypatch.setenv(n, v)
    torch.manual_seed(0)
    prepare, out, flags = make()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = prepare(stream)
    call()                                               # what the library asks a device once is known now
    torch.cuda.synchronize()
    want = out.clone()
    assert want.any()
    for _ in range(2):
        out.zero_()
        torch.cuda.synchronize()
        failed = []

        def work():
            try:
                call()
            except Exception as e:      # noqa: BLE001 (reported by the main thread)
                failed.append(repr(e))

        t = threading.Thread(target=work)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not failed, failed
        assert torch.equal(out, want) and int(flags.item()) == 0
