"""What ``DeviceWorkload.hidden_step`` puts into the caches and into the index queries: the packed projection's own parts,
cut here by their places in a row, with the norm weights of the seed."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa, synth
from oracle import formats as F
from oracle import layer as L
from oracle import prologue as Pr
from oracle import quant as Qz

from test_gpu_hidden_step import CASES, build

pytestmark = pytest.mark.gpu

D = 128


def by_token(a):
    """A cache [P, heads, 128, ...] as [P * 128, heads, ...]."""
    a = a.view(torch.int16) if a.dtype == torch.bfloat16 else a
    a = a.cpu().numpy()
    return a.transpose(0, 2, 1, *range(3, a.ndim)).reshape(-1, a.shape[1], *a.shape[3:])


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def check_turned(got_bits, rows, weight, positions):
    """bf16 rows against fp64: 2^-8 of their own rounding, 96 * 2^-24 of the kernel's fp32 steps."""
    n = Pr.rms_norm(rows.double().cpu().numpy(), weight, synth.PROLOGUE_EPS)
    f, gain = L.frequencies(D, synth.PROLOGUE_THETA)
    want = L.rotate(n, positions, f, gain, False)
    mag = np.tile(np.abs(n[..., :64]) + np.abs(n[..., 64:]), 2)
    assert (np.abs(F.bf16_to_f64(got_bits) - want) <= 2.0 ** -8 * np.abs(want) + 97 * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("kind,index", CASES)
def test_rows_in_the_caches(kind, index):
    dw, x, res, y = build(kind, index, seed=5)
    w = dw.w
    c, ic = dw.cache, dw.idx_cache
    held = {"k": c.k, "v": c.v, "k_scale": c.k_scale, "v_scale": c.v_scale}
    if index:
        held.update(keys=ic.keys, scale=ic.scale, block_scale=ic.block_scale)
    held = {n: t for n, t in held.items() if t is not None}
    before = {n: by_token(t) for n, t in held.items()}
    dw.hidden_step(x, res, y)
    torch.cuda.synchronize()
    assert dw.check_flags() == 0
    after = {n: by_token(t) for n, t in held.items()}
    H, G, I = w.n_heads, w.n_kv_heads, w.n_idx_heads
    packed = dw._layer["packed"]
    T = packed.shape[0]
    at = dw.new_slots.cpu().numpy()
    other = np.ones(len(after["k"]), dtype=bool)
    other[at] = False
    for n in held:
        assert np.array_equal(after[n][other], before[n][other]), n
        assert not np.array_equal(after[n][at], before[n][at]), n
    pos = (dw.lens.astype(np.int64)[:, None] - w.q_len + np.arange(w.q_len)).reshape(-1)
    weights = synth.norm_weights(w)

    def turned(rows, weight):
        """bf16 rows [T, G, D] as the keys of a call of their own into a bf16 cache of one token per slot."""
        wd = torch.from_numpy(weight).cuda()
        P = -(-T // 128)
        kc, vc = (torch.zeros((P, G, 128, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        dims = msa.make_dims(1, 1, H, G, G, max_blocks_per_seq=P, num_pages=P)
        q = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        msa.qkv_rope_insert(dims, q, rows.contiguous(), rows.contiguous(), None, None, torch.from_numpy(pos.astype(np.int32)).cuda(),
                            torch.arange(T, device="cuda"), msa.make_norm_rope(wd, wd, eps=synth.PROLOGUE_EPS),
                            msa.make_rope(D, synth.PROLOGUE_THETA), torch.empty_like(q), None, msa.KVCache(msa.BF16, kc, vc), None, flags)
        assert int(flags.item()) == 0
        got = by_token(kc)[:T].view(np.uint16)
        check_turned(got, rows, weight, pos)
        return got

    k = turned(packed[:, H:H + G], weights["k"])
    v = bits(packed[:, H + G:H + 2 * G])
    if w.kv_dtype == "bf16":
        assert np.array_equal(after["k"][at].view(np.uint16), k) and np.array_equal(after["v"][at].view(np.uint16), v)
    else:
        for name, row, g in (("k", k, c.k_global), ("v", v, c.v_global)):
            row = synth.bf16_bits_to_f32(row)
            if w.kv_dtype == "fp8":
                assert np.array_equal(after[name][at], Qz.quant_kv_fp8(row, np.float32(g)))
            else:
                codes, scales = Qz.quant_nvfp4(row, np.float32(g))
                assert np.array_equal(after[name][at], codes) and np.array_equal(after[name + "_scale"][at], scales)
    if not index:
        return
    assert np.array_equal(bits(dw._layer["q_idx"]), turned(packed[:, H + 2 * G:H + 2 * G + I], weights["idx_q"]))
    row = synth.bf16_bits_to_f32(turned(packed[:, H + 2 * G + I:], weights["idx_k"]))
    if w.idx_dtype == "nvfp4":
        codes, scales = Qz.quant_nvfp4(row, np.float32(ic.global_scale))
        assert np.array_equal(after["keys"][at], codes) and np.array_equal(after["block_scale"][at], scales)
    else:
        codes, scale = Qz.quant_index_keys_fp8(row)
        assert np.array_equal(after["keys"][at], codes) and np.array_equal(after["scale"][at].view(np.uint32), scale.view(np.uint32))
