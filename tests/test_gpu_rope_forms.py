"""msa_qkv_rope_insert against the fp64 oracle.

Bounds: outputs are the fp64 result rounded to bf16 (2^-8 relative). The kernel's fp32 error: with the norm, the mean of
squares (128 roundings of 2^-24, halved by the root), root and two products (4 * 2^-24); the rotation: cos and sin within
2^-22 of the gain, phases within 2^-24 of a turn at a frequency of at most one, i.e. 2^-21 (the sum of both under
12 * 2^-24), one product with the gain, 4 roundings: under 96 * 2^-24 of gain * (|a| + |b|) for the pair (a, b). Quantised caches are compared byte for
byte with the oracle's quantisers applied to the bf16 rows that the same call stores in a bf16 cache."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa, synth
from oracle import formats as F
from oracle import layer as L
from oracle import prologue as Pr
from oracle import quant as Qz

from paged import FP4_G, FP8_S, KINDS, bf16

pytestmark = pytest.mark.gpu

D, EPS, THETA = 128, 1e-6, 10000.0
SCALINGS = {"none": msa.ROPE_NONE, "linear": msa.ROPE_LINEAR, "parts": msa.ROPE_BY_PARTS, "turns": msa.ROPE_BY_TURNS}


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Case:
    """One packed row per token: queries, keys, values, index queries, index keys, and some elements of padding."""

    def __init__(self, T, G=4, H=None, kv="bf16", idx=None, R=128, interleaved=False, scaling="none", norm=True, seed=0,
                 max_pos=131072, pad=0, theta=THETA, size=1.0):
        rng = np.random.default_rng(seed)
        H = 16 * G if H is None else H
        self.T, self.G, self.H, self.kv, self.idx, self.R, self.inter = T, G, H, kv, idx, R, interleaved
        self.P = P = -(-T // 128) + 2
        heads = H + 2 * G + (2 * G if idx else 0)
        raw = rng.standard_normal((T, heads, D)) * rng.uniform(0.2, 5, (T, heads, 1)) * size
        flat = torch.full((T, heads * D + pad), float("nan"), dtype=torch.bfloat16)
        flat[:, :heads * D] = bf16(raw).reshape(T, -1)
        self.packed = flat.cuda()
        cut = lambda a, n: self.packed[:, a * D:(a + n) * D].unflatten(1, (n, D))
        self.q, self.k, self.v = cut(0, H), cut(H, G), cut(H + G, G)
        self.iq, self.ik = (cut(H + 2 * G, G), cut(H + 3 * G, G)) if idx else (None, None)
        self.pos = rng.integers(0, max_pos, T).astype(np.int32)
        self.pos[:min(T, 3)] = np.array([0, 1, max_pos - 1], dtype=np.int32)[:T]
        self.slots = rng.permutation(P * 128)[:T].astype(np.int64)
        if T > 4:
            self.slots[3] = -1
        self.w = {n: (1.0 + 0.1 * rng.standard_normal(D)).astype(np.float32) if norm else None for n in ("q", "k", "iq", "ik")}
        scale_args = dict(factor=4.0, trained_len=8192, low_turns=1.0, high_turns=32.0)
        self.rope = msa.make_rope(R, theta, int(interleaved), SCALINGS[scaling], **scale_args)
        self.freq, self.gain = L.frequencies(R, theta, scaling, 4.0, 8192.0, 1.0, 32.0)
        row = {"bf16": D, "fp8": D, "nvfp4": D // 2}[kv]
        z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device="cuda")
        g = {"bf16": 1.0, "fp8": FP8_S, "nvfp4": FP4_G}[kv]
        sc = [z(P, G, 128, 8), z(P, G, 128, 8)] if kv == "nvfp4" else [None, None]
        dt = torch.bfloat16 if kv == "bf16" else torch.uint8
        self.cache = msa.KVCache(KINDS[kv], z(P, G, 128, row, dtype=dt), z(P, G, 128, row, dtype=dt), *sc, g, g)
        self.ic = None
        if idx == "fp8":
            self.ic = msa.IndexCache(msa.FP8_E4M3, z(P, G, 128, D), z(P, G, 128, dtype=torch.float32))
        elif idx == "nvfp4":
            self.ic = msa.IndexCache(msa.NVFP4, z(P, G, 128, D // 2), None, z(P, G, 128, 8), FP4_G)
        self.wd = {n: None if a is None else torch.from_numpy(a).cuda() for n, a in self.w.items()}
        self.nr = msa.make_norm_rope(*(self.wd[n] for n in ("q", "k", "iq", "ik")), eps=EPS) if norm else None
        self.q_out = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
        self.iq_out = torch.zeros((T, G, D), dtype=torch.bfloat16, device="cuda") if idx else None
        self.pos_d, self.slots_d = torch.from_numpy(self.pos).cuda(), torch.from_numpy(self.slots).cuda()
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dims = msa.make_dims(1, 1, H, G, G, max_blocks_per_seq=P, num_pages=P)

    def run(self, flags=0, stream=None):
        msa.qkv_rope_insert(self.dims, self.q, self.k, self.v, self.iq, self.ik, self.pos_d, self.slots_d, self.nr, self.rope,
                            self.q_out, self.iq_out, self.cache, self.ic, self.flags, stream=stream)
        torch.cuda.synchronize()
        assert int(self.flags.item()) == flags

    def tok(self, a):
        return a.cpu().numpy().transpose(0, 2, 1, *range(3, a.dim())).reshape(self.P * 128, a.shape[1], *a.shape[3:])

    def cached(self, a):
        return self.tok(a.view(torch.int16)).view(np.uint16)

    def close(self, got_bits, x, name, rows=slice(None)):
        x = F.bf16_to_f64(_bits(x))[rows]
        y = x if self.w[name] is None else Pr.rms_norm(x, self.w[name], EPS)
        want = L.rotate(y, self.pos[rows], self.freq, self.gain, self.inter)
        R = self.R
        mag = np.abs(y)
        if self.inter:
            mag[..., :R] = self.gain * np.repeat(mag[..., 0:R:2] + mag[..., 1:R:2], 2, -1)
        else:
            mag[..., :R] = self.gain * np.tile(mag[..., :R // 2] + mag[..., R // 2:R], 2)
        lim = 2.0 ** -8 * np.abs(want) + 97 * 2.0 ** -24 * mag
        err = np.abs(F.bf16_to_f64(got_bits) - want)
        assert (err <= lim).all(), f"{name}: {(err / np.maximum(lim, 1e-300)).max():.3g}x the bound"

    def check(self):
        self.close(_bits(self.q_out), self.q, "q")
        live = self.slots >= 0
        if self.kv == "bf16":
            kc, vc = self.cached(self.cache.k), self.cached(self.cache.v)
            self.close(kc[self.slots[live]], self.k, "k", live)
            assert np.array_equal(vc[self.slots[live]], _bits(self.v)[live])
            assert int(kc.reshape(self.P * 128, -1).any(1).sum()) == live.sum()     # nothing else was written
        if self.idx:
            self.close(_bits(self.iq_out), self.iq, "iq")


@pytest.mark.parametrize("T", [1, 2, 7, 8, 70, 300, 3000])
@pytest.mark.parametrize("G,H", [(4, 64), (1, 8), (3, 15), (2, 2)])
@pytest.mark.parametrize("inter", [False, True])
def test_outputs_and_bf16_cache(T, G, H, inter):
    c = Case(T, G, H, seed=T + G, R=64, interleaved=inter)
    c.run()
    c.check()


@pytest.mark.parametrize("R", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_every_part_of_the_head(R, inter, norm):
    c = Case(40, 2, 12, idx="fp8", R=R, interleaved=inter, norm=norm, seed=R)
    c.run()
    c.check()


@pytest.mark.parametrize("scaling", ["none", "linear", "parts", "turns"])
@pytest.mark.parametrize("R", [64, 128])
def test_scalings(scaling, R):
    c = Case(60, scaling=scaling, R=R, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("max_pos,theta", [(2 ** 31 - 1, 10000.0), (2 ** 31 - 1, 1.5), (1024, 5e6)])
def test_far_positions(max_pos, theta):
    assert max_pos * 2.0 ** -53 < 2.0 ** -21               # the oracle's own angles
    c = Case(60, seed=4, max_pos=max_pos, theta=theta)
    c.run()
    c.check()


def test_negative_positions_turn_back():
    c = Case(30, seed=5, R=64)
    c.pos = -c.pos
    c.pos_d.neg_()
    c.run()
    c.check()


def test_half_whole_head_is_the_fused_prologue():
    """R = 128, half layout, no scaling: the same fp64 result as msa_qk_norm_rope_insert, each within its bound."""
    c = Case(90, seed=6)
    c.run()
    one = torch.zeros_like(c.q_out)
    msa.qk_norm_rope_insert(c.dims, c.q.contiguous(), c.k.contiguous(), c.v.contiguous(), None, None, c.pos_d, c.slots_d,
                            msa.make_norm_rope(c.wd["q"], c.wd["k"], eps=EPS, rope_theta=THETA), one, None, c.cache, None, c.flags)
    torch.cuda.synchronize()
    c.close(_bits(one), c.q, "q")
    c.check()


def test_padded_rows_contiguous_rows_and_in_place():
    c = Case(33, seed=7, pad=24, idx="fp8", R=96)
    c.run()
    c.check()
    first, keys = c.q_out.clone(), c.cache.k.clone()
    c.q, c.k, c.v, c.iq, c.ik = (t.contiguous() for t in (c.q, c.k, c.v, c.iq, c.ik))
    c.q_out.zero_(), c.cache.k.zero_()
    c.run()
    assert torch.equal(first, c.q_out) and torch.equal(keys, c.cache.k)
    c.q_out, c.iq_out = c.q, c.iq                           # q_out may be q where it is contiguous
    c.run()
    assert torch.equal(first, c.q)


@pytest.mark.parametrize("T,G,H", [(6000, 4, 64), (6000, 3, 15), (400, 2, 28), (5, 1, 6)])
def test_in_place_by_warps_per_token(T, G, H):
    """Queries turned where they lie, with rows on their way ahead of their turn: the bits of another place's."""
    c = Case(T, G, H, seed=17, kv="fp8", R=64)
    c.run()
    first = c.q_out.clone()
    for _ in range(2):
        c.q_out = c.q = c.packed[:, :H * D].unflatten(1, (H, D)).contiguous()
        c.run()
        assert torch.equal(first, c.q_out)


def test_two_calls_at_once():
    """Calls on two streams share nothing."""
    cs = [Case(T, seed=T, kv="nvfp4", idx="nvfp4") for T in (900, 40)]
    for c in cs:
        c.run()
    outs = lambda c: (c.q_out, c.iq_out, c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale, c.ic.keys, c.ic.block_scale)
    want = [[t.clone() for t in outs(c)] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for c, s in zip(cs, streams):
            msa.qkv_rope_insert(c.dims, c.q, c.k, c.v, c.iq, c.ik, c.pos_d, c.slots_d, c.nr, c.rope, c.q_out, c.iq_out,
                                c.cache, c.ic, c.flags, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for c, w in zip(cs, want) for a, b in zip(w, outs(c)))


@pytest.mark.parametrize("kv", ["fp8", "nvfp4"])
@pytest.mark.parametrize("idx", [None, "fp8", "nvfp4"])
@pytest.mark.parametrize("T,G,R,inter", [(70, 4, 128, False), (9, 1, 64, True), (40, 3, 48, False), (300, 2, 80, False)])
def test_quantised_caches_byte_exact(kv, idx, T, G, R, inter):
    ref = Case(T, G, kv="bf16", idx="fp8", seed=10, R=R, interleaved=inter)
    ref.run()
    c = Case(T, G, kv=kv, idx="fp8", seed=10, R=R, interleaved=inter)
    c.idx = idx
    if idx is None:
        c.iq = c.ik = c.iq_out = None
        c.ic = None
    elif idx == "nvfp4":
        z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
        c.ic = msa.IndexCache(msa.NVFP4, z(c.P, G, 128, D // 2), None, z(c.P, G, 128, 8), FP4_G)
    c.run()
    assert torch.equal(ref.q_out, c.q_out)
    at = c.slots[c.slots >= 0]
    kf = synth.bf16_bits_to_f32(ref.cached(ref.cache.k)[at])
    vf = synth.bf16_bits_to_f32(_bits(ref.v)[c.slots >= 0])
    if kv == "fp8":
        assert np.array_equal(c.tok(c.cache.k)[at], Qz.quant_kv_fp8(kf, np.float32(FP8_S)))
        assert np.array_equal(c.tok(c.cache.v)[at], Qz.quant_kv_fp8(vf, np.float32(FP8_S)))
    else:
        for got, gs, x in ((c.cache.k, c.cache.k_scale, kf), (c.cache.v, c.cache.v_scale, vf)):
            codes, scales = Qz.quant_nvfp4(x, np.float32(FP4_G))
            assert np.array_equal(c.tok(got)[at], codes) and np.array_equal(c.tok(gs)[at], scales)
    if idx is None:
        return
    # the index keys as bf16: the same rows through a call that takes them as its keys, with their weights
    as_k = Case(T, G, kv="bf16", idx="fp8", seed=10, R=R, interleaved=inter)
    as_k.k, as_k.nr = as_k.ik, msa.make_norm_rope(as_k.wd["q"], as_k.wd["ik"], as_k.wd["iq"], as_k.wd["ik"], eps=EPS)
    as_k.run()
    xf = synth.bf16_bits_to_f32(as_k.cached(as_k.cache.k)[at])
    assert torch.equal(ref.iq_out, c.iq_out)
    if idx == "fp8":
        codes, scale = Qz.quant_index_keys_fp8(xf)
        assert np.array_equal(c.tok(c.ic.keys)[at], codes)
        assert np.array_equal(c.tok(c.ic.scale)[at].view(np.uint32), scale.view(np.uint32))
    else:
        codes, scales = Qz.quant_nvfp4(xf, np.float32(FP4_G))
        assert np.array_equal(c.tok(c.ic.keys)[at], codes) and np.array_equal(c.tok(c.ic.block_scale)[at], scales)


@pytest.mark.parametrize("inter", [False, True])
def test_infinities_stay_with_their_pair(inter):
    """Without a norm, dims that pass and pairs that hold no infinity or NaN are as without them."""
    c = Case(20, 1, 8, R=64, interleaved=inter, norm=False, seed=11)
    c.run()
    want = c.q_out.clone()
    c.q[3, :, 100], c.q[5, :, 127], c.q[7, :, 6], c.q[9, :, 66] = float("inf"), float("nan"), float("-inf"), float("inf")
    c.run()
    other = 7 if inter else 38
    for t, dims in ((3, [100]), (5, [127]), (7, [6, other]), (9, [66])):
        keep = [d for d in range(D) if d not in dims]
        assert torch.equal(c.q_out[t, :, keep], want[t, :, keep]) and not torch.isfinite(c.q_out[t][:, dims]).any()
    assert (c.q_out[3, :, 100] == float("inf")).all() and (c.q_out[9, :, 66] == float("inf")).all()


@pytest.mark.parametrize("power", [-66, 66, 120])
def test_magnitudes(power):
    """Squares that leave fp32's range."""
    c = Case(12, seed=12, size=2.0 ** power, R=64)
    c.run()
    c.check()


def test_bad_and_negative_slots_and_zero_rows():
    c = Case(20, kv="fp8", idx="fp8", seed=13)
    c.packed.zero_()
    c.slots_d[5] = c.P * 128 + 3
    c.run(flags=msa.FLAG_BAD_SLOT)
    assert not (c.cache.k & 0x7F).any() and not c.ic.keys.any() and not c.ic.scale.any() and not c.q_out.any()


def test_no_token_writes_its_neighbours():
    """Every slot negative: queries turn, the caches stay as they are."""
    c = Case(40, kv="nvfp4", idx="nvfp4", seed=14)
    c.slots_d.fill_(-1)
    for t in (c.cache.k, c.cache.v, c.cache.k_scale, c.ic.keys, c.ic.block_scale):
        t.fill_(0x5A)
    c.run()
    assert all((t == 0x5A).all() for t in (c.cache.k, c.cache.v, c.cache.k_scale, c.ic.keys, c.ic.block_scale))
    c.close(_bits(c.q_out), c.q, "q")


def test_batch_size_does_not_change_results_and_graph():
    c = Case(3000, seed=15, R=64)
    c.run()
    few = Case(3000, seed=15, R=64)
    few.q, few.k, few.v, few.pos_d, few.slots_d, few.q_out = (t[:5] for t in (few.q, few.k, few.v, few.pos_d, few.slots_d, few.q_out))
    few.run()
    assert torch.equal(c.q_out[:5], few.q_out)
    want = c.q_out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        msa.qkv_rope_insert(c.dims, c.q, c.k, c.v, None, None, c.pos_d, c.slots_d, c.nr, c.rope, c.q_out, None, c.cache, None, c.flags)
    c.q_out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, c.q_out)


def test_packed_rows_past_4_gib():
    """260,000 tokens of 66 heads: offsets of the packed rows and the queries past 32 bits; the last tokens are those of a
    short call."""
    T = 260_000
    P = -(-T // 128)
    packed = torch.zeros((T, 66, 128), dtype=torch.bfloat16, device="cuda")
    n = 300
    packed[-n:] = torch.randn((n, 66, 128), device="cuda").bfloat16()
    rope = msa.make_rope(64)
    pos = torch.arange(T, device="cuda").int()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(p, pos, slots, P):
        t = p.shape[0]
        dims = msa.make_dims(1, 1, 16, 1, 1, max_blocks_per_seq=P, num_pages=P)
        kc, vc = (torch.zeros((P, 1, 128, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = torch.empty((t, 16, 128), dtype=torch.bfloat16, device="cuda")
        msa.qkv_rope_insert(dims, p[:, 40:56], p[:, 64:65], p[:, 65:66], None, None, pos, slots, None, rope, q, None,
                            msa.KVCache(msa.BF16, kc, vc), None, flags)
        return q, kc.view(-1, 128), vc.view(-1, 128)

    q, k, v = call(packed, pos, torch.arange(T, device="cuda"), P)
    q1, k1, v1 = call(packed[-n:].clone(), pos[-n:].contiguous(), torch.arange(n, device="cuda"), 3)
    assert int(flags.item()) == 0
    assert torch.equal(q[-n:], q1) and torch.equal(k[T - n:T], k1[:n]) and torch.equal(v[T - n:T], v1[:n])
    assert q1.any() and not q[:-n].any()
