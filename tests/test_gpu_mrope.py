"""QK-norm + rotary on several axes + insert against the fp64 oracle.

Bounds: outputs are the fp64 result rounded to bf16, off by at most one bf16 step
where the kernel's fp32 error crosses a rounding border. That error: the mean of
squares (128 roundings, 2^-24 each, halved by the root), root, division, two
products (5 roundings) and the rotation (cos and sin within 2^-22, 3 roundings):
under 80 * 2^-24 of |a| + |b| for the pair (a, b). Quantised caches are compared
byte for byte with the oracle's quantisers applied to the bf16 rows that the same
call stores in a bf16 cache."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa, synth
from oracle import formats as F
from oracle import mrope as Mr
from oracle import prologue as Pr
from oracle import quant as Qz

from paged import FP4_G, FP8_S, KINDS, bf16

pytestmark = pytest.mark.gpu

D, EPS, THETA = 128, 1e-6, 10000.0


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


class Rope:
    def __init__(self, T, G=4, H=None, kv="bf16", idx=None, sections=(16, 24, 24), interleaved=False, seed=0,
                 max_pos=262144, theta=THETA, pos_pad=0):
        rng = np.random.default_rng(seed)
        self.T, self.G, self.H, self.kv, self.idx, self.theta = T, G, 16 * G if H is None else H, kv, idx, theta
        A = len(sections)
        P = -(-T // 128) + 2
        self.P = P
        raw = {n: (rng.standard_normal((T, c, D)) * rng.uniform(0.2, 5, (T, c, 1))).astype(np.float32)
               for n, c in (("q", self.H), ("k", G), ("v", G))}
        self.bits = {n: synth.f32_to_bf16_bits(a) for n, a in raw.items()}
        self.pos = rng.integers(0, max_pos, (A, T)).astype(np.int32)
        self.pos[:, :min(T, 3)] = np.array([0, 1, max_pos - 1], dtype=np.int32)[:T]
        self.slots = rng.permutation(P * 128)[:T].astype(np.int64)
        if T > 4:
            self.slots[3] = -1
        self.axes = msa.make_rope_axes(sections, interleaved)
        self.axis = Mr.sections_to_axis(sections, interleaved)
        self.w = {n: (1.0 + 0.1 * rng.standard_normal(D)).astype(np.float32) for n in ("q", "k")}
        row = {"bf16": D, "fp8": D, "nvfp4": D // 2}[kv]
        dt = torch.bfloat16 if kv == "bf16" else torch.uint8
        z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device="cuda")
        g = {"bf16": 1.0, "fp8": FP8_S, "nvfp4": FP4_G}[kv]
        sc = [z(P, G, 128, 8), z(P, G, 128, 8)] if kv == "nvfp4" else [None, None]
        self.cache = msa.KVCache(KINDS[kv], z(P, G, 128, row, dtype=dt), z(P, G, 128, row, dtype=dt), *sc, g, g)
        self.ic = None
        if idx == "fp8":
            self.ic = msa.IndexCache(msa.FP8_E4M3, z(P, G, 128, D), z(P, G, 128, dtype=torch.float32))
        elif idx == "nvfp4":
            self.ic = msa.IndexCache(msa.NVFP4, z(P, G, 128, D // 2), None, z(P, G, 128, 8), FP4_G)
        self.wd = {n: torch.from_numpy(a).cuda() for n, a in self.w.items()}
        self.q, self.k, self.v = (bf16(raw[n]).cuda() for n in "qkv")
        self.q_out = torch.zeros_like(self.q)
        self.iq_out = torch.zeros((T, G, D), dtype=torch.bfloat16, device="cuda")
        pos = np.full((A, T + pos_pad), 2 ** 30, dtype=np.int32)
        pos[:, :T] = self.pos
        self.pos_d = torch.from_numpy(pos).cuda()[:, :T]
        self.slots_d = torch.from_numpy(self.slots).cuda()
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dims = msa.make_dims(1, 1, self.H, G, G, max_blocks_per_seq=P, num_pages=P)

    def run(self, stream=None):
        nr = msa.make_norm_rope(self.wd["q"], self.wd["k"], self.wd["q"], self.wd["k"], EPS, self.theta)
        # the index branch is fed the query's first heads and the keys, with their weights
        iq = self.q[:, :self.G].contiguous() if self.idx else None
        msa.qk_norm_mrope_insert(self.dims, self.q, self.k, self.v, iq, self.k if self.idx else None, self.pos_d,
                                 self.slots_d, nr, self.axes, self.q_out, self.iq_out if self.idx else None, self.cache,
                                 self.ic, self.flags, stream=stream)
        torch.cuda.synchronize()

    def tok(self, a):
        return a.cpu().numpy().transpose(0, 2, 1, *range(3, a.dim())).reshape(self.P * 128, a.shape[1], *a.shape[3:])

    def close(self, got_bits, name):
        x = F.bf16_to_f64(self.bits[name])
        want = F.bf16_to_f64(Mr.norm_mrope(self.bits[name], self.w[name], self.pos, self.axis, EPS, self.theta))
        got = F.bf16_to_f64(got_bits)
        y = np.abs(Pr.rms_norm(x, self.w[name], EPS))
        pair = np.tile(y[..., :64] + y[..., 64:], 2)
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -126))) - 7)
        lim = step * 1.0000001 + 80 * 2.0 ** -24 * pair
        err = np.abs(got - want)
        assert (err <= lim).all(), f"{name}: {(err / lim).max():.3g}x the bound"
        assert np.mean(got_bits != Mr.norm_mrope(self.bits[name], self.w[name], self.pos, self.axis, EPS, self.theta)) < 0.01


@pytest.mark.parametrize("T", [1, 2, 7, 8, 70, 300, 3000])
@pytest.mark.parametrize("G,H", [(4, 64), (1, 8), (3, 15), (2, 2)])
def test_outputs_and_bf16_cache(T, G, H):
    r = Rope(T, G, H, seed=T + G)
    r.run()
    assert int(r.flags.item()) == 0
    r.close(_bits(r.q_out), "q")
    live = r.slots >= 0
    kc = r.tok(r.cache.k.view(torch.int16)).view(np.uint16)
    vc = r.tok(r.cache.v.view(torch.int16)).view(np.uint16)
    full = np.zeros_like(r.bits["k"])
    full[live] = kc[r.slots[live]]
    full[~live] = Mr.norm_mrope(r.bits["k"], r.w["k"], r.pos, r.axis, EPS, THETA)[~live]
    r.close(full, "k")
    assert np.array_equal(vc[r.slots[live]], r.bits["v"][live])
    assert int(kc.reshape(r.P * 128, -1).any(1).sum()) == live.sum()        # nothing else was written


@pytest.mark.parametrize("sections,inter", [((64,), False), ((16, 24, 24), False), ((24, 20, 20), True), ((0, 32, 32), False),
                                            ((16, 16, 16, 16), True), ((40, 24), False)])
def test_sections(sections, inter):
    r = Rope(50, sections=sections, interleaved=inter, seed=5)
    r.run()
    r.close(_bits(r.q_out), "q")


@pytest.mark.parametrize("max_pos,theta", [(2 ** 31 - 1, 10000.0), (2 ** 31 - 1, 1.5), (1024, 5e6), (4096, 3e38)])
def test_far_positions_and_bases(max_pos, theta):
    r = Rope(60, seed=6, max_pos=max_pos, theta=theta)
    r.run()
    # fp64 angles of the oracle: position * frequency is rounded once, 2^-53 relative
    assert max_pos * 2.0 ** -53 < 2.0 ** -21
    r.close(_bits(r.q_out), "q")


def test_negative_positions_turn_back():
    """A position offset may take a rotary position below zero."""
    r = Rope(30, seed=7)
    r.pos = -r.pos
    r.pos_d.neg_()
    r.run()
    r.close(_bits(r.q_out), "q")


def test_equal_axes_are_the_one_axis_rotation():
    """With equal positions on all axes both prologues hold to the same fp64 result; values may differ by a step."""
    r = Rope(90, seed=8)
    r.pos[:] = r.pos[0]
    r.pos_d.copy_(r.pos_d[:1].expand(3, -1).clone())
    r.run()
    one = torch.zeros_like(r.q)
    nr = msa.make_norm_rope(r.wd["q"], r.wd["k"], None, None, EPS, THETA)
    msa.qk_norm_rope_insert(r.dims, r.q, r.k, r.v, None, None, r.pos_d[0].contiguous(), r.slots_d, nr, one, None, r.cache,
                            None, r.flags)
    torch.cuda.synchronize()
    r.close(_bits(one), "q")
    r.close(_bits(r.q_out), "q")


def test_position_rows_apart_and_in_place():
    r = Rope(33, seed=9, pos_pad=7)
    r.run()
    r.close(_bits(r.q_out), "q")
    first = r.q_out.clone()
    r.q_out = r.q                                       # q_out may be q
    r.run()
    assert torch.equal(first.view(torch.int16), r.q.view(torch.int16))


@pytest.mark.parametrize("kv", ["fp8", "nvfp4"])
@pytest.mark.parametrize("idx", [None, "fp8", "nvfp4"])
@pytest.mark.parametrize("T,G", [(70, 4), (9, 1), (40, 3)])
def test_quantised_caches_byte_exact(kv, idx, T, G):
    ref = Rope(T, G, kv="bf16", seed=10)
    ref.run()
    r = Rope(T, G, kv=kv, idx=idx, seed=10)
    r.run()
    assert int(r.flags.item()) == 0
    at = r.slots[r.slots >= 0]
    kf = synth.bf16_bits_to_f32(ref.tok(ref.cache.k.view(torch.int16)).view(np.uint16)[at])
    vf = synth.bf16_bits_to_f32(ref.bits["v"])[r.slots >= 0]
    c = r.cache
    if kv == "fp8":
        assert np.array_equal(r.tok(c.k)[at], Qz.quant_kv_fp8(kf, np.float32(FP8_S)))
        assert np.array_equal(r.tok(c.v)[at], Qz.quant_kv_fp8(vf, np.float32(FP8_S)))
    else:
        for got, gs, x in ((c.k, c.k_scale, kf), (c.v, c.v_scale, vf)):
            codes, scales = Qz.quant_nvfp4(x, np.float32(FP4_G))
            assert np.array_equal(r.tok(got)[at], codes) and np.array_equal(r.tok(gs)[at], scales)
    if idx:
        assert torch.equal(r.iq_out.view(torch.int16), r.q_out[:, :G].contiguous().view(torch.int16))
    if idx == "fp8":
        codes, scale = Qz.quant_index_keys_fp8(kf)
        assert np.array_equal(r.tok(r.ic.keys)[at], codes)
        assert np.array_equal(r.tok(r.ic.scale)[at].view(np.uint32), scale.view(np.uint32))
    elif idx == "nvfp4":
        codes, scales = Qz.quant_nvfp4(kf, np.float32(FP4_G))
        assert np.array_equal(r.tok(r.ic.keys)[at], codes) and np.array_equal(r.tok(r.ic.block_scale)[at], scales)


def test_zero_rows_and_bad_slots():
    r = Rope(20, kv="fp8", idx="fp8", seed=11)
    r.k.zero_()
    r.q[2].zero_()
    r.slots_d[5] = r.P * 128 + 3
    r.run()
    assert int(r.flags.item()) == msa.FLAG_BAD_SLOT
    # 0 turned by a negative cosine is -0, whose E4M3 code 0x80 holds the same value; index codes of a zero scale are 0
    assert not (r.cache.k & 0x7F).any() and not r.ic.keys.any() and not r.ic.scale.any()
    assert not r.q_out[2].any() and torch.isfinite(r.q_out.float()).all()


def test_warps_per_token_do_not_change_results():
    """A token's rows give the same bits alone (one warp per four rows) and in a long batch (one warp per token)."""
    r = Rope(3000, seed=12)
    r.run()
    one = Rope(3000, seed=12)
    n = 5
    nr = msa.make_norm_rope(one.wd["q"], one.wd["k"], None, None, EPS, THETA)
    msa.qk_norm_mrope_insert(one.dims, one.q[:n], one.k[:n], one.v[:n], None, None, one.pos_d[:, :n], one.slots_d[:n], nr,
                             one.axes, one.q_out[:n], None, one.cache, None, one.flags)
    torch.cuda.synchronize()
    assert torch.equal(r.q_out[:n].view(torch.int16), one.q_out[:n].view(torch.int16))
