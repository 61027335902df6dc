"""Shared pieces of the dense paged-attention tests: caches in every format with
known fp64 values, the fp64 attention, and the bounds its GPU results are held to.

Bounds, with u(t) = half a step of a type (bf16 2^-8, fp32 2^-24) and, per query
row, A = sum_t softmax_t |v_t| (elementwise), n the number of tokens seen:
  * logits: 128 exact products summed in fp32 (at most 130 roundings) and one
    multiply by the scale: d_s <= 132 * 2^-24 * scale * max_t sum_d |q_d k_td|.
    For quantised caches the query may be held as two 4-bit-significand parts
    after a power-of-two scaling of its row, exact down to 2^-18 of its largest
    value: + 2^-18 * scale * max|q| * max_t sum_d |k_td|.
  * probabilities: rounded to bf16 or better, 2^-8 relative; those below 2^-23 of
    the largest may be lost: n * 2^-23 * max|v| absolute; 2^-21 for the
    exponential; the logit error moves them by d_s relative, twice (numerator and
    denominator).
  * sums of n terms in fp32: n * 2^-24 relative to A.
  * the output's rounding to bf16: 2^-8 |out|.
  * lse: d_s + 2^-21 + n * (2^-24 + 2^-23) + 2^-22 |lse| absolute.
"""
from __future__ import annotations

import numpy as np
import torch

from block_sparse_attention_07_gb300 import msa, synth
from oracle import formats as F
from oracle import quant as Qz

BS, D = 128, 128
FP8_S = float(np.float32(synth.FP8_KV_SYNTH_SCALE))
FP4_G = float(np.float32(synth.NVFP4_SYNTH_GLOBAL))
KINDS = {"bf16": msa.BF16, "fp8": msa.FP8_E4M3, "nvfp4": msa.NVFP4}


def bf16(x):
    return torch.from_numpy(synth.f32_to_bf16_bits(np.asarray(x, dtype=np.float32)).view(np.int16)).view(torch.bfloat16)


def encode(kind, x):
    """fp32 values [..., 128] -> (stored array, scales or None, fp64 values)."""
    if kind == "bf16":
        bits = synth.f32_to_bf16_bits(x)
        return bits, None, F.bf16_to_f64(bits)
    if kind == "fp8":
        code = Qz.quant_kv_fp8(x, FP8_S)
        return code, None, F.e4m3_decode(code) * FP8_S
    code, sc = Qz.quant_nvfp4(x, FP4_G)
    return code, sc, F.nvfp4_decode(code, sc, FP4_G)


class Case:
    """A paged cache holding requests of given lengths, every other byte poisoned with NaN patterns."""

    def __init__(self, lens, kind="bf16", G=4, group=16, Q=1, seed=0, q_scale=1.0, k_fn=None, spare=3, scale=None,
                 device="cuda", cols_extra=1):
        rng = np.random.default_rng(seed)
        self.lens, self.kind, self.G, self.group, self.Q = list(lens), kind, G, group, Q
        B, H = len(lens), G * group
        nb = [-(-max(n, 0) // BS) for n in lens]
        P = sum(nb) + spare
        self.P, self.NB = P, max(nb + [1]) + cols_extra
        perm = rng.permutation(P)
        self.table = np.full((B, self.NB), -1, dtype=np.int32)
        poison = {"bf16": (np.uint16, 0xFFFF, D), "fp8": (np.uint8, 0xFF, D), "nvfp4": (np.uint8, 0xFF, D // 2)}[kind]
        store = {n: np.full((P, G, BS, poison[2]), poison[1], dtype=poison[0]) for n in "kv"}
        sc = {n: np.full((P, G, BS, D // 16), 0x7F, dtype=np.uint8) for n in "kv"} if kind == "nvfp4" else None
        self.K, self.V = [], []
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :nb[b]] = perm[at:at + nb[b]]
            vals = {}
            for name in "kv":
                x = rng.standard_normal((max(n, 0), G, D)).astype(np.float32)
                if k_fn is not None and name == "k":
                    x = k_fn(x, b)
                code, s, val = encode(kind, x)
                vals[name] = val
                for t0 in range(0, n, BS):
                    page = self.table[b, t0 // BS]
                    m = min(BS, n - t0)
                    store[name][page, :, :m] = code[t0:t0 + m].transpose(1, 0, 2)
                    if s is not None:
                        sc[name][page, :, :m] = s[t0:t0 + m].transpose(1, 0, 2)
            self.K.append(vals["k"])
            self.V.append(vals["v"])
            at += nb[b]
        q = (rng.standard_normal((B, Q, H, D)) * q_scale).astype(np.float32)
        self.q_val = F.bf16_to_f64(synth.f32_to_bf16_bits(q))
        self.scale = 1.0 / np.sqrt(D) if scale is None else scale
        self.dims = msa.make_dims(B, Q, H, G, G, max_blocks_per_seq=self.NB, num_pages=P, softmax_scale=scale)
        dev = lambda a: (torch.from_numpy(a.view(np.int16)).view(torch.bfloat16) if a.dtype == np.uint16
                         else torch.from_numpy(a)).to(device)
        g = {"bf16": 1.0, "fp8": FP8_S, "nvfp4": FP4_G}[kind]
        self.cache = msa.KVCache(KINDS[kind], dev(store["k"]), dev(store["v"]), dev(sc["k"]) if sc else None,
                                 dev(sc["v"]) if sc else None, g, g)
        self.q = bf16(q).to(device)
        self.table_d = torch.from_numpy(self.table).to(device)
        self.lens_d = torch.tensor(self.lens, dtype=torch.int32).to(device)
        self.out = torch.full((B, Q, H, D), float("nan"), dtype=torch.bfloat16, device=device)
        self.lse = torch.full((B, Q, H), float("nan"), dtype=torch.float32, device=device)
        self.flags = torch.zeros(1, dtype=torch.int32, device=device)
        self.ws = torch.full((max(256, msa.paged_gqa_workspace_size(self.dims, KINDS[kind])),), 0xFF, dtype=torch.uint8,
                             device=device)

    def run(self, **kw):
        msa.paged_gqa_decode(self.dims, self.q, self.cache, self.table_d, self.lens_d, self.out, self.lse, self.ws,
                             self.flags, **kw)

    def expected(self, b, live_blocks=None):
        """fp64 (out, lse, A, d_s, n) of request b; live_blocks: those that count (all)."""
        Q, G, n = self.Q, self.G, self.group
        L = max(self.lens[b], 0)
        H = G * n
        out, lse = np.zeros((Q, H, D)), np.full((Q, H), -np.inf)
        A, ds, cnt = np.zeros((Q, H, D)), np.zeros((Q, H)), np.zeros(Q)
        tok = np.arange(L)
        keep = np.ones(L, bool) if live_blocks is None else np.isin(tok // BS, live_blocks)
        for j in range(Q):
            see = keep & (tok <= L - Q + j)
            cnt[j] = see.sum()
            if not see.any():
                continue
            for g in range(G):
                K, V = self.K[b][see, g], self.V[b][see, g]
                q = self.q_val[b, j, g * n:(g + 1) * n]
                s = self.scale * (q @ K.T)
                m = s.max(1, keepdims=True)
                e = np.exp(s - m)
                z = e.sum(1, keepdims=True)
                w = e / z
                hs = slice(g * n, (g + 1) * n)
                out[j, hs] = w @ V
                lse[j, hs] = (m + np.log(z))[:, 0]
                A[j, hs] = w @ np.abs(V)
                d = 132 * 2.0 ** -24 * self.scale * (np.abs(q) @ np.abs(K).T).max(1)
                if self.kind != "bf16":
                    d = d + 2.0 ** -18 * self.scale * np.abs(q).max(1) * np.abs(K).sum(1).max()
                ds[j, hs] = d
        return out, lse, A, ds, cnt

    def check(self, which=None, live_blocks=None, flags=0):
        torch.cuda.synchronize()
        assert int(self.flags.item()) == flags
        got, glse = self.out.float().cpu().numpy().astype(np.float64), self.lse.cpu().numpy().astype(np.float64)
        for b in range(len(self.lens)) if which is None else which:
            out, lse, A, ds, n = self.expected(b, None if live_blocks is None else live_blocks.get(b))
            vmax = np.abs(self.V[b]).max() if len(self.V[b]) else 0.0
            n3 = n[:, None, None]
            lim = (2.0 ** -8 * np.abs(out) + A * (2.0 ** -8 + 2.0 ** -21 + 2 * ds[..., None] + n3 * 2.0 ** -24)
                   + n3 * 2.0 ** -23 * vmax + 1e-30)
            err = np.abs(got[b] - out)
            assert np.isfinite(got[b]).all(), f"request {b}: non-finite output"
            assert (err <= lim).all(), f"request {b} (L={self.lens[b]}): output off by {(err / lim).max():.3g}x its bound"
            fin = np.isfinite(lse)
            assert np.array_equal(np.isneginf(glse[b]), ~fin), f"request {b}: empty rows differ"
            nn = np.broadcast_to(n[:, None], lse.shape)
            llim = ds + 2.0 ** -21 + nn * (2.0 ** -24 + 2.0 ** -23) + 2.0 ** -22 * np.abs(np.where(fin, lse, 0.0))
            lerr = np.abs(np.where(fin, glse[b] - np.where(fin, lse, 0.0), 0.0))
            assert (lerr <= llim).all(), f"request {b} (L={self.lens[b]}): lse off by {(lerr / llim).max():.3g}x its bound"
