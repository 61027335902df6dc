"""A full-attention layer's step, as a program runs it: metadata from lengths, norm + rotary + insert, attention; a
prompt, decode steps and a speculative step, eager and from captured graphs, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa, synth
from block_sparse_attention_07_gb300.workload import DeviceWorkload
from oracle import formats as F
from oracle import mrope as Mr
from oracle import msa as omsa
from oracle import run as orun

import parity
from paged import FP4_G, FP8_S, KINDS, bf16, encode

pytestmark = pytest.mark.gpu

G, GROUP, D, EPS, THETA = 2, 8, 128, 1e-6, 10000.0
H = G * GROUP


class Layer:
    def __init__(self, B, NB, pages, kv, seed):
        self.rng = np.random.default_rng(seed)
        self.B, self.NB, self.P, self.kv = B, NB, pages, kv
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        self.table, self.ctx, self.seq, self.starts = i32(B, NB).fill_(-1), i32(B), i32(B), i32(B + 1)
        self.head, self.head_out, self.flags = i32(1), i32(1), i32(1)
        self.free = torch.from_numpy(self.rng.permutation(pages).astype(np.int32)).cuda()
        row = D // 2 if kv == "nvfp4" else D
        nan = lambda *s: torch.full(s, 0xFF, dtype=torch.uint8, device="cuda")
        g = {"bf16": 1.0, "fp8": FP8_S, "nvfp4": FP4_G}[kv]
        if kv == "bf16":
            store = [nan(pages, G, 128, 2 * D).view(torch.bfloat16) for _ in range(2)] + [None, None]
        else:
            store = [nan(pages, G, 128, row) for _ in range(2)]
            store += [nan(pages, G, 128, 8).fill_(0x7F) for _ in range(2)] if kv == "nvfp4" else [None, None]
        self.cache = msa.KVCache(KINDS[kv], *store, g, g)
        self.w = {n: (1 + 0.1 * self.rng.standard_normal(D)).astype(np.float32) for n in "qk"}
        self.wd = {n: torch.from_numpy(x).cuda() for n, x in self.w.items()}
        self.nr = msa.make_norm_rope(self.wd["q"], self.wd["k"], eps=EPS, rope_theta=THETA)
        self.axes = msa.make_rope_axes((16, 24, 24))
        self.axis = Mr.sections_to_axis((16, 24, 24))
        self.K, self.V = [np.zeros((0, G, D))] * B, [np.zeros((0, G, D))] * B

    def buffers(self, T, Q):
        b = dict(new=torch.zeros(self.B, dtype=torch.int32, device="cuda"), T=T, Q=Q,
                 slots=torch.empty(T, dtype=torch.int64, device="cuda"),
                 pos=torch.empty((3, T), dtype=torch.int32, device="cuda"),
                 lse=torch.empty((self.B, Q, H), device="cuda"))
        for n, h in (("q", H), ("k", G), ("v", G), ("q_out", H)):
            b[n] = torch.zeros((T, h, D), dtype=torch.bfloat16, device="cuda")
        b["out"] = torch.empty((self.B, Q, H, D), dtype=torch.bfloat16, device="cuda")
        b["dims"] = msa.make_dims(self.B, Q, H, G, G, max_blocks_per_seq=self.NB, num_pages=self.P)
        b["ws"] = torch.empty(msa.paged_gqa_workspace_size(b["dims"], self.cache.dtype), dtype=torch.uint8, device="cuda")
        return b

    def issue(self, b, attend=True):
        msa.build_step(b["dims"], self.ctx, b["new"], self.free, self.head, self.table, self.seq, self.starts, b["slots"],
                       b["pos"], self.head_out, self.flags)
        msa.qk_norm_mrope_insert(b["dims"], b["q"], b["k"], b["v"], None, None, b["pos"], b["slots"], self.nr, self.axes,
                                 b["q_out"], None, self.cache, None, self.flags)
        if attend:
            q = b["q_out"][:self.B * b["Q"]].view(self.B, b["Q"], H, D)
            msa.paged_gqa_decode(b["dims"], q, self.cache, self.table, self.seq, b["out"], b["lse"], b["ws"], self.flags)
        self.ctx.copy_(self.seq)
        self.head.copy_(self.head_out)

    def feed(self, b, new):
        """Random projections of a step; the oracle's K and V grow with them (before the call changes ctx)."""
        ctx = [len(k) for k in self.K]
        b["new"].copy_(torch.tensor(new, dtype=torch.int32))
        raw = {n: self.rng.standard_normal((b["T"], h, D)).astype(np.float32) for n, h in (("q", H), ("k", G), ("v", G))}
        for n, x in raw.items():
            b[n].copy_(bf16(x))
        pos = np.concatenate([c + np.arange(n) for c, n in zip(ctx, new)])
        bits = {n: synth.f32_to_bf16_bits(x)[:len(pos)] for n, x in raw.items()}
        p3 = np.tile(pos, (3, 1))
        self.q_want = Mr.norm_mrope(bits["q"], self.w["q"], p3, self.axis, EPS, THETA)
        kf = synth.bf16_bits_to_f32(Mr.norm_mrope(bits["k"], self.w["k"], p3, self.axis, EPS, THETA))
        vf = synth.bf16_bits_to_f32(bits["v"])
        at = 0
        for i, n in enumerate(new):
            self.K[i] = np.concatenate([self.K[i], encode(self.kv, kf[at:at + n])[2]])
            self.V[i] = np.concatenate([self.V[i], encode(self.kv, vf[at:at + n])[2]])
            at += n

    def check(self, b):
        torch.cuda.synchronize()
        assert int(self.flags.item()) == 0
        Q = b["Q"]
        got, lse = b["out"].float().cpu().numpy(), b["lse"].cpu().numpy()
        q = F.bf16_to_f64(self.q_want).reshape(self.B, Q, H, D)
        for i in range(self.B):
            L = len(self.K[i])
            assert int(self.seq[i]) == L
            for j in range(Q):
                n = L - Q + j + 1
                for g in range(G):
                    hs = slice(g * GROUP, (g + 1) * GROUP)
                    s = q[i, j, hs] @ self.K[i][:n, g].T / np.sqrt(D)
                    m = s.max(1, keepdims=True)
                    e = np.exp(s - m)
                    o = e @ self.V[i][:n, g] / e.sum(1, keepdims=True)
                    # the chain's own roundings (a query or key value one bf16 step off, a code one step off) are
                    # covered by the bounds the other attention tests of the framework use
                    err = np.abs(got[i, j, hs] - o)
                    assert err.max() <= 4e-2 and err.mean() <= 4e-3, (i, j, g, err.max(), err.mean())
                    assert np.abs(lse[i, j, hs] - (m + np.log(e.sum(1, keepdims=True)))[:, 0]).max() <= 2e-2


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
def test_prompt_then_decode_then_speculation(kv):
    B = 3
    layer = Layer(B, NB=6, pages=20, kv=kv, seed=1)
    prompt = [130, 1, 300]
    b = layer.buffers(sum(prompt) + 9, 1)
    layer.feed(b, prompt)
    layer.issue(b, attend=False)
    torch.cuda.synchronize()
    assert layer.seq.tolist() == prompt and (b["slots"][sum(prompt):] == -1).all()
    one, spec = layer.buffers(B, 1), layer.buffers(B * 4, 4)
    for _ in range(2):
        layer.feed(one, [1] * B)
        layer.issue(one)
        layer.check(one)
    layer.feed(spec, [4] * B)
    layer.issue(spec)
    layer.check(spec)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "nvfp4"])
def test_captured_steps_cross_a_block_border(kv):
    """One captured decode step replayed while every request grows past the end of a page."""
    B = 2
    layer = Layer(B, NB=4, pages=10, kv=kv, seed=2)
    prompt = [126, 254]
    b = layer.buffers(sum(prompt), 1)
    layer.feed(b, prompt)
    layer.issue(b, attend=False)
    one = layer.buffers(B, 1)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    state = [t.clone() for t in (layer.ctx, layer.table, layer.head)]
    with torch.cuda.stream(stream):
        one["new"].fill_(1)
        layer.issue(one)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer.issue(one)
    for t, s in zip((layer.ctx, layer.table, layer.head), state):
        t.copy_(s)
    for _ in range(5):
        layer.feed(one, [1] * B)
        torch.cuda.synchronize()
        graph.replay()
        layer.check(one)


@pytest.mark.parametrize("kv,Q", [("bf16", 1), ("fp8", 8), ("nvfp4", 2)])
def test_workload_dense_step(kv, Q):
    """A full-attention layer beside a sparse one: same requests, own caches; eager, then replayed."""
    base = synth.WORKLOADS["nvfp4_256k" if kv == "nvfp4" else "b32_32k"]
    w = synth.scaled(base, batch=3, ctx=700, kv_dtype=kv, q_len=Q)
    src = parity.build(w)
    layer = DeviceWorkload.layer_like(src, 2)
    layer.dense_step()
    torch.cuda.synchronize()
    eager = layer.out.clone(), layer.lse.clone()
    g = layer.capture(layer.dense_step)
    layer.out.zero_()
    layer.lse.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert layer.check_flags() == 0
    assert torch.equal(layer.out, eager[0]) and torch.equal(layer.lse, eager[1])
    scale = synth.kv_scale(w)
    for bi, b in enumerate(layer.which):
        L = int(layer.lens[bi])
        req = synth.request(layer.w, b, L)
        K, V = (orun.cached_kv_rows(req[n], kv, scale) for n in "kv")
        out, lse = omsa.dense_gqa(orun.to_f32(req["q"]), K, V, L, w.softmax_scale)
        parity.check_attention(eager[0][bi].float().cpu().numpy(), eager[1][bi].cpu().numpy(), out, lse, f"{kv} b={b}")


def test_readme_example():
    """The README's second block runs as written after its first; with one token per request the output is its V."""
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    blocks = re.findall(r"```python\n(.*?)```", open(path, encoding="utf-8").read(), flags=re.S)
    env = {}
    for block in blocks[:2]:
        exec(compile(block, "README.md", "exec"), env)
    torch.cuda.synchronize()
    assert "paged_gqa_decode" in blocks[1]
    slots = env["slot_map"].tolist()
    assert slots == [int(env["free"][b]) * 128 for b in range(2)] and int(env["head_next"]) == 2
    for b, slot in enumerate(slots):
        v = env["cache"].v[slot // 128, :, slot % 128]
        assert torch.equal(env["out"][b, 0].view(4, 16, 128), v[:, None].expand(4, 16, 128))
