"""A layer's attention half from hidden states to hidden states (``DeviceWorkload.hidden_step``): every stage against the
fp64 oracle of the same inputs, the whole against the same calls one by one, eager and from a captured graph."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa, synth
from block_sparse_attention_07_gb300.workload import DeviceWorkload
from oracle import layer as L
from oracle import prologue as Pr


pytestmark = pytest.mark.gpu

HIDDEN = 2064                                                # ends inside a scale's group


def f64(t):
    return t.double().cpu().numpy()


def build(kind, index=True, seed=0):
    w = synth.scaled(synth.WORKLOADS[kind], batch=3, ctx=1500)
    dw = DeviceWorkload(w, "cuda", lens=np.array([1500, 129, 1153], dtype=np.int32), index_cache=index)
    T = 3 * w.q_len
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randn((T, HIDDEN), generator=gen, device="cuda").bfloat16()
    res = torch.randn((T, HIDDEN), generator=gen, device="cuda").bfloat16()
    return dw, x, res, torch.zeros((T, HIDDEN), dtype=torch.bfloat16, device="cuda")


CASES = [("b32_32k", True), ("spec8", True), ("fp8kv_32k", True), ("fp4_256k", True), ("spec8", False), ("nvfp4_256k", False)]


@pytest.mark.parametrize("kind,index", CASES)
def test_stages(kind, index):
    dw, x, res, y = build(kind, index)
    x0, r0 = f64(x), f64(res)
    dw.hidden_step(x, res, y)
    torch.cuda.synchronize()
    assert dw.check_flags() == 0
    st = dw._layer
    # norm and 8-bit rows: a step of E4M3 at most from the exact value (half a step, and the fp32 error at a border)
    h, n = L.add_norm(x0, r0, f64(st["norm"]), synth.PROLOGUE_EPS)
    assert (np.abs(f64(res) - h) <= 2.0 ** -8 * np.abs(h) * 1.001).all()
    got = L.dequant(st["x8"][0].cpu().numpy(), f64(st["x8"][1]))
    assert (np.abs(got - n) <= np.maximum(np.abs(n) * 2.0 ** -4, np.repeat(f64(st["x8"][1]), 128, 1)[:, :HIDDEN] * 2.0 ** -10) * 1.001).all()

    def product(a, w, out):
        want, size = L.linear(a[0].cpu().numpy(), f64(a[1]), w[0].cpu().numpy(), f64(w[1]))
        lim = (128 * 2.0 ** -23 + (a[1].shape[1] + 10) * 2.0 ** -24) * size
        assert (np.abs(f64(out) - want) <= lim + 2.0 ** -8 * (np.abs(want) + lim)).all()

    product(st["x8"], st["w_in"], st["packed"].flatten(1))
    # queries: the rotation of the projection's rows
    q = f64(st["parts"][0])
    wq = f64(dw._pro["weights"]["q"])
    f, gain = L.frequencies(128, synth.PROLOGUE_THETA)
    n = Pr.rms_norm(q, wq, synth.PROLOGUE_EPS)
    want = L.rotate(n, st["positions"].cpu().numpy(), f, gain, False)
    mag = np.tile(np.abs(n[..., :64]) + np.abs(n[..., 64:]), 2)
    assert (np.abs(f64(st["q"]) - want) <= 2.0 ** -8 * np.abs(want) + 97 * 2.0 ** -24 * mag).all()
    # the attention's output in 8 bits, and the output projection
    codes, scales = L.quant_rows(dw.out.float().cpu().numpy().reshape(st["o8"][0].shape))
    assert np.array_equal(st["o8"][0].cpu().numpy(), codes) and np.array_equal(st["o8"][1].cpu().numpy(), scales)
    product(st["o8"], st["w_out"], y)


@pytest.mark.parametrize("kind,index", CASES)
def test_attention_of_the_step(kind, index):
    """The attention in the middle is the library's own call on the step's queries and caches, bit for bit."""
    dw, x, res, y = build(kind, index, seed=1)
    dw.hidden_step(x, res, y)
    st, out, lse = dw._layer, dw.out.clone(), dw.lse.clone()
    q = st["q"].view(out.shape)
    if index:
        scores, sel = torch.empty_like(dw.scores), torch.empty_like(dw.selected)
        msa.index_score(dw.dims, st["q_idx"], msa.BF16, dw.idx_cache, dw.block_table_d, dw.seq_lens_d, scores, dw.flags)
        msa.select_blocks(dw.dims, scores, dw.seq_lens_d, sel, dw.flags)
        msa.sparse_gqa_decode(dw.dims, q, dw.cache, dw.block_table_d, dw.seq_lens_d, sel, dw.out, dw.lse, dw.workspace, dw.flags)
        assert torch.equal(scores, dw.scores) and torch.equal(sel, dw.selected)
    else:
        msa.paged_gqa_decode(dw.dims, q, dw.cache, dw.block_table_d, dw.seq_lens_d, dw.out, dw.lse, st["ws"], dw.flags)
    torch.cuda.synchronize()
    assert torch.equal(out, dw.out) and torch.equal(lse, dw.lse) and dw.check_flags() == 0


@pytest.mark.parametrize("kind,index", [("b32_32k", True), ("spec8", False)])
def test_captured_steps(kind, index):
    """A captured step replayed over changing inputs gives an eager step's bits; two layers one after the other share
    nothing but the residual stream."""
    dw, x, res, y = build(kind, index, seed=2)
    other, _, _, y2 = build(kind, index, seed=3)
    xs = [torch.randn_like(x) for _ in range(3)]
    r0, want = res.clone(), []

    def both(stream=None):
        dw.hidden_step(x, res, y, stream)
        other.hidden_step(y, res, y2, stream)

    for new in xs:
        x.copy_(new)
        res.copy_(r0)
        both()
        want.append((res.clone(), y.clone(), y2.clone()))
    g = dw.capture(both)
    for new, w in zip(xs, want):
        x.copy_(new)
        res.copy_(r0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(w, (res, y, y2)))
    assert dw.check_flags() == 0 and other.check_flags() == 0


def test_other_rotary_form():
    dw, x, res, y = build("b32_32k", seed=4)
    r0 = res.clone()
    dw.hidden_step(x, res, y)
    first = dw._layer["q"].clone()
    res.copy_(r0)
    rope = msa.make_rope(64, synth.PROLOGUE_THETA, msa.ROPE_INTERLEAVED, msa.ROPE_BY_PARTS, 4.0, 4096)
    dw.hidden_step(x, res, y, rope=rope)
    torch.cuda.synchronize()
    q = dw._layer["q"]
    assert dw.check_flags() == 0
    n = Pr.rms_norm(f64(dw._layer["parts"][0]), f64(dw._pro["weights"]["q"]), synth.PROLOGUE_EPS)
    f, gain = L.frequencies(64, synth.PROLOGUE_THETA, "parts", 4.0, 4096.0)
    want = L.rotate(n, dw._layer["positions"].cpu().numpy(), f, gain, True)
    mag = np.abs(n)
    mag[..., :64] = gain * np.repeat(mag[..., 0:64:2] + mag[..., 1:64:2], 2, -1)
    assert (np.abs(f64(q) - want) <= 2.0 ** -8 * np.abs(want) + 97 * 2.0 ** -24 * mag).all()
    assert not torch.equal(first, q)
