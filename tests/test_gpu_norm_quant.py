"""msa_add_norm_quant against the fp64 oracle.

Bounds. h is one fp32 addition (2^-24). The mean of squares is a sum of at most 64 additions deep (8 passes x 8 values
in two chains, then ten exchange steps) of squares within 2^-24, so the root is off by at most 33 * 2^-24; root,
division and three products add five: |y - exact| <= 48 * 2^-24 |y|. bf16 adds 2^-8 |y|. A scale is one division of the
group's largest |y|: 50 * 2^-24. A code's value is y over the scale, within a reciprocal, a product and half a step of E4M3: 2^-4
relative, or 2^-10 where it is subnormal."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa, synth
from oracle import formats as F
from oracle import layer as L

from paged import bf16

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def check(h, y, out=None, codes=None, scales=None, res_out=None):
    if res_out is not None:
        u = U if res_out.dtype == torch.float32 else 2.0 ** -8
        assert (np.abs(f64(res_out) - h) <= (u + U) * np.abs(h) + 2.0 ** -140).all()
    if out is not None:
        assert (np.abs(f64(out) - y) <= (2.0 ** -8 + 48 * U) * np.abs(y) + 2.0 ** -130).all()
    if codes is not None:
        s = f64(scales)
        W = y.shape[1]
        top = np.stack([np.abs(y[:, g:g + 128]).max(1) for g in range(0, W, 128)], 1)
        assert (np.abs(s - top / 448) <= 52 * U * top / 448).all()
        v = F.e4m3_decode(codes.cpu().numpy()).astype(np.float64)
        want = y / np.maximum(np.repeat(top / 448, 128, 1)[:, :W], 1e-300)
        assert (np.abs(v - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 104 * U * np.abs(want)).all()
        assert (np.abs(v).max(1) == 448).sum() == (top.max(1) > 0).sum()


class Case:
    def __init__(self, T, W, res="bf16", seed=0, pad=0, size=1.0):
        rng = np.random.default_rng(seed)
        x = rng.standard_normal((T, W + pad)) * size * np.exp(rng.standard_normal(W + pad))
        self.x = bf16(x).cuda()[:, :W]
        self.res = None
        if res is not None:
            r = torch.from_numpy((3 * rng.standard_normal((T, W)) * size).astype(np.float32))
            self.res = (r if res == "f32" else r.bfloat16()).cuda()
        self.w = torch.from_numpy((1 + 0.1 * rng.standard_normal(W)).astype(np.float32)).cuda()
        # one row of guard behind every output
        self.full = dict(out=torch.full((T + 1, W), 7.0, dtype=torch.bfloat16, device="cuda"),
                         codes=torch.full((T + 1, W), 7, dtype=torch.uint8, device="cuda"),
                         scales=torch.full((T + 1, -(-W // 128)), 7.0, device="cuda"))
        if res is not None:
            self.full["residual_out"] = torch.full((T + 1, W), 7.0, dtype=self.res.dtype, device="cuda")
        self.T = T

    def run(self, weight=True, outs=("out", "codes", "scales", "residual_out"), eps=1e-6, **kw):
        o = {n: t[:self.T] for n, t in self.full.items() if n in outs}
        msa.add_norm_quant(self.x, self.w if weight else None, residual=self.res, eps=eps, **dict(o, **kw))
        torch.cuda.synchronize()
        for n, t in self.full.items():
            assert (t[self.T:] == 7).all() and (n in outs or (t == 7).all()), n
        h, y = L.add_norm(f64(self.x), None if self.res is None else f64(self.res), f64(self.w) if weight else None, eps)
        check(h, y, o.get("out"), o.get("codes"), o.get("scales"), o.get("residual_out"))
        return o


@pytest.mark.parametrize("res", [None, "bf16", "f32"])
@pytest.mark.parametrize("T,W", [(1, 16), (1, 4096), (2, 112), (3, 128), (5, 144), (7, 1040), (300, 272), (333, 5008), (320, 8192),
                                 (2, 16384), (310, 16384), (9, 12304), (1, 8208), (2050, 4096), (700, 12304),
                                 (600, 16384), (1900, 4432)])
def test_sizes(T, W, res):
    Case(T, W, res, seed=T + W).run()


@pytest.mark.parametrize("outs", [("out",), ("codes", "scales"), ("out", "residual_out"), ("codes", "scales", "residual_out")])
@pytest.mark.parametrize("weight", [True, False])
def test_each_output_alone(outs, weight):
    Case(6, 400, seed=1).run(weight=weight, outs=outs)


def test_rows_apart():
    Case(11, 256, seed=2, pad=24).run()
    Case(400, 2064, "f32", seed=3, pad=8).run()


@pytest.mark.parametrize("T,W", [(1, 16), (40, 8192), (700, 1296)])
def test_rounding_alone_is_byte_exact(T, W):
    """Without norm and residual the values are the inputs': codes and scales are the rule's, bit for bit."""
    c = Case(T, W, None, seed=4)
    o = c.run(weight=False, outs=("codes", "scales"))
    codes, scales = L.quant_rows(c.x.float().cpu().numpy())
    assert np.array_equal(o["codes"].cpu().numpy(), codes) and np.array_equal(o["scales"].cpu().numpy(), scales)


def test_in_place():
    c = Case(50, 1024, "f32", seed=5)
    h, y = L.add_norm(f64(c.x), f64(c.res), f64(c.w), 1e-6)
    x = c.x.contiguous()
    msa.add_norm_quant(x, c.w, residual=c.res, residual_out=c.res, out=x)
    torch.cuda.synchronize()
    check(h, y, out=x, res_out=c.res)


@pytest.mark.parametrize("T,W", [(2100, 4096), (1900, 4432), (6, 16384)])
def test_in_place_with_rows_ahead(T, W):
    """The same where rows are copied ahead of their turn, both streams in place; twice, the same bits."""
    c = Case(T, W, "bf16", seed=8)
    h, y = L.add_norm(f64(c.x), f64(c.res), f64(c.w), 1e-6)
    got = []
    for _ in range(2):
        x, r = c.x.clone(), c.res.clone()
        msa.add_norm_quant(x, c.w, residual=r, residual_out=r, out=x)
        torch.cuda.synchronize()
        assert ("ring" in msa.last_dispatch()) == (T > 100)
        got.append((x, r))
    check(h, y, out=got[0][0], res_out=got[0][1])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_two_calls_at_once():
    """Calls on two streams share nothing."""
    cs = [Case(T, 4096, "bf16", seed=T) for T in (2100, 64)]
    outs = [{n: t[:c.T] for n, t in c.full.items()} for c in cs]
    want = [{n: t.clone() for n, t in c.run().items()} for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for c, o, s in zip(cs, outs, streams):
            msa.add_norm_quant(c.x, c.w, residual=c.res, stream=s, **o)
    torch.cuda.synchronize()
    assert all(torch.equal(w[n], o[n]) for w, o in zip(want, outs) for n in w)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
@pytest.mark.parametrize("power", [-120, -70, -30, 30, 66, 120])
def test_magnitudes(power, eps):
    """Squares that leave fp32's range on either side."""
    rng = np.random.default_rng(power + 200)
    x = bf16(rng.uniform(0.5, 2.0, (4, 512)) * 2.0 ** power * rng.choice([-1, 1], (4, 512))).cuda()
    out = torch.empty_like(x)
    w = torch.ones(512, device="cuda")
    msa.add_norm_quant(x, w, out=out, eps=eps)
    torch.cuda.synchronize()
    h, y = L.add_norm(f64(x), None, f64(w), float(np.float32(eps)))
    check(h, y, out=out)


def test_zeros_infinities_and_nan():
    x = torch.zeros((5, 384), dtype=torch.bfloat16, device="cuda")
    x[1] = 1.0
    x[2, 130] = float("nan")
    x[3, 5], x[3, 6] = float("inf"), 3.0
    x[4, 200] = 2.0                                            # zeros in the groups around
    w = torch.ones(384, device="cuda")
    out, codes, scales = torch.empty_like(x), torch.empty((5, 384), dtype=torch.uint8, device="cuda"), torch.empty((5, 3), device="cuda")
    msa.add_norm_quant(x, w, out=out, codes=codes, scales=scales)
    torch.cuda.synchronize()
    assert not out[0].any() and not codes[0].any() and not scales[0].any()
    assert (out[1] == 1).all() and ((scales[1] * 448 - 1).abs() <= 1e-6).all()      # 1 / sqrt(1 + eps)
    assert out[2].isnan().all()
    assert out[3, 5].isnan() and not out[3, :5].any() and not out[3, 6:].any()
    v = codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, 1)
    assert v[2].isnan().all() and v[3, :128].isnan().all() and not v[3, 128:].any()
    assert scales[4, 0] == 0 and scales[4, 2] == 0 and (codes[4] == 0).sum() == 383
    # without the norm: a group that holds an infinity or a NaN is NaN where its scale is applied, the others are not
    msa.add_norm_quant(x, None, codes=codes, scales=scales)
    torch.cuda.synchronize()
    v = codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, 1)
    assert v[3, :128].isnan().all() and v[2, 128:256].isnan().all() and not v[2, :128].any() and not v[2, 256:].any()


def test_zero_row_without_eps_is_nan_as_the_formula():
    x = torch.zeros((1, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    msa.add_norm_quant(x, torch.ones(128, device="cuda"), out=out, eps=0.0)
    assert out.isnan().all()


def test_repeats_streams_and_graph():
    c = Case(200, 4096, seed=6)
    first = {n: t.clone() for n, t in c.run().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = {n: t[:c.T] for n, t in c.full.items()}
    with torch.cuda.stream(side):
        for t in o.values():
            t.zero_()
        msa.add_norm_quant(c.x, c.w, residual=c.res, **o)
    side.synchronize()
    assert all(torch.equal(first[n], t) for n, t in o.items())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        msa.add_norm_quant(c.x, c.w, residual=c.res, **o)
    for t in o.values():
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first[n], t) for n, t in o.items())


def test_many_rows_past_4_gib():
    """Row offsets past 32 bits: 140,000 rows of 16,384 values, the last ones checked."""
    T, W = 140000, 16384
    x = torch.zeros((T, W), dtype=torch.bfloat16, device="cuda")
    x[-3:] = bf16(np.random.default_rng(7).standard_normal((3, W))).cuda()
    codes, scales = torch.full((T, W), 9, dtype=torch.uint8, device="cuda"), torch.empty((T, W // 128), device="cuda")
    msa.add_norm_quant(x, None, codes=codes, scales=scales)
    torch.cuda.synchronize()
    want, ws = L.quant_rows(x[-3:].float().cpu().numpy())
    assert np.array_equal(codes[-3:].cpu().numpy(), want) and np.array_equal(scales[-3:].cpu().numpy(), ws)
    assert not codes[:-3].any()
