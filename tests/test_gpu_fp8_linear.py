"""msa_fp8_linear against the fp64 oracle.

Bound, with S = sum_k |a w| of the values (scales included) and KB groups of K: within a group 128 products, exact in
fp32, are added by the tensor core with at least 24 bits kept of the largest partial sum, at most 2^-23 lost per
addition: 128 * 2^-23 S. Outside, one product of scales, KB fused additions and at most 8 more where several CTAs share
K: (KB + 10) * 2^-24 S. The output's rounding: 2^-8 |out| for bf16, 2^-24 for fp32."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa
from oracle import formats as F
from oracle import layer as L

pytestmark = pytest.mark.gpu


def _codes(rng, rows, K):
    x = np.clip(rng.standard_normal((rows, K)) * 60, -448, 448).astype(np.float32)
    return torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8)


class Case:
    def __init__(self, T, N, K, dtype=torch.bfloat16, seed=0, pad=0):
        rng = np.random.default_rng(seed)
        KB = -(-K // 128)
        self.T, self.N, self.K, self.KB = T, N, K, KB
        self.a, self.w = _codes(rng, T, K).cuda(), _codes(rng, N, K).cuda()
        # scales of unequal size: a wrong one, or a group left out, is far outside the bound
        self.sa = torch.from_numpy(np.exp(rng.uniform(-3, 3, (T, KB))).astype(np.float32)).cuda()
        self.sw = torch.from_numpy((np.exp(rng.uniform(-3, 3, (-(-N // 128), KB))) * 1e-4).astype(np.float32)).cuda()
        self.full = torch.full((T + 1, N + pad), 7.0, dtype=dtype, device="cuda")
        self.out = self.full[:T, :N]
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        msa.fp8_linear(self.a, self.sa, self.w, self.sw, self.out, self.flags, stream=stream)
        torch.cuda.synchronize()
        assert int(self.flags.item()) == 0
        assert (self.full[self.T:] == 7).all() and (self.full[:, self.N:] == 7).all()       # nothing beside the outputs

    def check(self, rows=None):
        rows = slice(None) if rows is None else rows
        want, size = L.linear(self.a[rows].cpu().numpy(), self.sa[rows].cpu().numpy(), self.w.cpu().numpy(), self.sw.cpu().numpy())
        got = self.out[rows].double().cpu().numpy()
        u = 2.0 ** -24 if self.out.dtype == torch.float32 else 2.0 ** -8
        lim = (128 * 2.0 ** -23 + (self.KB + 10) * 2.0 ** -24) * size
        lim = lim + u * (np.abs(want) + lim)
        err = np.abs(got - want)
        assert (err <= lim).all(), f"{(err / np.maximum(lim, 1e-300)).max():.3g}x the bound, {np.argwhere(err > lim)[:4]}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 128, 128), (2, 130, 256), (15, 300, 400), (16, 128, 1040), (17, 1000, 512), (32, 257, 2064),
                                   (33, 640, 640), (64, 200, 4112), (65, 129, 128), (100, 1280, 1024), (128, 384, 272),
                                   (129, 260, 2048), (300, 700, 1296), (1, 4096, 8192), (700, 1000, 304), (1030, 515, 640)])
def test_sizes(T, N, K, dtype):
    c = Case(T, N, K, dtype, seed=T + N + K)
    c.run()
    c.check()


@pytest.mark.parametrize("split", [1, 2, 3, 5, 7, 8])
@pytest.mark.parametrize("T,N,K", [(1, 200, 1040), (40, 300, 2176), (128, 128, 4096), (9, 130, 1152)])
def test_every_split(monkeypatch, split, T, N, K):
    monkeypatch.setenv("MSA_LINEAR_SPLIT", str(split))
    c = Case(T, N, K, seed=split)
    c.run()
    assert msa.last_dispatch().endswith(f"split={split}")
    c.check()


@pytest.mark.parametrize("T", [1, 20, 64])
def test_both_sizes_of_the_rows_form(T):
    """Few tiles take a whole SM each, many share one; over two CTAs per SM they follow one another."""
    for N, K, deep in ((1280, 2048, True), (28672, 272, False), (60000, 144, False)):
        c = Case(T, N, K, seed=T)
        c.run()
        assert (" deep" in msa.last_dispatch()) == deep, msa.last_dispatch()
        c.check()


@pytest.mark.parametrize("split", [1, 2, 3, 4])
@pytest.mark.parametrize("T,N,K", [(1, 300, 512), (129, 130, 1040), (256, 256, 2048), (257, 520, 4096), (600, 1300, 528)])
def test_pairs(monkeypatch, split, T, N, K):
    """Two CTAs per tile, its K on one to four pairs, whatever the number of tokens."""
    monkeypatch.setenv("MSA_LINEAR_SPLIT", str(split))
    monkeypatch.setenv("MSA_LINEAR_FORM", "pairs")
    for dtype, pad in ((torch.bfloat16, 0), (torch.float32, 5)):
        c = Case(T, N, K, dtype, seed=split, pad=pad)
        c.run()
        assert "pairs" in msa.last_dispatch() and msa.last_dispatch().endswith(f"split={split}")
        c.check()


@pytest.mark.parametrize("form,T", [("rows", 9), ("rows", 40), ("rows", 60), ("rows", 150), ("pairs", 300)])
@pytest.mark.parametrize("N", [1, 3, 4, 7, 8, 17, 127, 129, 130, 131, 255, 258, 300, 517])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_what_lies_behind_a_row(monkeypatch, dtype, N, form, T):
    """Rows that end anywhere in their last 16 bytes, at a stride of whole ones and at the next odd one."""
    monkeypatch.setenv("MSA_LINEAR_FORM", form)
    for pad in (-N % 8, -N % 8 + 8, 1):
        for split in (1, 2):
            monkeypatch.setenv("MSA_LINEAR_SPLIT", str(split))
            c = Case(T, N, 256, dtype, seed=N, pad=pad)
            c.run()
            assert msa.last_dispatch().split()[1] == form and msa.last_dispatch().endswith(f"split={split}")
            c.check()


@pytest.mark.parametrize("form,T,split", [("rows", 9, 2), ("rows", 150, 3), ("pairs", 300, 1), ("pairs", 300, 2), ("pairs", 300, 3)])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_scales_off_16_bytes(monkeypatch, off, form, T, split):
    """Scales need boundaries of four bytes alone, also where a row of them is a multiple of 16 bytes."""
    monkeypatch.setenv("MSA_LINEAR_FORM", form)
    monkeypatch.setenv("MSA_LINEAR_SPLIT", str(split))
    c = Case(T, 300, 1024, seed=off)
    for name in ("sa", "sw"):
        x = getattr(c, name)
        room = torch.full((x.numel() + 8,), float("nan"), device="cuda")
        room[off:off + x.numel()] = x.flatten()
        setattr(c, name, room[off:off + x.numel()].view(x.shape))
    c.run()
    assert msa.last_dispatch().split()[1] == form and msa.last_dispatch().endswith(f"split={split}")
    c.check()


@pytest.mark.parametrize("T", [130, 300])
def test_rows_form_with_many_tokens(monkeypatch, T):
    monkeypatch.setenv("MSA_LINEAR_FORM", "rows")
    c = Case(T, 300, 1040, seed=T)
    c.run()
    assert "rows" in msa.last_dispatch()
    c.check()


@pytest.mark.parametrize("T", [1, 20, 64, 200])
def test_long_k(T):
    """More blocks of K than one table of scales holds, on one CTA and shared."""
    c = Case(T, 256, 128 * 70 + 48, torch.float32, seed=T)
    c.run()
    c.check()


def test_rows_of_the_output_apart():
    for T, N, pad, dtype in ((5, 300, 20, torch.bfloat16), (70, 256, 3, torch.float32), (300, 130, 6, torch.bfloat16), (300, 256, 1, torch.bfloat16)):
        c = Case(T, N, 256, dtype, seed=pad, pad=pad)
        c.run()
        c.check()


@pytest.mark.parametrize("T", [3, 64, 300])
def test_zero_scales_and_nan_codes(T):
    c = Case(T, 260, 512, seed=8)
    c.sa[1] = 0.0
    c.sw[1, 2] = 0.0
    c.run()
    c.check()
    assert not c.out[1].any()
    c.a[2, 300] = 0x7F
    c.w[129, 7] = 0xFF
    c.run()
    bad = torch.zeros_like(c.out, dtype=torch.bool)
    bad[2], bad[:, 129] = True, True
    assert torch.equal(c.out.isnan(), bad)


def test_rows_do_not_see_one_another():
    """A request's output is the same bits whatever the other rows of the batch hold."""
    c = Case(48, 512, 2048, seed=9)
    c.run()
    first = c.out.clone()
    c.a[:20] = _codes(np.random.default_rng(10), 20, 2048).cuda()
    c.sa[:20] *= 3
    c.run()
    assert torch.equal(first[20:], c.out[20:]) and not torch.equal(first[:20], c.out[:20])


def test_large_sampled():
    """A prompt's chunk; sampled rows against the oracle."""
    c = Case(2049, 3200, 1024, seed=11)
    c.run()
    c.check(rows=torch.tensor([0, 1, 127, 128, 255, 256, 1023, 1900, 2046, 2047, 2048]))


@pytest.mark.parametrize("form,T", [("rows", 300), ("pairs", 300), ("rows", 75)])
def test_output_past_4_gib(monkeypatch, form, T):
    """Offsets of the output past 32 bits."""
    monkeypatch.setenv("MSA_LINEAR_FORM", form)
    N, K = 1_200_000_000 // T // 4096 * 4096, 16
    rng = np.random.default_rng(12)
    a = _codes(rng, T, K).cuda()
    w = _codes(rng, 4096, K).cuda().repeat(-(-N // 4096), 1)[:N].contiguous()
    sa, sw = torch.ones((T, 1), device="cuda"), torch.ones((-(-N // 128), 1), device="cuda")
    out, flags = torch.empty((T, N), dtype=torch.float32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.fp8_linear(a, sa, w, sw, out, flags)
    assert int(flags.item()) == 0
    for i in range(4096, N, 4096):                            # the weight repeats
        assert torch.equal(out[:, :4096], out[:, i:i + 4096]), i
    want, size = L.linear(a.cpu().numpy(), sa.cpu().numpy(), w[:4096].cpu().numpy(), sw[:32].cpu().numpy())
    assert (np.abs(out[:, :4096].double().cpu().numpy() - want) <= 200 * 2.0 ** -23 * size).all()


@pytest.mark.parametrize("T", [7, 64, 500])
def test_repeats_streams_and_graph(T):
    c = Case(T, 1000, 1536, seed=13)
    c.run()
    first = c.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.out.zero_()
        msa.fp8_linear(c.a, c.sa, c.w, c.sw, c.out, c.flags)
    side.synchronize()
    assert torch.equal(first, c.out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        msa.fp8_linear(c.a, c.sa, c.w, c.sw, c.out, c.flags)
    for _ in range(3):
        c.out.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, c.out) and int(c.flags.item()) == 0


@pytest.mark.parametrize("sizes", [((64, 2560, 2048), (64, 2560, 2048)), ((600, 2560, 2048), (9, 2560, 4096)),
                                   ((600, 2560, 2048), (700, 1280, 4096)), ((100, 4096, 4096), (64, 20480, 512))])
def test_two_calls_at_once(sizes):
    """Calls on two streams share nothing."""
    cs = [Case(*n, seed=14 + i) for i, n in enumerate(sizes)]
    for c in cs:
        c.run()
    want = [c.out.clone() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for c, s in zip(cs, streams):
            msa.fp8_linear(c.a, c.sa, c.w, c.sw, c.out, c.flags, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(w, c.out) for w, c in zip(want, cs))
