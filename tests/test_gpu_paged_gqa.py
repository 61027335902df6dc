"""Dense paged GQA decode against the fp64 attention (bounds: tests/paged.py)."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa

from paged import Case

pytestmark = pytest.mark.gpu

KV = ("bf16", "fp8", "nvfp4")


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("lens", [[1], [2], [127, 128, 129], [640, 1, 257], [5000], [128] * 5 + [4097]],
                         ids=lambda v: "-".join(map(str, v)))
def test_lengths(kind, lens):
    c = Case(lens, kind, seed=len(lens) + lens[0])
    c.run()
    c.check()


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("G,group", [(4, 16), (1, 8), (3, 5), (8, 1), (2, 12), (1, 16)])
@pytest.mark.parametrize("Q", [1, 2, 3, 8])
def test_head_layouts_and_positions(kind, G, group, Q):
    """Rows per KV head from 1 to 128; positions straddling a block edge; requests shorter than Q."""
    c = Case([1, Q, 130, 128 + Q // 2, 700], kind, G, group, Q, seed=G * 100 + group * 10 + Q)
    c.run()
    c.check()


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("Q", [1, 8])
def test_unused_places_and_bad_lengths(kind, Q):
    """Length 0: output 0 and lse -inf, no flag. Negative and too long: the same, flagged."""
    c = Case([0, 300, 0, 0, 129, 0], kind, Q=Q, seed=3)
    c.run()
    c.check()
    c.lens_d[0], c.lens_d[2] = -5, c.NB * 128 + 1
    c.out.fill_(float("nan"))
    c.run()
    c.check(flags=msa.FLAG_BAD_SEQLEN)


def test_only_unused_places():
    c = Case([0, 0, 0], "bf16", seed=4)
    c.run()
    c.check()


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_bad_page_is_skipped_and_flagged(kind, bad):
    c = Case([900, 513], kind, seed=5)
    c.table_d[0, 3] = bad
    c.table_d[1, 4] = bad                            # the last, partial block
    c.run()
    c.check(live_blocks={0: [0, 1, 2, 4, 5, 6, 7], 1: [0, 1, 2, 3]}, flags=msa.FLAG_BAD_PAGE)


@pytest.mark.parametrize("kind", KV)
def test_every_page_bad(kind):
    c = Case([200], kind, seed=6)
    c.table_d.fill_(-7)
    c.run()
    c.check(live_blocks={0: []}, flags=msa.FLAG_BAD_PAGE)


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("shape", ["rising", "falling", "one", "far"])
def test_running_maximum(kind, shape):
    """Logits that rise or fall over the length, one token that outweighs the others by far, and maxima
    hundreds of powers of two apart between blocks."""
    def fn(x, b):
        t = np.arange(len(x), dtype=np.float32)[:, None, None]
        n = max(len(x) - 1, 1)
        f = {"rising": 3 * t / n, "falling": 3 * (1 - t / n), "one": np.where(t == n // 2, 5.0, 0.01),
             "far": np.where((t // 128) % 2 == 0, 0.02, 6.0)}[shape]
        return (x * f).astype(np.float32)

    c = Case([1500, 300], kind, seed=7, q_scale=8.0, k_fn=fn)
    c.run()
    c.check()


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -100, 2.0 ** -20, 2.0 ** 20])
def test_query_magnitudes(kind, q_scale):
    c = Case([200, 129], kind, seed=8, q_scale=q_scale, scale=1.0 / (128 ** 0.5 * max(q_scale, 1.0)))
    c.run()
    c.check()


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("group,Q", [(16, 1), (8, 4), (16, 8)])
def test_more_rows_than_ctas_and_split_rows(kind, group, Q):
    """Many short rows (several per CTA) beside one that every CTA shares."""
    c = Case([130] * 90 + [30000, 64], kind, 2, group, Q, seed=9)
    c.run()
    c.check(which=[0, 45, 89, 90, 91])


@pytest.mark.parametrize("kind", KV)
def test_repeats_are_bit_identical(kind):
    """Joins run in a fixed order, so repeated calls give the same bits."""
    c = Case([4000, 77, 9000], kind, seed=10)
    c.run()
    torch.cuda.synchronize()
    first = (c.out.clone(), c.lse.clone())
    for _ in range(10):
        c.run()
    torch.cuda.synchronize()
    assert torch.equal(first[0].view(torch.int16), c.out.view(torch.int16)) and torch.equal(first[1], c.lse)
    c.check()


@pytest.mark.parametrize("kind", KV)
def test_captured_graph_serves_changing_lengths(kind):
    """One graph, replayed while the lengths in its buffer change; another graph and a direct call with workspaces of
    their own in between."""
    c = Case([1000, 600], kind, seed=11)
    other = Case([2000], kind, seed=12)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c.run()
        other.run()
    stream.synchronize()
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c.run()
    with torch.cuda.graph(graph2, stream=stream):
        other.run()
    full_k, full_v = list(c.K), list(c.V)
    for lens in ([1000, 600], [1, 599], [0, 256], [900, 0], [1000, 600]):
        c.lens = lens
        c.lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        c.K, c.V = [k[:n] for k, n in zip(full_k, lens)], [v[:n] for v, n in zip(full_v, lens)]
        c.out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        graph2.replay()
        c.check()
        other.check()


def test_one_workspace_for_calls_in_turn():
    """Calls of other formats, rows and lengths take turns on one workspace, with anything written to it in between."""
    cases = [Case([5000], "bf16", 1, 16, seed=20), Case([9000, 300], "fp8", 2, 8, 3, seed=21), Case([700] * 9, "nvfp4", 4, seed=22),
             Case([20000], "fp8", 1, 16, 8, seed=23), Case([3000, 4000], "bf16", 1, 16, 8, seed=24), Case([30000], "nvfp4", 1, 4, seed=25)]
    ws = torch.empty(max(c.ws.numel() for c in cases), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(3)
    for turn in range(3):
        for i in rng.permutation(len(cases)):
            c = cases[i]
            c.ws = ws
            c.out.fill_(float("nan"))
            for _ in range(1 + turn):
                c.run()
            c.check(which=range(1))
            if turn == 1:
                ws.random_(0, 256)
            elif turn == 2:
                ws.zero_()


@pytest.mark.parametrize("kind", KV)
def test_two_streams_at_once(kind):
    cases = [Case([3000, 10], kind, seed=13), Case([128, 4000], kind, Q=4, group=8, seed=14)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    for c in cases:
        c.check()


def test_lse_may_be_left_out():
    c = Case([333], "bf16", seed=15)
    msa.paged_gqa_decode(c.dims, c.q, c.cache, c.table_d, c.lens_d, c.out, None, c.ws, c.flags)
    c.lse.copy_(torch.from_numpy(c.expected(0)[1]).float())
    c.check()


def test_largest_batch():
    """4,096 requests, most of them unused places or a single block."""
    lens = [(i * 37) % 150 for i in range(4096)]
    c = Case(lens, "fp8", 1, 8, seed=16)
    c.run()
    c.check(which=[0, 1, 2, 100, 2047, 2048, 4095])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_offsets_past_32_bits(kind):
    """The last pages of a cache whose K lies past 4 GiB."""
    import paged
    c = Case([400, 129], kind, seed=17)
    row = 2 if kind == "bf16" else 1
    P = 2 ** 32 // (4 * 128 * 128 * row) + c.P + 8
    big = []
    for t in (c.cache.k, c.cache.v):
        x = torch.empty((P,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda")
        x[P - c.P:] = t
        big.append(x)
    c.cache.k, c.cache.v = big
    c.table_d = torch.where(c.table_d >= 0, c.table_d + (P - c.P), c.table_d)
    c.dims.num_pages = P
    c.run()
    c.check()
    assert paged.BS == 128


@pytest.mark.parametrize("seed", range(24))
def test_random_steps(seed):
    rng = np.random.default_rng(1000 + seed)
    kind = KV[seed % 3]
    G, group, Q = int(rng.choice([1, 2, 3, 4, 8])), int(rng.integers(1, 17)), int(rng.integers(1, 9))
    B = int(rng.integers(1, 24))
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(3000), B))]
    for i in rng.integers(0, B, B // 6):
        lens[i] = 0
    c = Case(lens, kind, G, group, Q, seed=seed)
    c.run()
    c.check(which=range(min(B, 6)))


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("Q", [1, 8])
def test_few_requests_in_a_large_batch(kind, Q):
    """Two live requests among 4,094 unused places, at the front, apart, and at the end."""
    for at in ([0, 1], [5, 3000], [4094, 4095]):
        lens = [0] * 4096
        lens[at[0]], lens[at[1]] = 700, 300
        c = Case(lens, kind, 1, 16, Q, seed=26)
        c.run()
        c.check(which=at + [2, 4000])


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("G,group,Q", [(4, 16, 1), (1, 8, 2), (3, 5, 1), (8, 1, 8), (2, 1, 1)])
def test_wide_block_table(kind, G, group, Q):
    """A table with room for a million tokens per request; short and empty requests in it."""
    c = Case([1, 700, 0, 128, 2049, -3, 129], kind, G, group, Q, seed=27, cols_extra=8192)
    c.run()
    c.check(which=[0, 1, 2, 3, 4, 6], flags=msa.FLAG_BAD_SEQLEN)


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -100, 2.0 ** 20])
def test_wide_block_table_query_magnitudes(kind, q_scale):
    c = Case([300, 900], kind, 2, 8, 1, seed=28, q_scale=q_scale, scale=2.0 ** -20 if q_scale > 1 else None,
             cols_extra=8192)
    c.run()
    c.check()


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("Q", [1, 2, 8])
def test_bad_pages_while_page_0_was_never_written(kind, Q):
    """The kernels put page 0 in a bad page's place; what it holds must not matter."""
    c = Case([900, 300, 128], kind, Q=Q, seed=29)
    table = c.table.copy()
    table[0, 2], table[1, 2] = c.P, -1
    table[table == 0] = 2 ** 31 - 1
    for t, fill in ((c.cache.k, 0xFF), (c.cache.v, 0xFF), (c.cache.k_scale, 0x7F), (c.cache.v_scale, 0x7F)):
        if t is not None:
            t[0].view(torch.uint8).fill_(fill)
    c.table_d.copy_(torch.from_numpy(table))
    c.run()
    nb = [8, 3, 1]
    live = {b: [i for i in range(nb[b]) if 0 < table[b, i] < c.P] for b in range(3)}
    c.check(live_blocks=live, flags=msa.FLAG_BAD_PAGE)


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -100, 2.0 ** -20, 2.0 ** 20])
def test_query_magnitudes_with_many_rows(kind, q_scale):
    c = Case([200, 129], kind, G=2, Q=4, seed=30, q_scale=q_scale, scale=1.0 / (128 ** 0.5 * max(q_scale, 1.0)))
    c.run()
    c.check()


@pytest.mark.parametrize("kind", ["fp8", "nvfp4"])
@pytest.mark.parametrize("Q", [1, 2, 4])
def test_logits_too_small_for_fp32(kind, Q):
    """Queries of 2^-60 over keys of 1e-30: their factors' product underflows; the attention is the plain mean."""
    c = Case([200, 129, 1], kind, G=2, Q=Q, seed=31, q_scale=2.0 ** -60)
    was, c.cache.k_global = c.cache.k_global, 1e-30
    c.K = [k * (1e-30 / was) for k in c.K]
    c.run()
    c.check()


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("Q,wide", [(1, False), (1, True), (2, False), (4, False)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_queries_that_are_no_numbers(kind, Q, wide, bad):
    """A head whose query holds a NaN or an infinity: NaN there, the other heads bit for bit as without it."""
    c = Case([3000, 128, 70], kind, G=2, Q=Q, seed=32, cols_extra=8192 if wide else 1)
    c.run()
    torch.cuda.synchronize()
    out, lse = c.out.clone(), c.lse.clone()
    hit = torch.zeros_like(lse, dtype=torch.bool)
    for b, j, h, d in ((0, 0, 3, 0), (0, Q - 1, 17, 127), (1, 0, 31, 64), (2, Q - 1, 0, 5)):
        c.q[b, j, h, d] = bad
        hit[b, j, h] = True
    c.run()
    torch.cuda.synchronize()
    assert torch.isnan(c.out[hit]).all() and torch.isnan(c.lse[hit]).all()
    assert torch.equal(c.out[~hit], out[~hit]) and torch.equal(c.lse[~hit], lse[~hit])


@pytest.mark.parametrize("kind", KV)
@pytest.mark.parametrize("Q,wide", [(1, False), (1, True), (2, False), (4, False)])
def test_keys_that_are_no_numbers(kind, Q, wide):
    """A NaN in a live key: NaN for the heads of that KV head, the others bit for bit as without it."""
    c = Case([3000, 128], kind, G=2, Q=Q, seed=33, cols_extra=8192 if wide else 1)
    c.run()
    torch.cuda.synchronize()
    out, lse = c.out.clone(), c.lse.clone()
    store = (c.cache.k_scale if kind == "nvfp4" else c.cache.k).view(torch.uint8)
    for b, t in ((0, 1500), (1, 0)):
        store[int(c.table[b, t // 128]), 1, t % 128, 2:4] = 0x7F if kind != "bf16" else 0xFF
    c.run()
    torch.cuda.synchronize()
    assert torch.isnan(c.out[:, :, 16:]).all() and torch.isnan(c.lse[:, :, 16:]).all()
    assert torch.equal(c.out[:, :, :16], out[:, :, :16]) and torch.equal(c.lse[:, :, :16], lse[:, :, :16])
