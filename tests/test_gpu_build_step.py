"""Step metadata on the GPU against the token-by-token oracle: whole numbers, so equal."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa
from oracle import step as ostep

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, ctx, new, NB, free_extra=5, head=0, T=None, axes=1, offset=False, seed=0, F=None, pages=None,
                 pos_pad=0):
        rng = np.random.default_rng(seed)
        B = len(ctx)
        used = [min(-(-max(c, 0) // 128), NB) for c in ctx]
        need = sum(max(0, -(-(c + n) // 128) - -(-c // 128)) for c, n in zip(ctx, new) if c >= 0 and n >= 0)
        F = head + need + free_extra if F is None else F
        self.P = sum(used) + F if pages is None else pages
        perm = rng.permutation(sum(used) + F).astype(np.int32)
        table = rng.integers(-9, -1, (B, NB)).astype(np.int32)        # columns that nothing may touch
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = perm[at:at + u]
            at += u
        self.ctx, self.new, self.table, self.free = np.array(ctx), np.array(new), table, perm[at:]
        self.head, self.axes = head, axes
        self.T = sum(max(n, 0) for n in new) if T is None else T
        self.offset = rng.integers(-600, 5, B).astype(np.int32) if offset else None
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
        self.d = dict(ctx=i32(ctx), new=i32(new), free=i32(self.free), head=i32([head]), table=i32(table),
                      seq=torch.full((B,), -77, dtype=torch.int32, device="cuda"),
                      starts=torch.full((B + 1,), -77, dtype=torch.int32, device="cuda"),
                      slots=torch.full((self.T,), -77, dtype=torch.int64, device="cuda"),
                      pos=torch.full((axes, self.T + pos_pad), -77, dtype=torch.int32, device="cuda"),
                      out=torch.full((1,), -77, dtype=torch.int32, device="cuda"),
                      off=i32(self.offset) if offset else None)
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dims = msa.make_dims(B, 1, max_blocks_per_seq=NB, num_pages=self.P)

    def run(self, stream=None, prepare=False):
        d = self.d
        return msa.build_step(self.dims, d["ctx"], d["new"], d["free"], d["head"], d["table"], d["seq"], d["starts"],
                              d["slots"], d["pos"][:, :self.T], d["out"], self.flags, pos_offset=d["off"],
                              stream=stream, prepare=prepare)

    def check(self):
        torch.cuda.synchronize()
        w = ostep.build_step(self.ctx, self.new, self.free, self.head, self.table, self.P, self.T, self.axes, self.offset)
        got = {k: None if v is None else v.cpu().numpy() for k, v in self.d.items()}
        assert np.array_equal(got["table"], w["table"])
        assert np.array_equal(got["seq"], w["seq_lens"])
        assert np.array_equal(got["starts"], w["token_starts"])
        assert np.array_equal(got["slots"], w["slots"])
        assert np.array_equal(got["pos"][:, :self.T], w["positions"])
        assert (got["pos"][:, self.T:] == -77).all()
        assert int(got["out"][0]) == w["free_head"]
        assert int(self.flags.item()) == w["flags"]
        return w


@pytest.mark.parametrize("ctx,new", [
    ([0], [1]), ([127], [1]), ([128], [1]), ([0, 0, 0], [0, 5, 0]), ([5, 128, 255, 0], [1, 1, 1, 1]),
    ([100, 0, 3], [1000, 129, 128]), ([4095] * 7, [8] * 7), ([0], [5000])])
@pytest.mark.parametrize("axes", [1, 3])
def test_lengths(ctx, new, axes):
    s = Step(ctx, new, NB=48, axes=axes, offset=axes > 1, head=2)
    s.run()
    assert s.check()["flags"] == 0


@pytest.mark.parametrize("pad", [1, 2, 3, 4, 777, 5000])
def test_padding_tokens(pad):
    s = Step([200, 0, 31], [7, 300, 1], NB=8, T=308 + pad, axes=4, pos_pad=pad % 3)
    s.run()
    assert s.check()["flags"] == 0


@pytest.mark.parametrize("B", [255, 256, 257, 1000, 4096])
def test_large_batches(B):
    rng = np.random.default_rng(B)
    ctx, new = rng.integers(0, 3000, B), rng.integers(0, 40, B)
    s = Step(ctx.tolist(), new.tolist(), NB=26, T=int(new.sum()) + 17, offset=True, seed=B)
    s.run()
    assert s.check()["flags"] == 0


def test_free_list_runs_out():
    """Requests from the first that does not fit on get no pages; those that need none still run."""
    s = Step([0, 100, 128, 5, 127], [300, 1, 200, 1, 1], NB=8, head=1, F=5)
    s.run()
    w = s.check()
    assert w["flags"] == msa.FLAG_NO_PAGES and w["seq_lens"].tolist() == [300, 101, 128, 6, 128]


@pytest.mark.parametrize("head", [-1, 9])
def test_free_head_out_of_range(head):
    s = Step([0, 100], [3, 1], NB=4, F=6)
    s.head = head
    s.d["head"].fill_(head)
    s.run()
    assert s.check()["flags"] == msa.FLAG_NO_PAGES


def test_bad_lengths():
    s = Step([-3, 10, 500, 1000, 0], [2, -4, 600, 30, 3], NB=8)
    s.run()
    assert s.check()["flags"] == msa.FLAG_BAD_SEQLEN


def test_more_tokens_than_places():
    s = Step([0, 10, 20], [100, 50, 3], NB=8, T=120)
    s.run()
    w = s.check()
    assert w["flags"] == msa.FLAG_BAD_SEQLEN and w["token_starts"].tolist() == [0, 100, 120, 120]


def test_huge_lengths_do_not_overflow():
    big = 2 ** 31 - 1
    s = Step([big, big, 4], [big, big, 2], NB=4, T=64, F=3, pages=100)
    s.run()
    assert s.check()["flags"] == msa.FLAG_BAD_SEQLEN


def test_bad_pages():
    s = Step([100, 0, 300], [60, 300, 1], NB=8)
    s.free[1] = s.P + 4
    s.d["free"][1] = s.P + 4
    s.table[2, 2] = -1                                    # the cached part's last block
    s.d["table"][2, 2] = -1
    s.run()
    assert s.check()["flags"] == msa.FLAG_BAD_PAGE


def test_steps_in_turn_on_the_device():
    """Two captured steps that hand lengths and the free list's head to each other, replayed."""
    B, NB, steps = 3, 6, 40
    ctx0 = [3, 120, 250]
    s = Step(ctx0, [1] * B, NB=NB, free_extra=16)
    a = s.d
    seq2, out2 = torch.empty_like(a["seq"]), torch.empty_like(a["out"])
    ctx = a["ctx"]

    def two():
        args = (a["starts"], a["slots"], a["pos"])
        msa.build_step(s.dims, ctx, a["new"], a["free"], a["head"], a["table"], seq2, *args, out2, s.flags)
        msa.build_step(s.dims, seq2, a["new"], a["free"], out2, a["table"], a["seq"], *args, a["out"], s.flags)
        ctx.copy_(a["seq"])
        a["head"].copy_(a["out"])

    keep = (ctx.clone(), a["table"].clone(), a["head"].clone())
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        two()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        two()
    for t, k in zip((ctx, a["table"], a["head"]), keep):
        t.copy_(k)
    for _ in range(steps // 2):
        graph.replay()
    torch.cuda.synchronize()
    table, head, lens = s.table.copy(), 0, list(ctx0)
    for _ in range(steps):
        w = ostep.build_step(lens, [1] * B, s.free, head, table, s.P, B)
        table, head, lens = w["table"], w["free_head"], w["seq_lens"].tolist()
    assert np.array_equal(a["table"].cpu().numpy(), table) and a["seq"].tolist() == lens
    assert np.array_equal(a["slots"].cpu().numpy(), w["slots"]) and int(a["head"].item()) == head
    assert int(s.flags.item()) == 0


@pytest.mark.parametrize("seed", range(12))
def test_random_steps(seed):
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 60))
    ctx = rng.integers(-2 if seed % 4 == 0 else 0, 1200, B)
    new = rng.integers(-1 if seed % 4 == 1 else 0, int(rng.integers(2, 400)), B)
    s = Step(ctx.tolist(), new.tolist(), NB=int(rng.integers(8, 16)), head=int(rng.integers(0, 4)),
             T=int(max(1, np.maximum(new, 0).sum() + rng.integers(-20 if seed % 3 == 0 else 0, 50))),
             axes=int(rng.integers(1, 5)), offset=bool(seed % 2), seed=seed,
             F=int(rng.integers(4, 200)) if seed % 4 == 3 else None)
    s.run()
    s.check()
