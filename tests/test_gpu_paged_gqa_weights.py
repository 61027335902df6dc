"""Dense paged GQA decode, the V side: weights of every size reach the output, from the block they belong to.

All values of V here are at least 0, so that the sum of softmax_t |v_t| is the output itself and every bound is relative
to it, with u(t) half a step of a type (bf16 2^-8, f16 2^-11, fp32 2^-24) and n the tokens seen:
  * the output's rounding to bf16: 2^-8;
  * a weight's rounding: bf16 caches 2^-8. FP8 and NVFP4 caches: 2^-11 as an f16 that is held times 2^7, whose
    subnormal half-step is 2^-25: 2^-32 of the largest weight, absolute; the three 8-bit parts that FP8 caches split it
    into add half a step of the last one, 2^-17 held times 2^7 * 2^7: 2^-31. Together under 2^-30 of the largest weight;
  * the exponential: 2^-21; the logits move a weight by twice their own error (numerator and denominator);
  * logits: 132 * 2^-24 * scale * max_t sum_d |q_d k_td|, and, for queries held as two 8-bit parts, 2^-22 of the row's
    largest value per dim (128 dims): 2^-22 * scale * max|q| * max_t sum_d |k_td|;
  * fp32 sums of n terms, two of them (numerator, denominator): 2 n * 2^-24."""
import numpy as np
import pytest
import torch

from paged import BS, D, Case, encode

pytestmark = pytest.mark.gpu

# cache type, query heads per KV head, positions, wide block table: one line per form of the kernel
FORMS = [("bf16", 16, 1, False), ("bf16", 16, 1, True), ("bf16", 8, 4, False),
         ("fp8", 16, 1, False), ("fp8", 16, 2, False), ("fp8", 16, 4, False),
         ("nvfp4", 16, 1, False), ("nvfp4", 16, 2, False), ("nvfp4", 16, 4, False)]


def put(c, name, b, x):
    """Replaces request b's K or V by x [tokens, G, D] (fp32), in the cache and in the expected values."""
    code, scales, val = encode(c.kind, x)
    store, sc = getattr(c.cache, name), getattr(c.cache, name + "_scale")
    for t0 in range(0, len(x), BS):
        page, m = int(c.table[b, t0 // BS]), min(BS, len(x) - t0)
        a = torch.from_numpy(np.ascontiguousarray(code[t0:t0 + m].transpose(1, 0, 2)).view(np.int16 if c.kind == "bf16" else np.uint8))
        store[page, :, :m] = (a.view(torch.bfloat16) if c.kind == "bf16" else a).cuda()
        if sc is not None:
            sc[page, :, :m] = torch.from_numpy(np.ascontiguousarray(scales[t0:t0 + m].transpose(1, 0, 2))).cuda()
    (c.K if name == "k" else c.V)[b] = val


def logit_error(c, b, q):
    """Bound of a logit's error, per head: q [H, D]."""
    G, n = c.G, c.group
    ds = np.zeros(len(q))
    for g in range(G):
        a, K = np.abs(q[g * n:(g + 1) * n]), np.abs(c.K[b][:, g])
        ds[g * n:(g + 1) * n] = 132 * 2.0 ** -24 * c.scale * (a @ K.T).max(1)
        if c.kind != "bf16":
            ds[g * n:(g + 1) * n] += 2.0 ** -22 * c.scale * a.max(1) * K.sum(1).max()
    return ds[:, None]


def check(c, b, got, glse):
    """got [Q, H, D], glse [Q, H] of a request with request b's tokens and queries."""
    out, lse, A, _, cnt = c.expected(b)
    vmax = c.V[b].max()
    for j in range(c.Q):
        n, ds = cnt[j], logit_error(c, b, c.q_val[b, j])
        assert np.array_equal(A[j], out[j])                                # V is not negative
        # the largest weight is at most e^(largest logit - lse) <= 1
        rel = 2.0 ** -8 + (2.0 ** -8 if c.kind == "bf16" else 2.0 ** -11) + 2.0 ** -21 + 2 * ds + 2 * n * 2.0 ** -24
        lim = out[j] * rel * (1 + 2.0 ** -6) + (0.0 if c.kind == "bf16" else n * 2.0 ** -30 * vmax)
        err = np.abs(got[j] - out[j])
        assert (err <= lim).all(), f"position {j}: output off by {(err / lim).max():.3g}x its bound"
        llim = ds[:, 0] + 2.0 ** -21 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(lse[j])
        assert (np.abs(glse[j] - lse[j]) <= llim).all(), f"position {j}: lse"


def results(c):
    torch.cuda.synchronize()
    assert int(c.flags.item()) == 0
    return c.out.double().cpu().numpy(), c.lse.double().cpu().numpy()


@pytest.mark.parametrize("kind,group,Q,wide", FORMS)
@pytest.mark.parametrize("lens", [[30000, 129], [2000, 5, 777, 4096]], ids=lambda v: "-".join(map(str, v)))
def test_every_block_adds_its_own_values(kind, group, Q, wide, lens):
    """Block i has large values in dims i mod 64 and 64 + (i / 64) mod 64 and small ones elsewhere: a block left out,
    taken twice or taken from another place moves those dims by several per cent."""
    c = Case(lens, kind, 2, group, Q, seed=40, cols_extra=8192 if wide else 1)
    rng = np.random.default_rng(41)
    for b, n in enumerate(lens):
        v = rng.uniform(0.0, 0.05, (n, 2, D)).astype(np.float32)
        for t0 in range(0, n, BS):
            i = t0 // BS
            v[t0:t0 + BS, :, i % 64] += 2.0 + 0.25 * (i % 5)
            v[t0:t0 + BS, :, 64 + i // 64 % 64] += 1.0 + 0.25 * (i % 7)
        put(c, "v", b, v)
    c.run()
    out, lse = results(c)
    for b in range(len(lens)):
        check(c, b, out[b], lse[b])


def shared_pages(c, copies):
    """Makes c a batch of `copies` requests that all read request 0's pages (a shared prompt), with its queries."""
    from block_sparse_attention_07_gb300 import msa
    c.dims.batch = copies
    c.q = c.q[:1].expand(copies, -1, -1, -1).contiguous()
    c.table_d = c.table_d[:1].expand(copies, -1).contiguous()
    c.lens_d = c.lens_d[:1].expand(copies).contiguous()
    c.out = torch.full((copies,) + tuple(c.out.shape[1:]), float("nan"), dtype=c.out.dtype, device="cuda")
    c.lse = torch.full((copies,) + tuple(c.lse.shape[1:]), float("nan"), device="cuda")
    c.ws = torch.empty(msa.paged_gqa_workspace_size(c.dims, c.cache.dtype), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("kind,group,Q,wide", FORMS)
@pytest.mark.parametrize("nats", [8.0, 14.0, 15.5, 17.0])
@pytest.mark.parametrize("even", [True, False])
def test_many_small_weights_beside_a_large_one(kind, group, Q, wide, nats, even):
    """One token whose logit lies `nats` above those of 4,000 others, and whose V is 0: the output is the others' sum.
    The others' logits are equal, or spread over half a unit. Whole rows lie inside one CTA (300 of them)."""
    n = 4000
    c = Case([n], kind, 1, group, Q, seed=42, q_scale=0.0, cols_extra=8192 if wide else 1)
    rng = np.random.default_rng(43)
    q = np.full(c.q_val.shape, nats / (c.scale * D), dtype=np.float32)
    c.q = torch.from_numpy(q).to(torch.bfloat16).cuda()
    c.q_val = c.q.double().cpu().numpy()
    k = np.zeros((n, 1, D), dtype=np.float32)
    if not even:
        k += rng.uniform(-0.25, 0.25, (n, 1, 1)).astype(np.float32) / nats
    k[5] = 1.0
    v = rng.uniform(0.5, 1.0, (n, 1, D)).astype(np.float32)
    v[5] = 0.0
    put(c, "k", 0, k)
    put(c, "v", 0, v)
    shared_pages(c, 300)
    c.run()
    out, lse = results(c)
    for b in (0, 1, 2, 77, 150, 298, 299):
        check(c, 0, out[b], lse[b])


@pytest.mark.parametrize("kind,group,Q,wide", FORMS)
def test_queries_with_one_large_dim(kind, group, Q, wide):
    """A query value 2^9 to 2^11 times the others', in a dim where the keys are 0: the others decide, with all the bits
    they have (8; the last one set). One token, so that lse is the logit."""
    c = Case([1, 300], kind, 2, group, Q, seed=44)
    h = np.arange(c.q_val.shape[2])
    q = np.empty(c.q_val.shape, dtype=np.float32)
    q[...] = (1 + 2.0 ** -7 * (1 + 2 * (h % 8)))[:, None]
    q[..., 0] = 2.0 ** (9 + h // 2 % 3)
    c.q = torch.from_numpy(q).to(torch.bfloat16).cuda()
    c.q_val = c.q.double().cpu().numpy()
    rng = np.random.default_rng(46)
    for b, n in enumerate(c.lens):
        k = rng.uniform(0.5, 1.0, (n, 2, D)).astype(np.float32)
        k[..., 0] = 0.0
        put(c, "k", b, k)
        put(c, "v", b, rng.uniform(0.5, 1.0, (n, 2, D)).astype(np.float32))
    c.run()
    out, lse = results(c)
    j = Q - 1                                              # (a request of one token has it at its last position)
    ds = logit_error(c, 0, c.q_val[0, j])[:, 0]
    want = np.concatenate([c.scale * c.q_val[0, j, g * group:(g + 1) * group] @ c.K[0][0, g] for g in range(2)])
    assert (np.abs(lse[0, j] - want) <= ds + 2.0 ** -21 + 2.0 ** -22 * np.abs(want)).all()
    check(c, 1, out[1], lse[1])
