"""The full-attention layer's calls refuse tensors whose addresses their kernels must not get. CPU only: nothing launches."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    from block_sparse_attention_07_gb300 import _build
    _build.build()
    from block_sparse_attention_07_gb300 import msa
    return msa


class Fake:
    """A tensor as the checks see it, on a device of the test's choice."""

    def __init__(self, t, device):
        self.t, self.device = t, torch.device(device)

    def __getattr__(self, name):
        return getattr(self.t, name)


def z(*shape, dt=torch.int32):
    return torch.zeros(shape, dtype=dt)


def calls(m):
    """name -> (function of the arguments, arguments): every tensor on the CPU."""
    bf, u8 = torch.bfloat16, torch.uint8
    d = m.make_dims(2, 1, max_blocks_per_seq=4, num_pages=8)
    step = dict(ctx_lens=z(2), new_lens=z(2), free_pages=z(4), free_head=z(1), block_table=z(2, 4), seq_lens=z(2),
                token_starts=z(3), slot_mapping=z(8, dt=torch.int64), positions=z(3, 8), free_head_out=z(1), flags=z(1),
                pos_offset=z(2))
    gqa = dict(q=z(2, 1, 64, 128, dt=bf), k=z(8, 4, 128, 64, dt=u8), v=z(8, 4, 128, 64, dt=u8), k_scale=z(8, 4, 128, 8, dt=u8),
               v_scale=z(8, 4, 128, 8, dt=u8), block_table=z(2, 4), seq_lens=z(2), out=z(2, 1, 64, 128, dt=bf),
               lse=z(2, 1, 64, dt=torch.float32), workspace=z(m.paged_gqa_workspace_size(d, m.NVFP4), dt=u8), flags=z(1))
    rope = dict(q=z(3, 64, 128, dt=bf), k=z(3, 4, 128, dt=bf), v=z(3, 4, 128, dt=bf), idx_q=z(3, 4, 128, dt=bf),
                idx_k=z(3, 4, 128, dt=bf), positions=z(3, 3), slot_mapping=z(3, dt=torch.int64), q_out=z(3, 64, 128, dt=bf),
                idx_q_out=z(3, 4, 128, dt=bf), k_cache=z(8, 4, 128, 128, dt=u8), v_cache=z(8, 4, 128, 128, dt=u8),
                idx_keys=z(8, 4, 128, 128, dt=u8), idx_scale=z(8, 4, 128, dt=torch.float32), flags=z(1))
    weights = {n: z(128, dt=torch.float32) for n in ("wq", "wk", "wiq", "wik")}
    rope.update(weights)

    def run_gqa(k, v, k_scale, v_scale, **a):
        m.paged_gqa_decode(d, cache=m.KVCache(m.NVFP4, k, v, k_scale, v_scale), **a)

    def run_rope(k_cache, v_cache, idx_keys, idx_scale, wq, wk, wiq, wik, **a):
        m.qk_norm_mrope_insert(d, nr=m.make_norm_rope(wq, wk, wiq, wik), axes=m.make_rope_axes((16, 24, 24)),
                               cache=m.KVCache(m.FP8_E4M3, k_cache, v_cache),
                               idx_cache=m.IndexCache(m.FP8_E4M3, idx_keys, idx_scale), **a)

    return {"step": (lambda **a: m.build_step(d, **a), step), "gqa": (run_gqa, gqa), "rope": (run_rope, rope)}


HELD = {"step": ("ctx_lens", "new_lens", "free_pages", "free_head", "block_table", "seq_lens", "token_starts", "slot_mapping",
                 "positions", "free_head_out", "pos_offset", "flags"),
        "gqa": ("q", "k", "v", "k_scale", "v_scale", "block_table", "seq_lens", "out", "lse", "workspace", "flags"),
        "rope": ("q", "k", "v", "idx_q", "idx_k", "positions", "slot_mapping", "q_out", "idx_q_out", "k_cache", "v_cache",
                 "idx_keys", "idx_scale", "wq", "wk", "wiq", "wik", "flags")}


@pytest.mark.parametrize("call", sorted(HELD))
@pytest.mark.parametrize("where", ["cpu", "cuda:1"])
def test_tensors_off_the_current_gpu(m, monkeypatch, call, where):
    """One tensor in host memory, or on another GPU than the current one, the others where they belong."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m, "_stream", lambda stream: None)
    run, args = calls(m)[call]
    reached = []
    monkeypatch.setattr(m, "_call", lambda *a: reached.append(a[3]))
    run(**{n: Fake(t, "cuda:0") for n, t in args.items()})
    assert len(reached) == 1                                       # all of them in place: the call is made
    for name in HELD[call]:
        with pytest.raises(m.MSAError) as e:
            run(**{n: Fake(t, where if n == name else "cuda:0") for n, t in args.items()})
        assert e.value.status == m.ERR_INVALID_ARG and "device" in str(e.value), name
    assert len(reached) == 1


@pytest.mark.parametrize("call", sorted(HELD))
def test_host_tensors_reach_no_kernel(m, monkeypatch, call):
    run, args = calls(m)[call]
    monkeypatch.setattr(m, "_call", lambda *a: pytest.fail("the call was made"))
    with pytest.raises(m.MSAError) as e:
        run(**args)
    assert e.value.status == m.ERR_INVALID_ARG


@pytest.mark.parametrize("call,name,bad", [
    ("step", "flags", z(1, dt=torch.int64)), ("step", "flags", z(0)), ("gqa", "flags", z(1, dt=torch.uint8)),
    ("gqa", "flags", z(8)[::2]), ("rope", "flags", z(1, dt=torch.float32)),
    ("gqa", "workspace", z(1 << 24, dt=torch.uint8)[::2]),
    ("rope", "wq", z(128, dt=torch.bfloat16)), ("rope", "wk", z(64, dt=torch.float32)),
    ("rope", "wiq", z(256, dt=torch.float32)[::2]), ("rope", "wik", z(1, 128, dt=torch.float32)),
    ("rope", "idx_keys", z(8, 4, 128, 64, dt=torch.uint8)), ("rope", "idx_keys", z(4, 4, 128, 128, dt=torch.uint8)),
    ("rope", "idx_scale", z(8, 4, 128, dt=torch.bfloat16)), ("rope", "idx_scale", z(8, 4, 64, dt=torch.float32)),
    ("rope", "idx_scale", None)])
def test_wrong_flags_workspaces_weights_and_index_caches(m, monkeypatch, call, name, bad):
    """Everything on the GPU, one argument of another type, length or layout than the kernel takes it for."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m, "_stream", lambda stream: None)
    monkeypatch.setattr(m, "_call", lambda *a: pytest.fail("the call was made"))
    run, args = calls(m)[call]
    with pytest.raises(m.MSAError) as e:
        run(**{n: None if (t := bad if n == name else a) is None else Fake(t, "cuda:0") for n, a in args.items()})
    assert e.value.status == m.ERR_INVALID_ARG


def test_nvfp4_index_cache(m, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m, "_stream", lambda stream: None)
    made = []
    monkeypatch.setattr(m, "_call", lambda *a: made.append(a[3]))
    _, args = calls(m)["rope"]
    a = {n: Fake(t, "cuda:0") for n, t in args.items() if not n.startswith(("w", "idx_keys", "idx_scale", "k_cache", "v_cache"))}
    f = lambda *s, dt=torch.uint8: Fake(z(*s, dt=dt), "cuda:0")
    w = [f(128, dt=torch.float32) for _ in range(4)]
    d = m.make_dims(2, 1, max_blocks_per_seq=4, num_pages=8)
    for keys, scales, status in ((f(8, 4, 128, 64), f(8, 4, 128, 8), None), (f(8, 4, 128, 128), f(8, 4, 128, 8), m.ERR_INVALID_ARG),
                                 (f(8, 4, 128, 64), f(8, 4, 128, 4), m.ERR_INVALID_ARG), (f(8, 4, 128, 64), None, m.ERR_INVALID_ARG)):
        def go():
            m.qk_norm_mrope_insert(d, nr=m.make_norm_rope(*w), axes=m.make_rope_axes((64,)), cache=m.KVCache(
                m.FP8_E4M3, f(8, 4, 128, 128), f(8, 4, 128, 128)), idx_cache=m.IndexCache(m.NVFP4, keys, None, scales),
                **dict(a, positions=f(1, 3, dt=torch.int32)))
        if status is None:
            go()
        else:
            with pytest.raises(m.MSAError) as e:
                go()
            assert e.value.status == status
    assert made == ["msa_qk_norm_mrope_insert"]


@pytest.mark.parametrize("call,names", [("step", ("seq_lens", "block_table", "flags")), ("gqa", ("out", "k", "flags")),
                                        ("rope", ("k", "q_out", "flags"))])
def test_missing_tensors(m, call, names):
    run, args = calls(m)[call]
    for name in names:
        with pytest.raises(m.MSAError) as e:
            run(**dict(args, **{name: None}))
        assert e.value.status == m.ERR_INVALID_ARG, name


def test_index_scales_off_their_type(m):
    """fp32 scales of an FP8 index cache off a 4-byte boundary."""
    at = ctypes.c_void_p(0x10000)
    d = m.make_dims(2, 1, max_blocks_per_seq=4, num_pages=8)
    nr, kv = m.NormRope(0x10000, 0x10000, 0x10000, 0x10000, 1e-6, 1e4), m._KVCache(m.BF16, at, at, None, None, 1.0, 1.0)
    ic, axes = m._IndexCache(m.FP8_E4M3, at, ctypes.c_void_p(0x10002), None, 1.0), m.make_rope_axes((64,))
    got = m.lib.msa_qk_norm_mrope_insert(ctypes.byref(d), at, at, at, at, at, at, 3, at, 3, ctypes.byref(nr), ctypes.byref(axes),
                                         at, at, ctypes.byref(kv), ctypes.byref(ic), at, None)
    assert got == m.ERR_INVALID_ARG
