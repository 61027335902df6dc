"""Refusals of the full-attention layer's calls, and the oracle pieces they are tested with. CPU only: nothing launches."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def m():
    from block_sparse_attention_07_gb300 import _build
    _build.build()
    from block_sparse_attention_07_gb300 import msa
    return msa


FAKE = ctypes.c_void_p(0x10000)


def _dims(m, **kw):
    d = m.make_dims(2, 1, max_blocks_per_seq=4, num_pages=8)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _gqa(m, d=None, q=FAKE, kv=None, table=FAKE, lens=FAKE, out=FAKE, ws=FAKE, n=1 << 40, flags=FAKE):
    kv = m._KVCache(m.BF16, FAKE, FAKE, None, None, 1.0, 1.0) if kv is None else kv
    d = _dims(m) if d is None else d
    return m.lib.msa_paged_gqa_decode(ctypes.byref(d), q, ctypes.byref(kv), table, lens, out, None, ws, n, flags, None)


def test_paged_gqa_shapes(m):
    for bad in (dict(head_dim=64), dict(block_size=64), dict(q_len=9), dict(n_heads=65), dict(n_heads=68),
                dict(n_kv_heads=65, n_heads=65), dict(batch=4097), dict(max_blocks_per_seq=2 ** 24 + 1),
                dict(num_pages=2 ** 22 + 1)):
        assert _gqa(m, _dims(m, **bad)) == m.ERR_UNSUPPORTED, bad
        assert m.paged_gqa_workspace_size(_dims(m, **bad), m.BF16) == 0
    for bad in (dict(batch=0), dict(q_len=0), dict(num_pages=0), dict(n_heads=-4), dict(softmax_scale=0.0),
                dict(softmax_scale=float("nan")), dict(softmax_scale=float("inf"))):
        assert _gqa(m, _dims(m, **bad)) == m.ERR_INVALID_ARG, bad
    assert m.lib.msa_paged_gqa_decode(None, FAKE, None, FAKE, FAKE, FAKE, None, FAKE, 0, FAKE, None) == m.ERR_INVALID_ARG


def test_paged_gqa_pointers_and_types(m):
    for name in ("q", "table", "lens", "out", "flags"):
        assert _gqa(m, **{name: None}) == m.ERR_INVALID_ARG, name
    assert _gqa(m, q=ctypes.c_void_p(0x10008)) == m.ERR_INVALID_ARG
    assert _gqa(m, ws=None) == m.ERR_WORKSPACE
    assert _gqa(m, ws=ctypes.c_void_p(0x10010)) == m.ERR_WORKSPACE
    need = m.paged_gqa_workspace_size(_dims(m), m.BF16)
    assert need > 0 and _gqa(m, n=need - 1) == m.ERR_WORKSPACE
    kv = lambda *a: m._KVCache(*a)
    assert _gqa(m, kv=kv(m.F32, FAKE, FAKE, None, None, 1.0, 1.0)) == m.ERR_UNSUPPORTED
    assert _gqa(m, kv=kv(m.BF16, FAKE, None, None, None, 1.0, 1.0)) == m.ERR_INVALID_ARG
    assert _gqa(m, kv=kv(m.NVFP4, FAKE, FAKE, FAKE, None, 1.0, 1.0)) == m.ERR_INVALID_ARG
    for g in (0.0, -1.0, float("nan"), float("inf")):
        assert _gqa(m, kv=kv(m.FP8_E4M3, FAKE, FAKE, None, None, g, 1.0)) == m.ERR_INVALID_ARG
        assert _gqa(m, kv=kv(m.NVFP4, FAKE, FAKE, FAKE, FAKE, 1.0, g)) == m.ERR_INVALID_ARG


def _step(m, **kw):
    a = dict(dims=_dims(m), ctx=FAKE, new=ctypes.c_void_p(0x20000), free=FAKE, F=4, head=FAKE, off=None, table=FAKE,
             seq=ctypes.c_void_p(0x30000), starts=FAKE, slots=FAKE, pos=FAKE, axes=1, stride=8, T=8,
             out=ctypes.c_void_p(0x40000), flags=FAKE)
    a.update(kw)
    d = a["dims"]
    return m.lib.msa_build_step(ctypes.byref(d) if d else None, a["ctx"], a["new"], a["free"], a["F"], a["head"],
                                a["off"], a["table"], a["seq"], a["starts"], a["slots"], a["pos"], a["axes"],
                                a["stride"], a["T"], a["out"], a["flags"], None)


def test_build_step_refusals(m):
    for name in ("ctx", "new", "free", "head", "table", "seq", "starts", "slots", "pos", "out", "flags"):
        assert _step(m, **{name: None}) == m.ERR_INVALID_ARG, name
    assert _step(m, dims=None) == m.ERR_INVALID_ARG
    for bad in (dict(T=0), dict(F=-1), dict(axes=0), dict(stride=7), dict(slots=ctypes.c_void_p(0x10008)), dict(seq=FAKE),
                dict(out=FAKE), dict(dims=_dims(m, batch=0)), dict(dims=_dims(m, num_pages=0))):
        assert _step(m, **bad) == m.ERR_INVALID_ARG, bad
    for bad in (dict(axes=5), dict(dims=_dims(m, batch=4097)), dict(dims=_dims(m, block_size=64))):
        assert _step(m, **bad) == m.ERR_UNSUPPORTED, bad


def _mrope(m, dims=None, axes=None, kv=None, ic=None, nr=None, T=3, stride=3, **p):
    a = dict(q=FAKE, k=FAKE, v=FAKE, iq=None, ik=None, pos=FAKE, slots=FAKE, qo=FAKE, iqo=None, flags=FAKE)
    a.update(p)
    d = _dims(m) if dims is None else dims
    axes = m.make_rope_axes((16, 24, 24)) if axes is None else axes
    kv = m._KVCache(m.BF16, FAKE, FAKE, None, None, 1.0, 1.0) if kv is None else kv
    nr = m.NormRope(0x10000, 0x10000, None, None, 1e-6, 1e4) if nr is None else nr
    return m.lib.msa_qk_norm_mrope_insert(ctypes.byref(d), a["q"], a["k"], a["v"], a["iq"], a["ik"], a["pos"], stride,
                                          a["slots"], T, ctypes.byref(nr), ctypes.byref(axes), a["qo"], a["iqo"],
                                          ctypes.byref(kv), ctypes.byref(ic) if ic else None, a["flags"], None)


def test_mrope_refusals(m):
    for name in ("q", "k", "v", "pos", "slots", "qo", "flags"):
        assert _mrope(m, **{name: None}) == m.ERR_INVALID_ARG, name
    assert _mrope(m, q=ctypes.c_void_p(0x10004)) == m.ERR_INVALID_ARG
    assert _mrope(m, T=-1) == m.ERR_INVALID_ARG and _mrope(m, stride=2) == m.ERR_INVALID_ARG
    assert _mrope(m, T=0, q=None) == m.OK and m.last_dispatch() == "qk_norm_mrope_insert empty"
    ax = m.make_rope_axes((32, 32))
    ax.axis[63] = 2
    assert _mrope(m, axes=ax) == m.ERR_INVALID_ARG
    assert _mrope(m, axes=m.RopeAxes(5)) == m.ERR_UNSUPPORTED and _mrope(m, axes=m.RopeAxes(0)) == m.ERR_INVALID_ARG
    for nr in ((0x10000, 0x10000, None, None, -1.0, 1e4), (0x10000, 0x10000, None, None, 1e-6, 1.0), (0x10000, None, None, None, 1e-6, 1e4)):
        assert _mrope(m, nr=m.NormRope(*nr)) == m.ERR_INVALID_ARG
    assert _mrope(m, iq=FAKE) == m.ERR_INVALID_ARG                                 # half an index branch
    nr = m.NormRope(0x10000, 0x10000, 0x10000, 0x10000, 1e-6, 1e4)
    ic = m._IndexCache(m.F32, FAKE, None, None, 1.0)
    assert _mrope(m, iq=FAKE, ik=FAKE, iqo=FAKE, nr=nr, ic=ic) == m.ERR_UNSUPPORTED
    assert _mrope(m, dims=_dims(m, n_heads=72)) == m.ERR_UNSUPPORTED


def test_rope_axes_maps(m):
    from oracle import mrope
    for sec, inter in (((64,), False), ((16, 24, 24), False), ((24, 20, 20), True), ((16, 16, 16, 16), True)):
        ax = m.make_rope_axes(sec, inter)
        assert list(ax.axis) == mrope.sections_to_axis(sec, inter) and ax.num_axes == len(sec)
    for sec, inter in (((16, 24, 23), False), ((), False), ((70, -6), False), ((16, 24, 24), True), ((13,) * 5, False)):
        with pytest.raises(m.MSAError):
            m.make_rope_axes(sec, inter)


def test_tensor_checks(m):
    """Wrong types, shapes and layouts are refused before any pointer is passed on."""
    import torch
    d = _dims(m)
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)
    good = dict(ctx_lens=z(2), new_lens=z(2), free_pages=z(4), free_head=z(1), block_table=z(2, 4), seq_lens=z(2),
                token_starts=z(3), slot_mapping=z(8, dt=torch.int64), positions=z(3, 8), free_head_out=z(1), flags=z(1))
    for name, t in (("ctx_lens", z(3)), ("new_lens", z(2, dt=torch.int64)), ("block_table", z(4, 2).T), ("seq_lens", z(4)[::2]),
                    ("slot_mapping", z(8)), ("positions", z(3, 7)), ("positions", z(8, 3).T)):
        with pytest.raises(m.MSAError) as e:
            m.build_step(d, **dict(good, **{name: t}))
        assert e.value.status == m.ERR_INVALID_ARG and name in str(e.value)
    bf = torch.bfloat16
    q, cache = z(2, 1, 64, 128, dt=bf), m.KVCache(m.BF16, z(8, 4, 128, 128, dt=bf), z(8, 4, 128, 128, dt=bf))
    args = dict(q=q, cache=cache, block_table=z(2, 4), seq_lens=z(2), out=torch.zeros_like(q), lse=None, workspace=None, flags=z(1))
    for name, t in (("q", z(2, 1, 128, 64, dt=bf).transpose(2, 3)), ("q", q.float()), ("out", z(2, 1, 32, 128, dt=bf)),
                    ("cache", m.KVCache(m.BF16, cache.k, cache.v[:4])), ("cache", m.KVCache(m.FP8_E4M3, cache.k, cache.v)),
                    ("cache", m.KVCache(m.NVFP4, z(8, 4, 128, 64, dt=torch.uint8), z(8, 4, 128, 64, dt=torch.uint8)))):
        with pytest.raises(m.MSAError) as e:
            m.paged_gqa_decode(d, **dict(args, **{name: t}))
        assert e.value.status == m.ERR_INVALID_ARG


def test_oracle_step_by_hand():
    """Two requests: one crosses into a new block, one starts empty; one padding token."""
    from oracle import step
    w = step.build_step([127, 0], [2, 1], [7, 5, 6], 0, np.array([[3, -1], [-1, -1]]), 8, 4, axes=2, pos_offset=[10, 0])
    assert w["table"].tolist() == [[3, 7], [5, -1]] and w["seq_lens"].tolist() == [129, 1]
    assert w["token_starts"].tolist() == [0, 2, 3] and w["free_head"] == 2 and w["flags"] == 0
    assert w["slots"].tolist() == [3 * 128 + 127, 7 * 128, 5 * 128, -1]
    assert w["positions"].tolist() == [[137, 138, 0, 0]] * 2


def test_oracle_mrope_with_equal_axes_is_the_one_axis_rotation():
    from oracle import mrope, prologue
    rng = np.random.default_rng(0)
    x, w, pos = rng.standard_normal((5, 2, 128)), rng.standard_normal(128), rng.integers(0, 9999, 5)
    got = mrope.norm_mrope(x, w, np.tile(pos, (3, 1)), mrope.sections_to_axis((16, 24, 24)), 1e-6, 1e4)
    assert np.array_equal(got, prologue.norm_rope(x, w, pos, 1e-6, 1e4))


def test_pointers_off_their_type(m):
    odd = ctypes.c_void_p(0x50002)
    for name in ("table", "lens", "flags"):
        assert _gqa(m, **{name: odd}) == m.ERR_INVALID_ARG, name
    assert m.lib.msa_paged_gqa_decode(ctypes.byref(_dims(m)), FAKE, ctypes.byref(m._KVCache(m.BF16, FAKE, FAKE, None, None, 1.0, 1.0)),
                                      FAKE, FAKE, FAKE, odd, FAKE, 1 << 40, FAKE, None) == m.ERR_INVALID_ARG
    for name in ("ctx", "new", "free", "head", "off", "table", "seq", "starts", "pos", "out", "flags"):
        assert _step(m, **{name: odd}) == m.ERR_INVALID_ARG, name
    assert _gqa(m, _dims(m, softmax_scale=2.5e38)) == m.ERR_INVALID_ARG
    for name in ("pos", "slots", "flags"):
        assert _mrope(m, **{name: odd}) == m.ERR_INVALID_ARG, name
    assert _mrope(m, slots=ctypes.c_void_p(0x50004)) == m.ERR_INVALID_ARG
