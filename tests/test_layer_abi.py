"""Refusals of the operators around the attention, and msa_make_rope. CPU only: nothing launches."""
import ctypes
import math

import numpy as np
import pytest
import torch

FAKE, ODD4, ODD8 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x50002), ctypes.c_void_p(0x50004)


@pytest.fixture(scope="module")
def m():
    from block_sparse_attention_07_gb300 import _build
    _build.build()
    from block_sparse_attention_07_gb300 import msa
    return msa


def _norm(m, T=2, W=128, x=FAKE, stride=128, res=None, res_out=None, kind=1, weight=FAKE, eps=1e-6, out=FAKE, codes=None, scales=None):
    return m.lib.msa_add_norm_quant(T, W, x, stride, res, res_out, kind, weight, eps, out, codes, scales, None)


def test_norm_refusals(m):
    for bad in (dict(T=-1), dict(W=0), dict(x=None), dict(stride=127), dict(stride=132), dict(out=None), dict(codes=FAKE),
                dict(scales=FAKE), dict(res_out=FAKE), dict(eps=-1.0), dict(eps=math.nan), dict(eps=2.0), dict(x=ODD8),
                dict(out=ODD8), dict(weight=ODD8), dict(res=ODD8), dict(res=FAKE, res_out=ODD8), dict(codes=ODD8, scales=FAKE),
                dict(codes=FAKE, scales=ODD4), dict(stride=136, out=FAKE)):
        assert _norm(m, **bad) == m.ERR_INVALID_ARG, bad
    for bad in (dict(W=120, stride=120), dict(W=16400, stride=16400), dict(res=FAKE, kind=m.FP8_E4M3)):
        assert _norm(m, **bad) == m.ERR_UNSUPPORTED, bad
    assert _norm(m, T=0, x=None) == m.OK and m.last_dispatch() == "add_norm_quant empty"


def _linear(m, T=2, N=256, K=128, a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, out=FAKE, kind=1, stride=256, flags=FAKE):
    return m.lib.msa_fp8_linear(T, N, K, a, sa, w, sw, out, kind, stride, flags, None)


def test_linear_refusals(m):
    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(out=None),
                dict(flags=None), dict(stride=255), dict(a=ODD8), dict(w=ODD8), dict(out=ODD8), dict(sa=ODD4), dict(sw=ODD4),
                dict(flags=ODD4)):
        assert _linear(m, **bad) == m.ERR_INVALID_ARG, bad
    for bad in (dict(K=120), dict(kind=m.FP8_E4M3), dict(T=2 ** 24 + 1), dict(N=2 ** 24 + 1, stride=2 ** 25), dict(K=2 ** 24 + 16),
                dict(N=2 ** 24, K=2 ** 16, stride=2 ** 24)):
        assert _linear(m, **bad) == m.ERR_UNSUPPORTED, bad
    assert _linear(m, T=0, a=None, out=None) == m.OK and m.last_dispatch() == "fp8_linear empty"


def _dims(m, **kw):
    d = m.make_dims(2, 1, max_blocks_per_seq=4, num_pages=8)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _rope(m, dims=None, rope=None, nr=0, kv=None, ic=None, T=3, **p):
    a = dict(q=FAKE, qs=64 * 128, k=FAKE, ks=512, v=FAKE, vs=512, iq=None, iqs=512, ik=None, iks=512, pos=FAKE, slots=FAKE,
             qo=ctypes.c_void_p(0x20000), iqo=None, flags=FAKE)
    a.update(p)
    d = _dims(m) if dims is None else dims
    rope = m.make_rope(64) if rope is None else rope
    nr = m.NormRope(0x10000, 0x10000, None, None, 1e-6, 1e4) if nr == 0 else nr
    kv = m._KVCache(m.BF16, FAKE, FAKE, None, None, 1.0, 1.0) if kv is None else kv
    return m.lib.msa_qkv_rope_insert(ctypes.byref(d), a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["iq"], a["iqs"],
                                     a["ik"], a["iks"], a["pos"], a["slots"], T, ctypes.byref(nr) if nr else None,
                                     ctypes.byref(rope), a["qo"], a["iqo"], ctypes.byref(kv), ctypes.byref(ic) if ic else None,
                                     a["flags"], None)


def test_rope_refusals(m):
    for name in ("q", "k", "v", "pos", "slots", "qo", "flags"):
        assert _rope(m, **{name: None}) == m.ERR_INVALID_ARG, name
    for bad in (dict(T=-1), dict(qs=64 * 128 - 8), dict(ks=504), dict(vs=504), dict(qs=64 * 128 + 4), dict(ks=516), dict(vs=516),
                dict(q=ODD8), dict(k=ODD8), dict(v=ODD8), dict(qo=ODD8), dict(pos=ODD4), dict(slots=ODD8), dict(flags=ODD4),
                dict(iq=FAKE), dict(iq=FAKE, ik=FAKE), dict(qo=FAKE, qs=65 * 128)):
        assert _rope(m, **bad) == m.ERR_INVALID_ARG, bad
    idx = dict(iq=FAKE, ik=FAKE, iqo=ctypes.c_void_p(0x30000), nr=m.NormRope(0x10000, 0x10000, 0x10000, 0x10000, 1e-6, 1e4))
    ic = m._IndexCache(m.FP8_E4M3, FAKE, FAKE, None, 1.0)
    for bad in (dict(iqs=504), dict(iks=516), dict(iq=ODD8), dict(ik=ODD8), dict(iqo=ODD8), dict(iqo=FAKE, iqs=520)):
        assert _rope(m, ic=ic, **dict(idx, **bad)) == m.ERR_INVALID_ARG, bad
    assert _rope(m, ic=m._IndexCache(m.F32, FAKE, None, None, 1.0), **idx) == m.ERR_UNSUPPORTED
    assert _rope(m, ic=m._IndexCache(m.FP8_E4M3, FAKE, ODD4, None, 1.0), **idx) == m.ERR_INVALID_ARG
    for nr in ((0x10000, None, None, None, 1e-6, 1e4), (0x10000, 0x10004, None, None, 1e-6, 1e4), (0x10000, 0x10000, None, None, -1.0, 1e4)):
        assert _rope(m, nr=m.NormRope(*nr)) == m.ERR_INVALID_ARG
    for field, val, want in (("layout", 2, m.ERR_INVALID_ARG), ("rotary_dim", 0, m.ERR_INVALID_ARG), ("rotary_dim", 24, m.ERR_UNSUPPORTED),
                             ("rotary_dim", 144, m.ERR_UNSUPPORTED), ("gain", math.nan, m.ERR_INVALID_ARG),
                             ("gain", math.inf, m.ERR_INVALID_ARG)):
        r = m.make_rope(64)
        setattr(r, field, val)
        assert _rope(m, rope=r) == want, field
    for bad in (math.nan, math.inf, 6.3, -6.3):
        r = m.make_rope(64)
        r.freq[31] = bad
        assert _rope(m, rope=r) == m.ERR_INVALID_ARG
    for bad in (dict(n_heads=72), dict(head_dim=64), dict(num_pages=2 ** 22 + 1)):
        assert _rope(m, dims=_dims(m, **bad)) == m.ERR_UNSUPPORTED, bad
    assert _rope(m, T=0, q=None, nr=None) == m.OK and m.last_dispatch() == "qkv_rope_insert empty"


def test_make_rope_against_the_oracle(m):
    from oracle import layer
    kinds = {"none": m.ROPE_NONE, "linear": m.ROPE_LINEAR, "parts": m.ROPE_BY_PARTS, "turns": m.ROPE_BY_TURNS}
    for R in (16, 64, 96, 128):
        for theta in (1.5, 1e4, 5e6):
            for kind, scaling in kinds.items():
                for factor, trained, low, high in ((4.0, 32768, 1.0, 32.0), (1.0, 4096, 1.0, 4.0), (40.0, 100, 0.5, 2.0)):
                    r = m.make_rope(R, theta, m.ROPE_INTERLEAVED, scaling, factor, trained, low, high)
                    f, gain = layer.frequencies(R, theta, kind, factor, float(trained), low, high)
                    assert r.rotary_dim == R and r.layout == 1 and abs(r.gain - gain) <= 2.0 ** -24 * gain
                    # a power (1 ulp of double each side), a ramp and two products: a few units of 2^-53, times the
                    # ramp's slope for an error of its argument
                    assert np.allclose(list(r.freq)[:R // 2], f, rtol=2.0 ** -45), (R, theta, kind, factor)
                    assert not any(list(r.freq)[R // 2:])


def test_make_rope_refusals(m):
    good = dict(rotary_dim=64, theta=1e4, layout=0, scaling=m.ROPE_BY_PARTS, factor=4.0, trained_len=4096, low_turns=1.0, high_turns=32.0)
    m.make_rope(**good)
    for bad in (dict(rotary_dim=0), dict(theta=1.0), dict(theta=math.nan), dict(theta=math.inf), dict(layout=2), dict(scaling=4),
                dict(scaling=-1), dict(factor=0.5), dict(factor=math.nan), dict(trained_len=0), dict(low_turns=0.0),
                dict(low_turns=32.0), dict(high_turns=math.inf), dict(trained_len=math.inf), dict(factor=math.inf)):
        with pytest.raises(m.MSAError) as e:
            m.make_rope(**dict(good, **bad))
        assert e.value.status == m.ERR_INVALID_ARG, bad
    for bad in (24, 8, 144):
        with pytest.raises(m.MSAError) as e:
            m.make_rope(**dict(good, rotary_dim=bad))
        assert e.value.status == m.ERR_UNSUPPORTED
    assert m.lib.msa_make_rope(None, 64, 1e4, 0, 0, 1.0, 0.0, 1.0, 2.0) == m.ERR_INVALID_ARG


# ------------------------------------------------------------------------------------ tensors of the binding --
class Fake:
    """A tensor as the checks see it, on a device of the test's choice."""

    def __init__(self, t, device):
        self.t, self.device = t, torch.device(device)

    def __getattr__(self, name):
        return getattr(self.t, name)


def z(*shape, dt=torch.float32):
    return torch.zeros(shape, dtype=dt)


def calls(m):
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    d = m.make_dims(2, 1, max_blocks_per_seq=4, num_pages=8)
    norm = dict(x=z(3, 144, dt=bf), weight=z(144), residual=z(3, 144, dt=bf), residual_out=z(3, 144, dt=bf), out=z(3, 144, dt=bf),
                codes=z(3, 144, dt=u8), scales=z(3, 2))
    linear = dict(a=z(3, 144, dt=u8), a_scales=z(3, 2), w=z(200, 144, dt=u8), w_scales=z(2, 2), out=z(3, 200), flags=z(1, dt=i32))
    rope = dict(q=z(3, 64, 128, dt=bf), k=z(3, 4, 128, dt=bf), v=z(3, 4, 128, dt=bf), idx_q=z(3, 4, 128, dt=bf), idx_k=z(3, 4, 128, dt=bf),
                positions=z(3, dt=i32), slot_mapping=z(3, dt=torch.int64), q_out=z(3, 64, 128, dt=bf), idx_q_out=z(3, 4, 128, dt=bf),
                k_cache=z(8, 4, 128, 128, dt=u8), v_cache=z(8, 4, 128, 128, dt=u8), idx_keys=z(8, 4, 128, 128, dt=u8),
                idx_scale=z(8, 4, 128), flags=z(1, dt=i32), wq=z(128), wk=z(128), wiq=z(128), wik=z(128))

    def run_rope(k_cache, v_cache, idx_keys, idx_scale, wq, wk, wiq, wik, **a):
        m.qkv_rope_insert(d, nr=m.make_norm_rope(wq, wk, wiq, wik), rope=m.make_rope(64), cache=m.KVCache(m.FP8_E4M3, k_cache, v_cache),
                          idx_cache=m.IndexCache(m.FP8_E4M3, idx_keys, idx_scale), **a)

    return {"norm": (m.add_norm_quant, norm), "linear": (m.fp8_linear, linear), "rope": (run_rope, rope)}


@pytest.mark.parametrize("call", ["norm", "linear", "rope"])
@pytest.mark.parametrize("where", ["cpu", "cuda:1"])
def test_tensors_off_the_current_gpu(m, monkeypatch, call, where):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m, "_stream", lambda stream: None)
    run, args = calls(m)[call]
    reached = []
    monkeypatch.setattr(m, "_call", lambda *a: reached.append(a[3]))
    run(**{n: Fake(t, "cuda:0") for n, t in args.items()})
    assert len(reached) == 1
    for name in args:
        with pytest.raises(m.MSAError) as e:
            run(**{n: Fake(t, where if n == name else "cuda:0") for n, t in args.items()})
        assert e.value.status == m.ERR_INVALID_ARG and "device" in str(e.value), name
    assert len(reached) == 1


@pytest.mark.parametrize("call", ["norm", "linear", "rope"])
def test_wrong_tensors(m, monkeypatch, call):
    """Another type, shape or layout; rows that lie on one another."""
    monkeypatch.setattr(m, "_call", lambda *a: pytest.fail("the call was made"))
    run, args = calls(m)[call]
    for name, t in args.items():
        other = torch.float64 if t.dtype != torch.float64 else torch.int8
        wrong = [t.to(other), torch.zeros((*t.shape[:-1], t.shape[-1] + 1), dtype=t.dtype)]
        if t.dim() > 1:
            wrong += [t.transpose(-1, -2), t[..., None].expand(*t.shape, 2)[..., 0],
                      torch.zeros((1, *t.shape[1:]), dtype=t.dtype).expand(t.shape)]
        if name == "flags":
            wrong = [t.to(other), t[:0]]
        if (call, name) == ("norm", "x"):
            wrong = [w for w in wrong if w.dtype != t.dtype or w.stride(-1) != 1 or w.stride(0) == 0]
        for w in wrong:
            with pytest.raises(m.MSAError) as e:
                run(**dict(args, **{name: w}))
            assert e.value.status == m.ERR_INVALID_ARG, (name, w.shape, w.stride(), w.dtype)


def test_missing_tensors(m):
    for call, names in (("linear", ("a", "a_scales", "w", "w_scales", "out", "flags")), ("norm", ("x",)),
                        ("rope", ("q", "k", "v", "q_out", "positions", "slot_mapping", "flags"))):
        run, args = calls(m)[call]
        for name in names:
            with pytest.raises(m.MSAError) as e:
                run(**dict(args, **{name: None}))
            assert e.value.status == m.ERR_INVALID_ARG, name


def test_strides_that_the_kernels_get(m, monkeypatch):
    """A single row's stride means nothing; views of packed rows keep theirs."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m, "_stream", lambda stream: None)
    monkeypatch.setattr(m, "_want_on_device", lambda *a, **k: None)
    got = []
    monkeypatch.setattr(m, "_call", lambda fn, args, *a: got.append(args))
    packed = z(5, 80, 128, dt=torch.bfloat16)
    d = m.make_dims(2, 1, max_blocks_per_seq=4, num_pages=8)
    cache = m.KVCache(m.FP8_E4M3, z(8, 4, 128, 128, dt=torch.uint8), z(8, 4, 128, 128, dt=torch.uint8))
    for T, want in ((5, 80 * 128), (1, None)):
        p = packed[:T]
        m.qkv_rope_insert(d, p[:, :64], p[:, 64:68], p[:, 68:72], None, None, z(T, dt=torch.int32), z(T, dt=torch.int64), None,
                          m.make_rope(), z(T, 64, 128, dt=torch.bfloat16), None, cache, None, z(1, dt=torch.int32))
        assert got[-1][2] == (want or 64 * 128) and got[-1][4] == got[-1][6] == (want or 512)
    wide = z(4, 500, dt=torch.bfloat16)
    m.add_norm_quant(wide[:, :160], None, out=z(4, 160, dt=torch.bfloat16))
    assert got[-1][3] == 500
    m.fp8_linear(z(4, 16, dt=torch.uint8), z(4, 1), z(100, 16, dt=torch.uint8), z(1, 1), wide[:, 3:103], z(1, dt=torch.int32))
    assert got[-1][9] == 500


def test_calls_without_tokens(m, monkeypatch):
    """Tensors without tokens have no addresses; the calls take them and launch nothing."""
    monkeypatch.setattr(m, "_stream", lambda stream: None)
    monkeypatch.setattr(m, "_want_on_device", lambda *a, **k: None)
    bf, u8 = torch.bfloat16, torch.uint8
    x, r, codes, scales = z(0, 256, dt=bf), z(0, 256, dt=bf), z(0, 256, dt=u8), z(0, 2)
    for outs in (dict(codes=codes, scales=scales), dict(out=x), dict(out=x, codes=codes, scales=scales)):
        for res in (dict(), dict(residual=r), dict(residual=r, residual_out=r), dict(residual=r.float(), residual_out=r.float())):
            m.add_norm_quant(x, z(256), **res, **outs)
            assert m.last_dispatch() == "add_norm_quant empty"
    flags = z(1, dt=torch.int32)
    m.fp8_linear(codes, scales, z(128, 256, dt=u8), z(1, 2), z(0, 128), flags)
    assert m.last_dispatch() == "fp8_linear empty"
    d = m.make_dims(2, 1, max_blocks_per_seq=4, num_pages=8)
    heads = z(0, 80, 128, dt=bf)
    cache = m.KVCache(m.FP8_E4M3, z(8, 4, 128, 128, dt=u8), z(8, 4, 128, 128, dt=u8))
    index = m.IndexCache(m.FP8_E4M3, z(8, 4, 128, 128, dt=u8), z(8, 4, 128))
    for idx in (False, True):
        w = (z(128),) * 4
        m.qkv_rope_insert(d, heads[:, :64], heads[:, 64:68], heads[:, 68:72], heads[:, 72:76] if idx else None,
                          heads[:, 76:] if idx else None, z(0, dt=torch.int32), z(0, dt=torch.int64), m.make_norm_rope(*w),
                          m.make_rope(), z(0, 64, 128, dt=bf), z(0, 4, 128, dt=bf) if idx else None, cache, index if idx else None, flags)
        assert m.last_dispatch() == "qkv_rope_insert empty"


def test_prepared_calls_are_the_plain_ones(m, monkeypatch):
    """A prepared call passes the same arguments, every time: addresses, missing ones, sizes, floats and host structs."""
    monkeypatch.setattr(m, "_stream", lambda stream: None)
    monkeypatch.setattr(m, "_want_on_device", lambda *a, **k: None)
    for run, args in calls(m).values():
        seen = []
        monkeypatch.setattr(m, "_call", lambda fn, a, keep, what, prepare: seen.append((fn, a, keep, what)))
        run(**args)
        fn, a, keep, what = seen[0]
        p = m.Prepared(fn, a, keep, what)
        types = [ctypes.c_void_p if issubclass(t, ctypes._Pointer) else t for t in fn.argtypes]
        got = []
        probe = ctypes.CFUNCTYPE(ctypes.c_int, *types)(lambda *x: got.append(x) or 0)
        bare = ctypes.CFUNCTYPE(ctypes.c_int)(ctypes.cast(probe, ctypes.c_void_p).value)
        typed = ctypes.CFUNCTYPE(ctypes.c_int, *fn.argtypes)(ctypes.cast(probe, ctypes.c_void_p).value)
        typed(*a)
        p._bare = bare
        p(), p()
        assert len(got) == 3 and got[0] == got[1] == got[2]
    bad = m.Prepared(m.lib.msa_add_norm_quant, (2, 120, FAKE, 120, None, None, 1, FAKE, 1e-6, FAKE, None, None, None), (), "norm")
    for _ in range(2):
        with pytest.raises(m.MSAError) as e:
            bad()
        assert e.value.status == m.ERR_UNSUPPORTED
