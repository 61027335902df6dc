"""Pins of the oracle of the operators around the attention: by hand, closed forms, library routines, invariants."""
import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import layer as L
from oracle import prologue as Pr


def test_norm_by_hand():
    h, y = L.add_norm([[1.0, 2.0]], [[2.0, 2.0]], np.array([1.0, 0.5]), 0.0)
    assert h.tolist() == [[3.0, 4.0]]                         # rms sqrt(12.5)
    assert np.allclose(y, [[3 / 12.5 ** 0.5, 2 / 12.5 ** 0.5]], rtol=1e-15)


def test_norm_is_torchs():
    rng = np.random.default_rng(0)
    x, r, w = rng.standard_normal((3, 48)), rng.standard_normal((3, 48)), rng.standard_normal(48)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x + r), (48,), torch.from_numpy(w), 1e-5)
    assert np.allclose(L.add_norm(x, r, w, 1e-5)[1], want.numpy(), rtol=1e-13)


def test_quant_rows_by_hand():
    y = np.zeros((2, 144), np.float32)
    y[0, :4] = [448.0, -1.0, 0.26, 17.0]                      # scale 1: 0.26 -> 0.25, 17 -> 17 ties to 16
    y[0, 130] = 896.0                                         # the short last group: scale 2
    codes, scales = L.quant_rows(y)
    assert scales.tolist() == [[1.0, 2.0], [0.0, 0.0]]
    assert F.e4m3_decode(codes)[0, :4].tolist() == [448.0, -1.0, 0.25, 16.0]
    assert F.e4m3_decode(codes)[0, 130] == 448.0 and not codes[1].any()


def test_quant_rows_round_trip():
    rng = np.random.default_rng(1)
    y = rng.standard_normal((5, 400)).astype(np.float32)
    v = L.dequant(*L.quant_rows(y))
    top = np.repeat(L.quant_rows(y)[1].astype(np.float64), 128, 1)[:, :400]
    # half a step: 2^-4 relative above 2^-6 of the scale, 2^-10 of it below
    assert (np.abs(v - y) <= np.maximum(np.abs(y) * 2.0 ** -4, top * 2.0 ** -10) * (1 + 1e-6)).all()


def test_linear_by_hand():
    one, two, half = (int(F.e4m3_encode(np.float32(v))) for v in (1.0, 2.0, 0.5))
    a = np.zeros((1, 256), np.uint8)
    w = np.zeros((130, 256), np.uint8)
    a[0, 0], a[0, 200] = two, one
    w[3, 0], w[129, 0], w[129, 200] = half, one, two
    y, size = L.linear(a, np.array([[3.0, 5.0]]), w, np.array([[1.0, 10.0], [100.0, 1000.0]]))
    assert y[0, 3] == 2 * 3 * 0.5 and y[0, 129] == 2 * 3 * 100 + 5 * 2 * 1000 and y.sum() == 3 + 10600
    assert np.array_equal(y, size)


def test_linear_is_torchs_product_of_the_values():
    rng = np.random.default_rng(2)
    a, w = (F.e4m3_encode(rng.standard_normal((n, 300)).astype(np.float32)) for n in (4, 260))
    sa, sw = rng.random((4, 3)), rng.random((3, 3))
    x = torch.from_numpy(a).view(torch.float8_e4m3fn).double() * torch.from_numpy(sa).repeat_interleave(128, 1)[:, :300]
    y = torch.from_numpy(w).view(torch.float8_e4m3fn).double()
    y = y * torch.from_numpy(sw).repeat_interleave(128, 0)[:260].repeat_interleave(128, 1)[:, :300]
    assert np.allclose(L.linear(a, sa, w, sw)[0], (x @ y.T).numpy(), rtol=1e-12, atol=1e-12)


def test_half_layout_is_the_prologues():
    rng = np.random.default_rng(3)
    x, pos = rng.standard_normal((6, 2, 128)), rng.integers(0, 9999, 6)
    f, gain = L.frequencies(128, 1e4)
    assert gain == 1.0 and np.allclose(L.rotate(x, pos, f, gain, False), Pr.rope(x, pos, 1e4), atol=1e-12)


@pytest.mark.parametrize("R", [16, 64, 128])
def test_interleaved_is_half_reordered(R):
    """Interleaved pairs are the half layout's after a permutation of the dims."""
    rng = np.random.default_rng(4)
    x, pos = rng.standard_normal((6, 2, 128)), rng.integers(0, 9999, 6)
    f, _ = L.frequencies(R, 1e4)
    order = np.concatenate([np.arange(0, R, 2), np.arange(1, R, 2), np.arange(R, 128)])
    got = L.rotate(x, pos, f, 1.25, True)[..., order]
    assert np.allclose(got, L.rotate(x[..., order], pos, f, 1.25, False), atol=1e-12)
    assert np.array_equal(L.rotate(x, pos, f, 1.25, True)[..., R:], x[..., R:])


def test_rotation_keeps_lengths_and_differences():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((1, 1, 128))
    f, _ = L.frequencies(64, 1e4, "linear", 4.0)
    r = lambda p: L.rotate(x, [p], f, 1.0, False)[0, 0]
    assert np.isclose(np.linalg.norm(r(777)), np.linalg.norm(x))
    assert np.isclose(r(40) @ r(100), r(1000) @ r(1060))     # depends on the distance only
    base, _ = L.frequencies(64, 1e4)
    assert np.allclose(r(400), L.rotate(x, [100], base, 1.0, False)[0, 0])


def test_scaled_frequencies():
    base, _ = L.frequencies(64, 1e4)
    for kind in ("parts", "turns"):
        f, gain = L.frequencies(64, 1e4, kind, 4.0, 4096.0, 1.0, 32.0)
        assert f[0] == base[0] and np.isclose(f[-1], base[-1] / 4)           # fast pairs keep, slow pairs stretch
        assert ((f <= base * (1 + 1e-15)) & (f >= base / 4 * (1 - 1e-15))).all() and (np.diff(f) < 0).all()
        assert gain == (0.1 * np.log(4.0) + 1 if kind == "parts" else 1.0)
        same, g1 = L.frequencies(64, 1e4, kind, 1.0, 4096.0, 1.0, 32.0)
        assert np.allclose(same, base, rtol=1e-15) and g1 == 1.0             # a factor of one changes nothing
