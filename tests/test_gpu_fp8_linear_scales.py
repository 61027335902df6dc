"""msa_fp8_linear with scales far from one, to fp32 outputs.

Bound as in test_gpu_fp8_linear where the product of two scales is a normal fp32 value. Below 2^-126 the product itself is
off by half of 2^-149, which every |a w| of its group's codes multiplies; and an output below 2^-126 is off by 2^-150 for each
of the KB + 8 additions and the rounding."""
import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import layer as L

from test_gpu_fp8_linear import Case

pytestmark = pytest.mark.gpu

# rows form of 16, 32, 64 and 128 tokens, pairs by themselves and sharing K
FORMS = [("rows", 9, 1), ("rows", 9, 3), ("rows", 30, 2), ("rows", 60, 1), ("rows", 60, 2), ("rows", 150, 1), ("rows", 150, 2),
         ("pairs", 300, 1), ("pairs", 300, 2)]


def scaled(form, T, split, monkeypatch, rows, blocks, seed):
    """A case whose row scales are times 2^rows[i] and block scales times 2^blocks[j], each drawn."""
    monkeypatch.setenv("MSA_LINEAR_FORM", form)
    monkeypatch.setenv("MSA_LINEAR_SPLIT", str(split))
    c = Case(T, 300, 656, torch.float32, seed=seed)
    rng = np.random.default_rng(seed)
    up = lambda t, powers: torch.from_numpy((t.cpu().numpy().astype(np.float64) * 2.0 ** rng.choice(powers, t.shape)).astype(np.float32)).cuda()
    c.sa, c.sw = up(c.sa, rows), up(c.sw, blocks)
    return c


def check(c):
    want, size = L.linear(*(t.cpu().numpy() for t in (c.a, c.sa, c.w, c.sw)))
    codes = np.abs(F.e4m3_decode(c.a.cpu().numpy()).astype(np.float64)) @ np.abs(F.e4m3_decode(c.w.cpu().numpy()).astype(np.float64)).T
    lim = (128 * 2.0 ** -23 + (c.KB + 10) * 2.0 ** -24) * size + codes * 2.0 ** -150 + (c.KB + 10) * 2.0 ** -150
    lim = lim + 2.0 ** -24 * (np.abs(want) + lim)
    err = np.abs(c.out.double().cpu().numpy() - want)
    assert np.isfinite(err).all() and (err <= lim).all(), (err / lim).max()
    return want


@pytest.mark.parametrize("form,T,split", FORMS)
@pytest.mark.parametrize("rows,blocks", [([-50], [-50]), ([45], [45]), ([-100, -90, 0], [80]), ([100], [-100, -80]), ([-120], [0, 10])])
def test_products_in_range(monkeypatch, form, T, split, rows, blocks):
    c = scaled(form, T, split, monkeypatch, rows, blocks, 21)
    c.run()
    f = c.sa.double().min() * c.sw.double().min(), c.sa.double().max() * c.sw.double().max()
    assert float(f[0]) > 2.0 ** -149 and float(f[1]) < 2.0 ** 128
    check(c)


@pytest.mark.parametrize("form,T,split", FORMS)
def test_small_products_keep_what_a_multiple_of_2_to_minus_149_can(monkeypatch, form, T, split):
    c = scaled(form, T, split, monkeypatch, [-60], [-75, -68, -60], 22)
    assert float((c.sa.double().max() * c.sw.double().min())) < 2.0 ** -126
    c.run()
    assert np.abs(check(c)).max() > 2.0 ** -126
    c.sa *= 2.0 ** -60                                   # products below 2^-150: zeros
    c.run()
    assert not c.out.any()


@pytest.mark.parametrize("form,T,split", FORMS)
def test_products_beyond_fp32(monkeypatch, form, T, split):
    """One row and one block whose product is infinite: their outputs alone are, those of zeros NaN."""
    c = scaled(form, T, split, monkeypatch, [0], [0], 23)
    c.sa[3, 1], c.sw[1, 1] = 2.0 ** 100, 2.0 ** 100
    c.w[130, 128:256] = 0                                # a group whose sum is zero
    c.run()
    bad = torch.zeros_like(c.out, dtype=torch.bool)
    bad[3, 128:256] = True
    assert torch.equal(~c.out.isfinite(), bad) and c.out[3, 130].isnan()
