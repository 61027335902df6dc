"""The codes of msa_add_norm_quant's groups are those of the quotients y / s.

The kernel does not divide: it multiplies by a reciprocal in two parts, v = RN(1 / d) and w = RN((1 - d v) v), a little
nearer zero where d is a step below a power of two, as RN(y v + RN(y w)). 1 - d v is exact, w is off by 2^-47 / d at most and
the inner product's rounding by 2^-48 y / d, so the result is RN(Q (1 + e)) of Q = y / d with |e| < 2^-46. Its E4M3 code can differ from RN(Q)'s only where the two lie on
different sides of a border m of E4M3, or one of them on it. m is an odd multiple of 2^-4 (of less where E4M3 is
subnormal) and y - m d a multiple of 2^-27 for d in [1, 2), so Q is m or 2^-29 away from it: that leaves a Q within 2^-46 of
an end of the interval that rounds to m, m + h with h = 2^-24, -2^-24, or -2^-25 below a power of two. There h d is within 2^-44
of a multiple of 2^-27, i.e. d within 2^-20 of a multiple of 1/8. All of those cases are gone through below, with room."""
from fractions import Fraction as Fr

import numpy as np
import pytest
import torch

from oracle import layer as L

BORDERS = sorted({Fr(n, 16) for n in range(17, 32, 2)} | {Fr(n, 8) for n in range(8, 16)})     # of quotients in [1, 2)


def rn(x):
    """A positive rational rounded to 24 bits, ties to even."""
    e = 0
    while x >= 2 ** (e + 1):
        e += 1
    while x < Fr(2) ** e:
        e -= 1
    step = Fr(2) ** (e - 23)
    return round(x / step) * step                              # (Python's round: half to even)


def near(x):
    """The floats around a rational."""
    c = rn(x)
    step = Fr(2) ** -23 if c < 2 else Fr(2) ** -22
    return [c + k * step for k in range(-2, 3)]


def parts(d, exception=True):
    """The reciprocal's two parts."""
    v = rn(1 / d)
    left = 1 - d * v
    assert left == 0 or rn(abs(left)) == abs(left)
    w = rn(abs(left) * v) * (1 if left > 0 else -1) if left else Fr(0)
    return v, rn(-w * (1 - Fr(2) ** -22)) * -1 if exception and d == 2 - Fr(2) ** -23 else w


def product(y, v, w):
    t = y * w
    return rn(y * v + (rn(abs(t)) * (1 if t > 0 else -1) if t else t))


def test_two_part_reciprocal_keeps_every_code():
    gone = 0
    for k in range(8, 17):
        for j in range(-12, 13):
            d = Fr(k, 8) + j * Fr(2) ** -23
            if not 1 <= d < 2:
                continue
            v, w = parts(d)
            for m in BORDERS:
                for h in (Fr(2) ** -24, -(Fr(2) ** (-25 if m == 1 else -24)), Fr(0)):
                    for y in near((m + h) * d):
                        got, want = product(y, v, w), rn(y / d)
                        gone += 1
                        assert (got > m) == (want > m) and (got < m) == (want < m), (d, m, y)
    assert gone > 40000


def test_simpler_products_would_not():
    """The rounded reciprocal alone breaks exact ties; the two parts without their exception put 2 / d, which is
    the float above a border, on the border."""
    d = rn(Fr(13, 7))
    assert any((rn(y * rn(1 / d)) > m) != (rn(y / d) > m) for m in BORDERS for y in near(m * d))
    d = 2 - Fr(2) ** -23
    assert product(Fr(2), *parts(d, False)) == 1 < rn(2 / d) == product(Fr(2), *parts(d))


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-110, -66, -40, 0, 40, 66, 110])
def test_values_next_to_borders(power):
    """Groups of fp32 values within a few steps of every border, over scales on both sides of 2^-64 and 2^64."""
    from block_sparse_attention_07_gb300 import msa
    rng = np.random.default_rng(power + 200)
    T, W = 400, 256
    s = (rng.uniform(1, 2, (T, 2)) * 2.0 ** power).astype(np.float32)
    s[:T // 2] = (rng.integers(8, 17, (T // 2, 2)) / 8 * 2.0 ** power * (1 + rng.integers(-6, 7, (T // 2, 2)) * 2.0 ** -23)).astype(np.float32)
    m = rng.choice([float(b) for b in BORDERS], (T, 2, 128)) * 2.0 ** rng.integers(-10, 9, (T, 2, 128))
    y = (np.minimum(m, 440.0) * s[..., None]).astype(np.float32)
    for _ in range(2):
        y = np.nextafter(y, np.where(rng.random(y.shape) < 0.5, np.float32(0), np.float32(3e38))).astype(np.float32)
    y[:, :, 0] = s * np.float32(448)                           # the group's largest
    y = (y * rng.choice([-1, 1], y.shape).astype(np.float32)).reshape(T, W)
    x = torch.zeros((T, W), dtype=torch.bfloat16, device="cuda")
    codes, scales = torch.empty((T, W), dtype=torch.uint8, device="cuda"), torch.empty((T, 2), device="cuda")
    msa.add_norm_quant(x, None, residual=torch.from_numpy(y).cuda(), codes=codes, scales=scales)
    want, ws = L.quant_rows(y)
    assert np.array_equal(scales.cpu().numpy(), ws) and np.array_equal(codes.cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("T,W", [(256, 8192), (2100, 4096), (333, 5008)])
def test_rounding_of_outputs_is_the_divisions(T, W):
    """bf16 values, of which many lie on a border exactly; the quotients taken by torch, scales by the kernel."""
    from block_sparse_attention_07_gb300 import msa
    torch.manual_seed(T)
    x = torch.randn((T, W), device="cuda").bfloat16()
    codes, scales = torch.empty((T, W), dtype=torch.uint8, device="cuda"), torch.empty((T, -(-W // 128)), device="cuda")
    msa.add_norm_quant(x, None, codes=codes, scales=scales)
    q = x.float() / scales.repeat_interleave(128, 1)[:, :W]
    assert torch.equal(codes, q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
