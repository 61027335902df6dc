"""The operators around a layer's attention: residual addition, RMS norm and FP8
rows; the product of FP8 rows and weights; rotary forms. In fp64.

TEST INFRASTRUCTURE (see the package docstring).

"MiniMax-M3.1-Flash Day-0 対応" (aisoku.org), section "最適化と数値", names the
fused projection, norm, rotary embedding and insert; the pages give no formulas.
The readings are this project's:

* h = x + r; y = h / sqrt(mean(h^2) + eps) * w; rows in 8 bits: per 128 values
  s = max|y| / 448, code = E4M3(y / s) (``quant_rows`` does that step in fp32
  with one rounding per operation, so that it is an exact function of y).
* out[t, n] = sum_g sa[t, g] sw[n / 128, g] sum_{k in g} a[t, k] w[n, k].
* rotary: pair i turns by position * freq_i, cosine and sine times a gain; pairs
  (i, i + R/2) or (2i, 2i + 1) of the first R dims.
"""
from __future__ import annotations

import math

import numpy as np

from . import formats, prologue

GROUP = 128


def add_norm(x, residual, weight, eps):
    """(h, y) in fp64."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    return h, h if weight is None else prologue.rms_norm(h, weight, eps)


def quant_rows(y):
    """fp32 [T, W] -> (codes uint8 [T, W], scales fp32 [T, ceil(W / 128)])."""
    y = np.asarray(y, dtype=np.float32)
    T, W = y.shape
    codes, scales = np.zeros((T, W), np.uint8), np.zeros((T, -(-W // GROUP)), np.float32)
    for g in range(scales.shape[1]):
        part = y[:, g * GROUP:(g + 1) * GROUP]
        s = (np.max(np.abs(part), axis=1) / np.float32(448.0)).astype(np.float32)
        scales[:, g] = s
        for t in np.flatnonzero(s):
            codes[t, g * GROUP:(g + 1) * GROUP] = formats.e4m3_encode((part[t] / s[t]).astype(np.float32))
    return codes, scales


def dequant(codes, scales, rows_per_scale=1):
    """fp64 values of codes [R, K] with scales [ceil(R / rows_per_scale), ceil(K / 128)]."""
    x = formats.e4m3_decode(codes).astype(np.float64)
    s = np.asarray(scales, dtype=np.float64)
    s = np.repeat(np.repeat(s, rows_per_scale, 0)[:x.shape[0]], GROUP, 1)[:, :x.shape[1]]
    return x * s


def linear(a, sa, w, sw):
    """(out, the same sum of magnitudes) in fp64."""
    x, y = dequant(a, sa), dequant(w, sw, GROUP)
    return x @ y.T, np.abs(x) @ np.abs(y).T


def frequencies(R, theta, scaling="none", factor=1.0, trained=0.0, low=1.0, high=32.0):
    """(radians per position of each pair, gain), written out one pair at a time."""
    out, gain = [], 1.0
    for i in range(R // 2):
        f = theta ** (-2.0 * i / R)
        if scaling == "linear":
            f = f / factor
        elif scaling == "parts":
            # the (real-valued) pair that makes u turns over the trained length
            pair = lambda u: math.log(trained / (u * 2 * math.pi)) / math.log(theta) * R / 2
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), R - 1)
            r = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = f / factor * r + f * (1 - r)
        elif scaling == "turns":
            turns = trained * f / (2 * math.pi)
            s = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = f * s + f / factor * (1 - s)
        out.append(f)
    if scaling == "parts":
        gain = 0.1 * math.log(factor) + 1.0
    return np.array(out), gain


def rotate(y, positions, freq, gain, interleaved):
    """y [T, heads, D] fp64, positions [T] -> fp64."""
    out = np.array(y, dtype=np.float64)
    n = len(freq)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        phi = np.asarray(positions, dtype=np.float64) * freq[i]
        c, s = gain * np.cos(phi)[:, None], gain * np.sin(phi)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., a] * s + y[..., b] * c
    return out
