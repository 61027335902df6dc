"""Rotary embedding with positions on several axes, in fp64.

TEST INFRASTRUCTURE (see the package docstring). Pair i (dims i and i + D/2) of
token t turns by phi = positions[axis[i], t] * theta^(-2i/D); norm and rounding
as in ``prologue``.
"""
from __future__ import annotations

import numpy as np

from . import formats, prologue


def sections_to_axis(sections, interleaved=False):
    """The axis of every pair, written out one pair at a time."""
    left = list(sections)
    axis = []
    if not interleaved:
        for a, n in enumerate(sections):
            axis += [a] * n
        return axis
    for i in range(sum(sections)):
        a = i % len(sections)
        if a == 0 or i // len(sections) >= sections[a]:
            a = 0
        axis.append(a)
        left[a] -= 1
    assert left == [0] * len(sections), left
    return axis


def norm_mrope(x, w, positions, axis, eps, theta):
    """x [T, heads, D] (bf16 bits or floats), positions [A, T], axis [D/2] -> bf16 bits."""
    if x.dtype == np.uint16:
        x = formats.bf16_to_f64(x)
    y = prologue.rms_norm(x, w, eps)
    D = y.shape[-1]
    out = np.empty_like(y)
    for i in range(D // 2):
        phi = np.asarray(positions[axis[i]], dtype=np.float64) * float(theta) ** (-2.0 * i / D)
        c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
        out[..., i] = y[..., i] * c - y[..., i + D // 2] * s
        out[..., i + D // 2] = y[..., i] * s + y[..., i + D // 2] * c
    return prologue.to_bf16(out)
