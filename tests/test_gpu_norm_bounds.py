"""msa_add_norm_quant's results in fp32 precision, as its scales show them.

Derived from the kernel's own order of operations. h is one rounding (2^-24). A thread adds the squares of at most 16 values in
two chains of 8 fused additions, joins them, and 5 + 5 exchange steps follow: 19 roundings; the width's reciprocal and the
product with it 2, eps 1, and h itself twice: the mean is within 24 * 2^-24, its root within 12 and one of its own, the
reciprocal one, two products and h one each: |y - exact| <= 17 * 2^-24 |y|. A scale is one division of the group's largest
|y|: 18 * 2^-24, and the terms of second order are below 2^-24 * 2^-15."""
import numpy as np
import pytest
import torch

from oracle import layer as L

from test_gpu_norm_quant import Case, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("res", [None, "bf16", "f32"])
@pytest.mark.parametrize("T,W", [(1, 4096), (64, 4096), (333, 5008), (2100, 4096), (3, 16384), (600, 16384), (40, 272)])
def test_scales(T, W, res):
    c = Case(T, W, res, seed=T + W + 1)
    o = c.run(outs=("codes", "scales"))
    _, y = L.add_norm(f64(c.x), None if c.res is None else f64(c.res), f64(c.w), float(np.float32(1e-6)))
    top = np.stack([np.abs(y[:, g:g + 128]).max(1) for g in range(0, W, 128)], 1) / 448
    err = np.abs(f64(o["scales"]) - top) / top
    assert (err <= 18.01 * 2.0 ** -24).all(), err.max() * 2 ** 24
    assert torch.isfinite(o["scales"]).all()
