"""msa_add_norm_quant: rows whose values differ by more than fp32's squares can hold.

Bounds as derived in test_gpu_norm_quant, for any value whose result is a normal number."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import msa
from oracle import formats as F
from oracle import layer as L

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("T,W", [(6, 512), (3, 9008)])
@pytest.mark.parametrize("large,small", [(62, -50), (62, -46), (66, -40), (100, -10), (-66, -100), (0, -100)])
def test_small_values_beside_large_ones(T, W, large, small):
    """The first group's values alone are large; the others' results are as exact as theirs."""
    rng = np.random.default_rng(large + 200)
    x = (rng.uniform(1, 2, (T, W)) * rng.choice([-1, 1], (T, W)) * 2.0 ** small).astype(np.float32)
    x[:, :128] *= np.float32(2.0 ** (large - small))
    w = (1 + 0.1 * rng.standard_normal(W)).astype(np.float32)
    codes, scales = torch.empty((T, W), dtype=torch.uint8, device="cuda"), torch.empty((T, -(-W // 128)), device="cuda")
    out = torch.empty((T, W), dtype=torch.bfloat16, device="cuda")
    msa.add_norm_quant(torch.zeros_like(out), torch.from_numpy(w).cuda(), residual=torch.from_numpy(x).cuda(), out=out, codes=codes,
                       scales=scales, eps=0.0)
    torch.cuda.synchronize()
    _, y = L.add_norm(np.zeros_like(x), x, w, 0.0)
    top = np.stack([np.abs(y[:, g:g + 128]).max(1) for g in range(0, W, 128)], 1)
    assert top.min() / 448 > 2.0 ** -126
    assert (np.abs(scales.double().cpu().numpy() - top / 448) <= 52 * U * top / 448).all()
    assert (np.abs(out.double().cpu().numpy() - y) <= (2.0 ** -8 + 48 * U) * np.abs(y)).all()
    v = F.e4m3_decode(codes.cpu().numpy()).astype(np.float64)
    want = y / np.repeat(top / 448, 128, 1)[:, :W]
    assert (np.abs(v - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 104 * U * np.abs(want)).all()
