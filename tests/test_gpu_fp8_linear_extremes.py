"""msa_fp8_linear at the largest sizes that it takes: 2^24 tokens, outputs or inputs. Bound as in test_gpu_fp8_linear, the
product taken in 64 bits by torch, a part at a time."""
import pytest
import torch

from block_sparse_attention_07_gb300 import msa

pytestmark = pytest.mark.gpu

MOST = 1 << 24


def codes(rows, K, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    out = torch.empty((rows, K), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // K)
    for i in range(0, rows, step):
        part = out[i:i + step]
        part.copy_((torch.randn(part.shape, generator=gen, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    return out


@pytest.mark.parametrize("T,N,K,dtype", [(MOST, 9, 16, torch.bfloat16), (MOST - 1, 130, 16, torch.bfloat16), (1, MOST, 16, torch.float32),
                                         (70, MOST - 3, 16, torch.bfloat16), (2, 3, MOST, torch.float32), (150, 3, MOST // 8, torch.float32)])
def test_most(T, N, K, dtype):
    KB, NB = -(-K // 128), -(-N // 128)
    a, w = codes(T, K, 1), codes(N, K, 2)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    sa, sw = (torch.exp(4 * torch.rand((r, KB), generator=gen, device="cuda") - 2) for r in (T, NB))
    out = torch.full((T, N), 7.0, dtype=dtype, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.fp8_linear(a, sa, w, sw, out, flags)
    torch.cuda.synchronize()
    assert int(flags.item()) == 0
    u = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8

    def values(c, s, i, rows_per_scale, k0, k1):
        """Rows i of codes, inputs k0 to k1, in 64 bits."""
        x = c[i, k0:k1].view(torch.float8_e4m3fn).double()
        f = s[i // rows_per_scale, k0 // 128:-(-k1 // 128)].double().repeat_interleave(128, 1)[:, :k1 - k0]
        return x * f

    step_t = max(1, (1 << 25) // max(N, min(K, 1 << 20)))
    step_k = 1 << 20
    step_n = 1 << 22
    for t0 in range(0, T, step_t):
        ts = torch.arange(t0, min(T, t0 + step_t), device="cuda")
        for n0 in range(0, N, step_n):
            ns = torch.arange(n0, min(N, n0 + step_n), device="cuda")
            want = size = 0
            for k0 in range(0, K, step_k):
                x, y = values(a, sa, ts, 1, k0, min(K, k0 + step_k)), values(w, sw, ns, 128, k0, min(K, k0 + step_k))
                want, size = want + x @ y.t(), size + x.abs() @ y.abs().t()
            lim = (128 * 2.0 ** -23 + (KB + 10) * 2.0 ** -24) * size
            lim = lim + u * (want.abs() + lim)
            got = out[t0:t0 + step_t, n0:n0 + step_n].double()
            assert ((got - want).abs() <= lim).all(), (t0, n0)
