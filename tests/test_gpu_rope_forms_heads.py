"""msa_qkv_rope_insert at the smallest and largest numbers of heads, with and without index rows; one token to many."""
import pytest

from test_gpu_rope_forms import Case

pytestmark = pytest.mark.gpu


HEADS = [(64, 1024, None), (64, 1024, "fp8"), (64, 64, "nvfp4"), (1, 1, None), (1, 1, "fp8"), (5, 5, "nvfp4"), (7, 112, "fp8"), (33, 66, None)]


@pytest.mark.parametrize("T,G,H,idx", [(T, *h) for T in (1, 3, 200, 5000) for h in HEADS if T * h[1] <= 210_000])
@pytest.mark.parametrize("inter,norm", [(False, True), (True, False)])
def test_heads(T, G, H, idx, inter, norm):
    c = Case(T, G, H, idx=idx, R=48, interleaved=inter, norm=norm, seed=T + G + H)
    c.run()
    c.check()
