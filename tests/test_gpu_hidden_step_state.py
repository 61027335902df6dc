"""What ``DeviceWorkload.hidden_step`` builds at its first call: whole before any stream uses it, and kept."""
import numpy as np
import pytest
import torch

from block_sparse_attention_07_gb300 import synth
from block_sparse_attention_07_gb300.workload import DeviceWorkload

pytestmark = pytest.mark.gpu


def build(kind="b32_32k", index=True):
    w = synth.scaled(synth.WORKLOADS[kind], batch=3, ctx=700)
    return DeviceWorkload(w, "cuda", lens=np.array([700, 129, 300], dtype=np.int32), index_cache=index)


def rows(dw, hidden, seed):
    T = 3 * dw.w.q_len
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x, r = (torch.randn((T, hidden), generator=gen, device="cuda").bfloat16() for _ in range(2))
    return x, r, torch.zeros_like(x)


def eager(kind, index, hidden, seed):
    dw = build(kind, index)
    x, r, y = rows(dw, hidden, seed)
    dw.hidden_step(x, r, y)
    torch.cuda.synchronize()
    assert dw.check_flags() == 0 and y.any()
    return r, y


@pytest.mark.parametrize("kind,index", [("b32_32k", True), ("b32_32k", False), ("spec8", True)])
@pytest.mark.parametrize("raw", [False, True])
def test_first_call_on_another_stream(kind, index, raw):
    """The weights are made on the current stream, late; the first step is on another one."""
    want = eager(kind, index, 2064, 1)
    dw = build(kind, index)
    x, r, y = rows(dw, 2064, 1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(40_000_000)                      # some 20 ms in front of the weights
    dw.hidden_step(x, r, y, stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert torch.equal(r, want[0]) and torch.equal(y, want[1])
    # the weights stay: again, after everything has come to rest
    torch.cuda.synchronize()
    x, r, y = rows(dw, 2064, 1)
    dw.hidden_step(x, r, y)
    torch.cuda.synchronize()
    assert torch.equal(r, want[0]) and torch.equal(y, want[1]) and dw.check_flags() == 0


def test_first_call_for_another_hidden_size():
    """A captured step keeps its weights and buffers while steps of other sizes are made."""
    want = {h: eager("b32_32k", True, h, 2) for h in (2064, 4096, 1040)}
    dw = build()
    x, r, y = rows(dw, 2064, 2)
    r0 = r.clone()
    dw.prepare_hidden_step(2064)
    g = dw.capture(lambda s: dw.hidden_step(x, r, y, s))
    for h in (4096, 1040):
        a = rows(dw, h, 2)
        dw.hidden_step(*a)
        torch.cuda.synchronize()
        assert torch.equal(a[1], want[h][0]) and torch.equal(a[2], want[h][1])
        fill = [torch.full((1 << 24,), float("nan"), device="cuda") for _ in range(8)]      # what was let go is reused
        del fill
        r.copy_(r0)
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r, want[2064][0]) and torch.equal(y, want[2064][1])
    assert dw.check_flags() == 0


def test_first_step_in_a_capture():
    """Refused by name; with prepare_hidden_step in front, a captured first step is an eager one's bits."""
    want = eager("spec8", False, 1040, 3)
    dw = build("spec8", False)
    x, r, y = rows(dw, 1040, 3)
    r0 = r.clone()
    with pytest.raises(RuntimeError, match="prepare_hidden_step"):
        dw.capture(lambda s: dw.hidden_step(x, r, y, s))
    assert torch.equal(r, r0)
    dw.prepare_hidden_step(1040)
    g = dw.capture(lambda s: dw.hidden_step(x, r, y, s))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, want[0]) and torch.equal(y, want[1]) and dw.check_flags() == 0


def test_outputs_in_fp32():
    """An fp32 y holds what a bf16 one rounds."""
    want = eager("b32_32k", True, 1040, 4)
    dw = build()
    x, r, y = rows(dw, 1040, 4)
    y = y.float()
    dw.hidden_step(x, r, y)
    torch.cuda.synchronize()
    assert torch.equal(y.bfloat16(), want[1]) and not torch.equal(y, want[1].float())


def test_first_call_by_the_default_streams_number():
    """Stream 0 by its number, and a first call on another stream inside a capture of the current one: refused by name."""
    want = eager("b32_32k", False, 1040, 5)
    dw = build("b32_32k", False)
    x, r, y = rows(dw, 1040, 5)
    r0 = r.clone()
    side = torch.cuda.Stream()
    with pytest.raises(RuntimeError, match="prepare_hidden_step"):
        dw.capture(lambda s: dw.hidden_step(x, r, y, side))
    assert torch.equal(r, r0)
    dw.hidden_step(x, r, y, 0)
    torch.cuda.synchronize()
    assert torch.equal(r, want[0]) and torch.equal(y, want[1]) and dw.check_flags() == 0
