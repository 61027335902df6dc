"""perf/more_operators.py: a pass works on the tensors that its state holds at that time, on the stream that is current."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def ops():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("measured_layer_operators", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.own = True
    return mod


CASES = {"norm": lambda o: o._norm("a", 5, 400, residual="f32", out="both"), "linear": lambda o: o._linear("a", 5, 200, 400),
         "rope": lambda o: o._rope("a", 5, kv="fp8", kv_heads=1, group=4)}


def outputs(x):
    x = list(x.values()) if isinstance(x, dict) else list(x) if isinstance(x, (list, tuple)) else [x]
    return [t.view(torch.uint8).clone() for t in x]


@pytest.mark.parametrize("op", list(CASES))
def test_replaced_tensors_are_the_ones_used(ops, op):
    """Each tensor of a state in turn is replaced by another seed's; a fresh state of the same tensors gives the outputs."""
    case = CASES[op](ops)
    one, two = ops.prepare(case, 1), ops.prepare(case, 2)
    first = outputs(ops.run(one))
    for name in [n for n, t in one.items() if isinstance(t, torch.Tensor)]:
        one[name] = two[name].clone()
        fresh = {n: t for n, t in one.items() if n != "kept"}
        got = outputs(ops.run(one))
        assert all(torch.equal(a, b) for a, b in zip(got, outputs(ops.run(fresh)))), name
        assert int(one["flags"].item()) == 0
    assert any(not torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("op", list(CASES))
def test_replaced_outputs_are_the_ones_written(ops, op):
    case = CASES[op](ops)
    s = ops.prepare(case, 3)
    want = outputs(ops.run(s))
    for name in ("out", "codes", "scales", "residual_out", "q_out", "k_cache", "v_cache"):
        if name in s:
            old = s[name]
            s[name] = torch.zeros_like(old)
            old.zero_()
    got = outputs(ops.run(s))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and any(t.any() for t in got)


@pytest.mark.parametrize("op", list(CASES))
def test_passes_follow_the_stream(ops, op):
    case = CASES[op](ops)
    s = ops.prepare(case, 4)
    want = outputs(ops.run(s))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = outputs(ops.run(s))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(s["kept"][-1]) == 2
