"""The first calls of a process, from eight host threads at one time: what the library looks up or asks the device once is whole
before any of them uses it. A process of its own per kind of call, several times."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys, threading
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import torch
from block_sparse_attention_07_gb300 import msa
import test_gpu_first_call_of_a_thread as one
kind = sys.argv[2]
made = [(one.linear(40) if kind == "linear" else one.attention("fp8", 1, kind == "sparse")) for _ in range(8)]
calls = [(m[0](torch.cuda.Stream()), m[1], m[2]) for m in made]
torch.cuda.synchronize()
barrier, failed = threading.Barrier(8), []
def work(i):
    barrier.wait()
    try:
        calls[i][0]()
    except Exception as e:
        failed.append(repr(e))
threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failed, failed
got = [c[1].clone() for c in calls]
for c in calls:
    c[1].zero_()
torch.cuda.synchronize()
for c in calls:
    c[0]()
torch.cuda.synchronize()
assert all(torch.equal(a, c[1]) and a.any() and int(c[2].item()) == 0 for a, c in zip(got, calls))
print("ok")
"""


@pytest.mark.parametrize("kind", ["sparse", "paged", "linear"])
def test_first_calls(kind):
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", PROGRAM, ROOT, kind], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-600:]
