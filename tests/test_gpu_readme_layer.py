"""The README's Python blocks run in a row; the last one's results against fp64."""
import os
import re

import numpy as np
import pytest
import torch

from oracle import layer as L

pytestmark = pytest.mark.gpu


def test_every_block_of_the_readme():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    with open(path, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)
    assert len(blocks) == 3
    torch.manual_seed(0)
    env = {}
    for block in blocks:
        exec(compile(block, "README.md", "exec"), env)
    torch.cuda.synchronize()
    # the projection of the rows that the norm wrote: 2^-8 of its own rounding, 128 * 2^-23 and 26 * 2^-24 of its sums
    want, size = L.linear(env["codes"].cpu().numpy(), env["scales"].cpu().numpy(), env["w8"].cpu().numpy(),
                          env["w_scales"].cpu().numpy())
    lim = (128 * 2.0 ** -23 + 26 * 2.0 ** -24) * size
    assert (np.abs(env["qkv"].double().cpu().numpy() - want) <= lim + 2.0 ** -8 * (np.abs(want) + lim)).all()
    # one token per request: the attention's output is its V, as the cache holds it
    v = env["heads"][:, env["H"] + env["G"]:]
    out = env["out"].view(env["T"], env["G"], -1, 128)
    assert torch.equal(out, v[:, :, None].expand_as(out))
