"""The gated recurrent block of README.md runs as written (needs an MI355X)."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_gated_block_example_runs():
    text = open(os.path.join(ROOT, "README.md")).read()
    block = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "gated_scan_step" in b]
    assert len(block) == 1
    env = {}
    exec(compile(block[0], "README.md", "exec"), env)
    torch.cuda.synchronize()
    assert env["out"].shape == (4, 2048, 1536) and env["out1"].shape == (4, 1536)
    for k, w in env["w"].items():
        assert w.grad is not None and torch.isfinite(w.grad.float()).all() and w.grad.any(), k
    assert torch.isfinite(env["state"]).all() and torch.isfinite(env["out1"].float()).all()
