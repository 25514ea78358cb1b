"""The gated delta layer of README.md runs as written (needs an MI355X)."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_gated_delta_example_runs():
    text = open(os.path.join(ROOT, "README.md")).read()
    block = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "gated_delta_step" in b]
    assert len(block) == 1
    env = {}
    exec(compile(block[0], "README.md", "exec"), env)
    torch.cuda.synchronize()
    assert env["o"].shape == (2, 512, 6, 128) and env["o1"].shape == (2, 6, 128) and env["y1"].shape == (2, 768)
    grad = env["w_in"].grad
    assert torch.isfinite(grad.float()).all() and grad.any()
    for name in ("o", "state", "o1", "y1"):
        assert torch.isfinite(env[name].float()).all(), name
