"""What the recurrences' torch ops keep and pass on (needs an MI355X)."""
import pytest
import torch

import selective_state_space_59_amd as ssm
from selective_state_space_59_amd import ssm as capi
from tests.delta_helpers import delta_case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _args():
    k = delta_case(2, 300, 2, 4, 64, 64, torch.bfloat16, seed=1)
    k.pop("l2norm")
    return k


def _spy(monkeypatch, name):
    calls, real = [], getattr(capi, name)

    def call(*a, **kw):
        calls.append(kw)
        return real(*a, **kw)
    monkeypatch.setattr(capi, name, call)
    return calls


def test_no_checkpoints_where_no_gradient_is_recorded(monkeypatch):
    """A learnable first state under no_grad, or inputs that ask for nothing: the forward writes no
    checkpoints, and gives the bits that it gives with them."""
    calls = _spy(monkeypatch, "gated_delta_fwd")
    k = _args()
    with torch.no_grad():
        plain = ssm.gated_delta(l2norm=True, **k)
    k["h0"] = k["h0"].requires_grad_()
    with torch.no_grad():
        learnable = ssm.gated_delta(l2norm=True, **k)
    recorded = ssm.gated_delta(l2norm=True, **k)
    assert [c["checkpoints"] is not None for c in calls] == [False, False, True]
    for o in (plain, learnable):
        assert torch.equal(o[0], recorded[0]) and torch.equal(o[1], recorded[1])
    assert not learnable[0].requires_grad and recorded[0].requires_grad


def test_gradients_of_the_outputs_that_were_used(monkeypatch):
    """A loss of the outputs alone, of the final state alone, and of both: what is not there is not read as
    zeros, and counts as zeros all the same."""
    calls = _spy(monkeypatch, "gated_delta_bwd")
    k = _args()
    n = torch.Generator().manual_seed(4)
    do = torch.randn(k["v"].shape, generator=n).bfloat16().to(DEV)
    dhf = torch.randn(k["h0"].shape, generator=n).to(DEV)
    names = ("q", "k", "v", "g", "beta", "h0")
    for of_o, of_state in ((True, False), (False, True), (True, True)):
        leaves = {m: k[m].clone().requires_grad_() for m in names}
        o, hf = ssm.gated_delta(l2norm=True, **leaves)
        outs = [(t, d) for t, d, used in ((o, do, of_o), (hf, dhf, of_state)) if used]
        torch.autograd.backward(*zip(*outs))
        assert (calls[-1]["dh_final"] is None) == (not of_state)
        want = ssm.gated_delta_bwd(*(k[m] for m in names[:5]), do if of_o else torch.zeros_like(do), l2norm=True,
                                   h0=k["h0"], dh_final=dhf if of_state else torch.zeros_like(dhf))
        for m in names:
            assert torch.equal(leaves[m].grad, want["d" + m]), m


def test_none_of_the_gated_scan_either(monkeypatch):
    calls = _spy(monkeypatch, "gated_scan_fwd")
    n = torch.Generator().manual_seed(2)
    x, gate = (torch.randn(2, 300, 64, generator=n).to(DEV) for _ in range(2))
    A = -torch.rand(64, generator=n).to(DEV)
    A.requires_grad_()
    with torch.no_grad():
        y, hf = ssm.gated_scan(x, gate, A=A)
    recorded = ssm.gated_scan(x, gate, A=A)
    assert [c["checkpoints"] is not None for c in calls] == [False, True]
    assert torch.equal(y, recorded[0]) and torch.equal(hf, recorded[1])
    assert not y.requires_grad and recorded[0].requires_grad
