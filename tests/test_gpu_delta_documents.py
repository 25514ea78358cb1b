"""Sequences packed into a row of the gated delta rule do not meet (needs an MI355X)."""
import pytest
import torch

import selective_state_space_59_amd as ssm
from tests.delta_helpers import delta_case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
IDS = dict(argvalues=[F32, BF], ids=["f32", "bf16"])
GRADS = ("dq", "dk", "dv", "dg", "dbeta")


def _given(k):
    B, L, _, K = k["q"].shape
    H, V = k["v"].shape[2:]
    return torch.empty(ssm.gated_delta_checkpoint_shape(B, L, H, K, V), device=DEV)


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("at", [17, 40, 64, 80])
def test_gradients_of_one_document_do_not_show_in_another(at, dtype):
    """Whatever arrives at the outputs behind a reset, the gradients ahead of it are the same bits."""
    k = delta_case(2, 130, 2, 4, 40, 24, dtype, seed=at)
    k["reset"] = torch.zeros(2, 130, dtype=torch.uint8, device=DEV)
    k["reset"][:, at] = 1
    do = torch.randn(k["v"].shape, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    behind = torch.zeros(1, 130, 1, 1, device=DEV, dtype=dtype)
    behind[:, at:] = 1
    one, other = (ssm.gated_delta_bwd(do=torch.where(behind == 1, x * do, do), **k) for x in (0.0, 1e6))
    for n in GRADS:
        assert torch.equal(one[n][:, :at], other[n][:, :at]), n
    assert torch.equal(one["dh0"], other["dh0"])


@pytest.mark.parametrize("dtype", **IDS)
def test_gradients_behind_a_dropped_state_of_infinities(dtype):
    """An entering state of infinities and NaNs, with the checkpoints its forward wrote and without: what
    does not depend on the state (dv, dh0), and all gradients behind the reset, are those of a state of zeros."""
    L = 150
    k = delta_case(2, L, 1, 2, 40, 24, dtype, seed=4)
    k["reset"] = torch.zeros(2, L, dtype=torch.bool, device=DEV)
    k["reset"][0, 0] = True
    k["reset"][1, 70] = True
    good = dict(k, h0=torch.zeros_like(k["h0"]))
    bad = dict(k, h0=k["h0"].clone())
    bad["h0"][0] = float("nan")
    bad["h0"][1] = float("inf")
    do = torch.randn(k["v"].shape, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    dhf = torch.randn(k["h0"].shape, generator=torch.Generator().manual_seed(2)).to(DEV)
    cks = _given(k), _given(k)
    for c, ck in zip((good, bad), cks):
        ssm.gated_delta_fwd(checkpoints=ck, **c)
    want = ssm.gated_delta_bwd(do=do, dh_final=dhf, checkpoints=cks[0], **good)
    for ck in (cks[1], None):
        got = ssm.gated_delta_bwd(do=do, dh_final=dhf, checkpoints=ck, **bad)
        assert torch.equal(got["dv"], want["dv"]) and torch.equal(got["dh0"], want["dh0"])
        for n in GRADS:
            assert torch.equal(got[n][0], want[n][0]) and torch.equal(got[n][1, 70:], want[n][1, 70:]), n
            assert torch.isfinite(got[n][1, 70:].float()).all(), n
