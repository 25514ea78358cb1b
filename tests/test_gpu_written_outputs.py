"""Calls that write into a tensor they are given count as in-place changes for autograd: a backward
whose saved tensor was overwritten raises instead of returning gradients of other values (needs
an MI355X)."""
import pytest
import torch

import selective_state_space_59_amd as ssm
from tests.recurrent_helpers import scan_case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32 = torch.float32


def _rows(*shape):
    return torch.randn(*shape, device=DEV)


def _writes():
    """{name: (call, the tensors it writes)} for every tensor a call of these operators may be given
    to write into."""
    B, L, D = 2, 130, 40
    k = scan_case("rate", B, L, D, F32, seed=1)
    one = {m: v[:, 0].contiguous() if m in ("x", "gate", "in_gate") else v for m, v in k.items() if m != "h0"}
    x, z, w = _rows(6, D), _rows(6, D), torch.ones(D, device=DEV)
    y, hf, ck = torch.empty_like(k["x"]), _rows(B, D), torch.empty(ssm.gated_checkpoint_shape(B, L, D), device=DEV)
    state, ys = _rows(B, D), _rows(B, D)
    res, out, zn = x.clone(), torch.empty_like(x), z.clone()
    return dict(
        scan=(lambda: ssm.gated_scan_fwd(y=y, h_final=hf, checkpoints=ck, **k), [y, hf, ck]),
        step=(lambda: ssm.gated_scan_step(state, y=ys, **one), [state, ys]),
        add_norm=(lambda: ssm.add_rmsnorm_fwd(x, w, res, y=out, res_out=res), [out, res]),
        gated_norm=(lambda: ssm.gated_rmsnorm_fwd(x, zn, w, y=zn), [zn]))


@pytest.mark.parametrize("name", ["scan", "step", "add_norm", "gated_norm"])
def test_every_given_output_is_marked(name):
    call, written = _writes()[name]
    before = [t._version for t in written]
    call()
    assert all(t._version > v for t, v in zip(written, before))
    with torch.inference_mode():  # where tensors have no versions the call runs as before
        call, _ = _writes()[name]
        call()


def test_a_stream_updated_in_place_before_its_backward():
    x, w = _rows(5, 48).requires_grad_(), torch.ones(48, device=DEV)
    stream = _rows(5, 48)
    y, _ = ssm.add_rmsnorm(x, w, stream)
    ssm.add_rmsnorm_fwd(_rows(5, 48), w, stream, res_out=stream)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_a_state_advanced_before_the_backward_that_entered_with_it():
    k = scan_case("decay", 2, 20, 24, F32, seed=2)
    state = k.pop("h0")
    x = k.pop("x").requires_grad_()
    y, _ = ssm.gated_scan(x, h0=state, **k)
    ssm.gated_scan_step(state, _rows(2, 24), _rows(2, 24), "decay")
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_a_gate_overwritten_by_its_norm():
    x, z, w = _rows(5, 48).requires_grad_(), _rows(5, 48), torch.ones(48, device=DEV)
    y = ssm.gated_rmsnorm(x, z, w)
    ssm.gated_rmsnorm_fwd(_rows(5, 48), z, w, y=z)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_outputs_of_their_own_disturb_nothing():
    """The differentiable ops' own writes (their checkpoints among them) and calls on other tensors
    leave a backward alone."""
    k = scan_case("rate", 2, 200, 40, F32, seed=3)
    x = k.pop("x").requires_grad_()
    y, hf = ssm.gated_scan(x, **k)
    r = ssm.add_rmsnorm(y, torch.ones(40, device=DEV), x)[0]
    out = ssm.gated_rmsnorm(r, k["gate"], torch.ones(40, device=DEV))
    ssm.gated_scan_step(hf.detach().clone(), _rows(2, 40), _rows(2, 40), "decay")
    out.sum().backward()
    assert torch.isfinite(x.grad).all()
