"""The selective scan's, the conv's, the block's and the SSD layer's calls that write into a tensor
they are given count as in-place changes for autograd (needs an MI355X)."""
import pytest
import torch

import selective_state_space_59_amd as ssm
from selective_state_space_59_amd import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32 = torch.float32


def _rows(*shape, dtype=F32):
    return torch.randn(*shape, device=DEV).to(dtype)


def _scan_inputs(B=2, L=40, D=32, N=16):
    return dict(x=_rows(B, L, D), delta=torch.rand(B, L, D, device=DEV), A=-torch.rand(D, N, device=DEV),
                Bm=_rows(B, L, N), Cm=_rows(B, L, N))


def _writes():
    """{name: (call, the tensors it writes)}."""
    B, L, D, N = 2, 40, 32, 16
    k = _scan_inputs(B, L, D, N)
    conv = _rows(D, 4)
    y, hf, cs = _rows(B, L, D), _rows(B, D, N), _rows(B, 3, D)
    ck = torch.empty(ssm.checkpoint_shape(B, L, D), device=DEV)
    y2, hf2, out, state, win = _rows(B, L, D), _rows(B, D, N), _rows(B, L, D), _rows(B, D, N), _rows(B, 3, D)
    t = lambda m: k[m][:, 0].contiguous()  # noqa: E731
    s = W.make_ssd_inputs(B, L, 4, 32, 1, 64, seed=1, device=DEV, gate=False, skip=False)
    sy, sh = torch.empty_like(s["x"]), torch.zeros(B, 4, 32, 64, device=DEV)
    st, sy1 = torch.zeros(B, 4, 32, 64, device=DEV), torch.empty_like(s["x"][:, 0].contiguous())
    c = lambda m: s[m][:, 0].contiguous()  # noqa: E731
    h = W.make_block_inputs(2, 64, 64, 128, 16, 4, device=DEV)
    names = ("norm_w", "w_in", "conv_w", "conv_b", "w_x", "w_dt", "dt_bias", "A", "Dskip", "w_out")
    return dict(
        scan=(lambda: ssm.selective_scan_fwd(**k, conv_w=conv, y=y, h_final=hf, conv_state_out=cs, checkpoints=ck),
              [y, hf, cs, ck]),
        noalloc=(lambda: ssm.selective_scan_fwd_noalloc(**k, y=y2, h_final=hf2), [y2, hf2]),
        conv=(lambda: ssm.causal_conv1d_silu(k["x"], conv, out=out), [out]),
        update=(lambda: ssm.state_update(state, t("x"), t("delta"), k["A"], t("Bm"), t("Cm"), conv_w=conv,
                                         conv_state=win), [state, win]),
        ssd=(lambda: ssm.ssd_fwd(s["x"], s["delta"], s["A"], s["Bm"], s["Cm"], y=sy, h_final=sh), [sy, sh]),
        ssd_step=(lambda: ssm.ssd_step(st, c("x"), c("delta"), s["A"], c("Bm"), c("Cm"), y=sy1), [st, sy1]),
        block=(lambda: ssm.mamba_block_fwd(h["h"], *(h[n] for n in names), out=h["h"]), [h["h"]]))


@pytest.mark.parametrize("name", ["scan", "noalloc", "conv", "update", "ssd", "ssd_step", "block"])
def test_every_given_output_is_marked(name):
    call, written = _writes()[name]
    before = [t._version for t in written]
    call()
    assert all(t._version > v for t, v in zip(written, before))


def test_a_state_advanced_before_the_backward_that_entered_with_it():
    k = _scan_inputs()
    x, state = k.pop("x").requires_grad_(), _rows(2, 32, 16)
    y, _ = ssm.selective_scan(x, **k, h0=state)
    t = lambda m: k[m][:, 0].contiguous()  # noqa: E731
    ssm.state_update(state, _rows(2, 32), t("delta"), k["A"], t("Bm"), t("Cm"))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_a_residual_stream_updated_by_a_block():
    """A stream that add_rmsnorm saved, then updated in place by the block call."""
    h = W.make_block_inputs(2, 64, 64, 128, 16, 4, device=DEV)
    names = ("norm_w", "w_in", "conv_w", "conv_b", "w_x", "w_dt", "dt_bias", "A", "Dskip", "w_out")
    x = _rows(2, 64, 64, dtype=torch.bfloat16).requires_grad_()
    y, _ = ssm.add_rmsnorm(x, torch.ones(64, device=DEV), h["h"])
    ssm.mamba_block_fwd(h["h"], *(h[n] for n in names), out=h["h"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
