"""The precision of bf16 calls of the gated delta rule (needs an MI355X): products with what was computed
carry 24 bits of it, which the fp32 results show (tests/test_delta_planes.py: operands of 16 bits do not
pass)."""
import numpy as np
import pytest
import torch

import selective_state_space_59_amd as ssm
from oracle import delta as R
from tests import delta_planes as P
from tests.delta_helpers import case64
from tests.recurrent_helpers import f64
from tests.test_delta_planes import run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _to(k):
    return {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in k.items()}


@pytest.mark.parametrize("shape", P.SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_operands_of_24_bits(shape):
    """States, checkpoints, errors, the first state's gradient and the gates', head by head."""
    B, L, Hk, H, K, V = shape
    k, do, dhf = P.case(*shape)
    ck = torch.empty(ssm.gated_delta_checkpoint_shape(B, L, H, K, V), device=DEV)
    _, hf = ssm.gated_delta_fwd(return_final_state=True, checkpoints=ck, **_to(k))
    d = ssm.gated_delta_bwd(do=do.to(DEV), dh_final=dhf.to(DEV), checkpoints=ck, **_to(k))
    d2 = ssm.gated_delta_bwd(do=do.to(DEV), dh_final=dhf.to(DEV), **_to(k))
    k64 = case64(k)
    _, state, states = R.gated_delta(keep=True, **k64)
    grads = R.gated_delta_bwd(do=f64(do), dh_final=f64(dhf), **k64)
    got = dict(h_final=f64(hf), ck=f64(ck), dh0=f64(d["dh0"]), dg=f64(d["dg"]), dh0_2=f64(d2["dh0"]), dg_2=f64(d2["dg"]))
    for b in range(B):
        for h in range(H):
            size = run(k, do, dhf, b, h)[1]
            off = dict(h_final=P.off(got["h_final"][b, h], state[b, h], L, state[b, h]))
            for c in range(ck.shape[0]):
                entering = states[64 * c][b, h]
                off["state %d" % c] = P.off(got["ck"][c, b, h, :K], entering, L, entering)
            for again in ("", "_2"):
                off["dh0" + again] = P.off(got["dh0" + again][b, h], grads["dh0"][b, h], L, grads["dh0"][b, h])
                off["dg" + again] = P.off(got["dg" + again][b, :, h], grads["dg"][b, :, h], L, size, P.DG_UNITS)
            print(shape, b, h, {n: round(float(x), 2) for n, x in off.items()}, flush=True)
            assert max(off.values()) < 1


@pytest.mark.parametrize("heads", [2, 3])
def test_segments_keep_them(heads):
    """The same across the segments of a long sequence, whose states pass through join_kernel."""
    B, L, K, V = 1, 64 * 40, 32, 24
    k, do, dhf = P.case(B, L, 1, heads, K, V)
    k["g"] = 0.2 * k["g"]
    _, hf = ssm.gated_delta_fwd(return_final_state=True, **_to(k))
    state = R.gated_delta(**case64(k))[1]
    for h in range(heads):
        off = P.off(f64(hf)[0, h], state[0, h], L, state[0, h])
        print(h, off, flush=True)
        assert off < 1
