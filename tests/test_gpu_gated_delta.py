"""The gated delta rule on the GPU against its fp64 definition (needs an MI355X)."""
import numpy as np
import pytest
import torch

import selective_state_space_59_amd as ssm
from oracle import delta as R
from tests.delta_helpers import bound, case64, close, delta_case
from tests.recurrent_helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
IDS = dict(argvalues=[F32, BF], ids=["f32", "bf16"])
# B, L, Hk, H, K, V: single steps, lengths around a chunk's, key and value widths off their tiles'
SHAPES = [(1, 1, 1, 1, 8, 8), (2, 2, 1, 2, 16, 24), (1, 63, 2, 2, 64, 64), (2, 64, 1, 1, 128, 128),
          (1, 65, 3, 6, 72, 40), (2, 130, 2, 4, 40, 136), (1, 300, 1, 4, 128, 256), (3, 200, 2, 2, 24, 8)]


def _one(k, grads=True, checkpoints=True, seed=0):
    B, L, Hk, K = k["q"].shape
    H, V = k["v"].shape[2:]
    ck = torch.full(ssm.gated_delta_checkpoint_shape(B, L, H, K, V), float("nan"), device=DEV) if checkpoints else None
    o, hf = ssm.gated_delta_fwd(return_final_state=True, checkpoints=ck, **k)
    if not grads:
        return o, hf
    g = torch.Generator().manual_seed(seed)
    do = torch.randn(B, L, H, V, generator=g).to(k["q"].dtype).to(DEV)
    dhf = 0.3 * torch.randn(B, H, K, V, generator=g).to(DEV) if "h0" in k else None
    return o, hf, do, dhf, ssm.gated_delta_bwd(do=do, dh_final=dhf, checkpoints=ck, **k)


def _check(k, what, **kw):
    print(what, flush=True)
    o, hf, do, dhf, got = _one(k, **kw)
    torch.cuda.synchronize()
    k64, rel = case64(k), bound(k)
    ro, rs = R.gated_delta(**k64)
    close(o, ro, rel, what + " o")
    close(hf, rs, rel, what + " h_final")
    ref = R.gated_delta_bwd(do=f64(do), dh_final=f64(dhf), **k64)
    assert set(ref) == set(got)
    for n, v in ref.items():
        close(got[n], v, rel, "%s %s" % (what, n))


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_gradients(shape, dtype):
    for i, (l2norm, doc, h0, beta, ck) in enumerate([(True, 0, False, 1.0, True), (True, 20, True, 2.0, True),
                                                     (False, 0, True, 1.0, False), (False, 3, False, 1.9, False)]):
        k = delta_case(*shape, dtype, seed=i, l2norm=l2norm, doc=doc, h0=h0, beta=beta)
        _check(k, "%s l2norm=%d doc=%d h0=%d ck=%d" % (shape, l2norm, doc, h0, ck), checkpoints=ck)


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("shape", [(64, 70, 2, 4, 16, 8), (32, 3, 8, 8, 128, 24), (16, 65, 4, 8, 72, 40), (86, 66, 1, 1, 64, 72)],
                         ids=lambda s: "x".join(map(str, s)))
def test_slices_of_32_channels(shape, dtype):
    """Chains enough for a workgroup to take 32 value channels, the last slice of 8, 24, 8 and 8 of them."""
    k = delta_case(*shape, dtype, seed=sum(shape), doc=40)
    _check(k, "%s" % (shape,))


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("shape", [(1, 2048, 1, 1, 128, 128), (1, 2100, 2, 2, 72, 24), (2, 2090, 1, 3, 40, 136),
                                   (1, 4100, 1, 2, 8, 8), (1, 2049, 4, 4, 128, 264),
                                   (1, 3100, 2, 16, 72, 104), (1, 3100, 1, 5, 16, 344)], ids=lambda s: "x".join(map(str, s)))
def test_segments(shape, dtype):
    """Sequences of 32 to 65 chunks and few heads, which are run in segments, in slices of 16 and (the last two)
    of 32 value channels; memories of more steps than a segment, resets in all, some and none of the segments."""
    for i, (l2norm, doc, h0, beta, ck) in enumerate([(True, 0, True, 2.0, True), (True, 600, True, 1.0, False),
                                                     (False, 40, False, 1.0, True)]):
        k = delta_case(*shape, dtype, seed=i, l2norm=l2norm, doc=doc, h0=h0, beta=beta)
        k["g"] = k["g"] * 0.02
        _check(k, "%s l2norm=%d doc=%d h0=%d ck=%d" % (shape, l2norm, doc, h0, ck), checkpoints=ck)


@pytest.mark.parametrize("dtype", **IDS)
def test_segments_of_states_that_are_dropped(dtype):
    """A state of infinities and NaNs, dropped in the first, a middle or the last segment, stays out of what
    follows; what comes before holds them, as the definition's does."""
    L = 64 * 39 + 20
    for at in (0, 70, 64 * 13 + 5, 64 * 38 + 1):
        k = delta_case(1, L, 1, 2, 64, 48, dtype, seed=at)
        k["reset"] = torch.zeros(1, L, dtype=torch.uint8, device=DEV)
        k["reset"][:, at] = 1
        zero = dict(k, h0=torch.zeros_like(k["h0"]))
        bad = dict(k, h0=k["h0"].clone())
        bad["h0"][:, :, ::3] = float("inf")
        bad["h0"][:, :, 1::3] = float("nan")
        o, hf = ssm.gated_delta_fwd(return_final_state=True, **bad)
        ro, rs = ssm.gated_delta_fwd(return_final_state=True, **zero)
        assert torch.equal(o[:, at:], ro[:, at:]) and torch.equal(hf, rs)


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("shape", [(1, 1, 1, 8, 8), (3, 2, 4, 128, 128), (5, 1, 3, 72, 40), (2, 4, 4, 64, 136),
                                   (130, 2, 2, 24, 32)], ids=lambda s: "x".join(map(str, s)))
def test_step(shape, dtype):
    B, Hk, H, K, V = shape
    for l2norm in (True, False):
        k = delta_case(B, 3, Hk, H, K, V, dtype, seed=B, l2norm=l2norm, doc=3)
        k64 = case64(k)
        ro, rs = R.gated_delta(**k64)
        state = k["h0"].clone()
        for t in range(3):
            at = {n: k[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta", "reset")}
            o = ssm.gated_delta_step(state, l2norm=l2norm, **at)
            close(o, ro[:, t], R.relative_bound(64, K, V), "step %d" % t)
        close(state, rs, 3 * R.relative_bound(64, K, V), "state")
