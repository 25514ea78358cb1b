"""What the check of the delta rule's precision can tell (no GPU needed): the chunk form with operands of
three bf16 numbers passes it, and does not with two in any one of its products."""
import numpy as np
import pytest
import torch

from oracle import delta as R
from tests import delta_planes as P
from tests.delta_helpers import case64
from tests.recurrent_helpers import f64


def run(k, do, dhf, b, h, planes=None):
    """The chunk form of row b's head h."""
    one = {n: f64(t)[b].astype(np.float32) for n, t in k.items() if n not in ("h0", "l2norm")}
    hk = h * k["q"].shape[2] // k["v"].shape[2]
    unit = lambda x: x / np.sqrt((x * x).sum(-1, keepdims=True) + np.float32(1e-6))  # noqa: E731
    f32 = lambda t: f64(t)[b, h].astype(np.float32)  # noqa: E731
    return P.head(unit(one["q"][:, hk]), unit(one["k"][:, hk]), one["v"][:, h], one["g"][:, h], one["beta"][:, h],
                  f32(k["h0"]), k["q"].shape[-1] ** -0.5, f64(do)[b, :, h].astype(np.float32), f32(dhf), planes)


def shares(shape, planes=None):
    k, do, dhf = P.case(*shape)
    k64 = case64(k)
    grads = R.gated_delta_bwd(do=f64(do), dh_final=f64(dhf), **k64)
    got, size = run(k, do, dhf, 0, 0, planes)
    L = shape[1]
    state, dstate = R.gated_delta(**k64)[1][0, 0], grads["dh0"][0, 0]
    return dict(h_final=P.off(got["h_final"], state, L, state), dh0=P.off(got["dh0"], dstate, L, dstate),
                dg=P.off(got["dg"], grads["dg"][0, :, 0], L, size, P.DG_UNITS))


@pytest.mark.parametrize("shape", P.SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_three_planes_pass(shape):
    assert max(shares(shape).values()) < 0.75


@pytest.mark.parametrize("of,name", [("h_final", n) for n in P.FORWARD] + [("dh0", n) for n in P.BACKWARD]
                         + [("dg", n) for n in P.GATES])
def test_two_planes_show(of, name):
    """A plane lost in one product shows at one of the shapes at least."""
    worst = max(shares(shape, {name: 2})[of] for shape in P.SHAPES)
    print(of, name, worst)
    assert worst > 1
