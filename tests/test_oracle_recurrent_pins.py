"""The fp64 definitions of the gated recurrence and the fused norms against other things than
themselves: closed forms, the pinned S6 oracle, torch autograd and finite differences."""
import numpy as np
import pytest
import torch

import oracle
from oracle import recurrent as R


def _inputs(mode, B=2, L=7, D=5, seed=0, in_gate=True, bias=True):
    g = np.random.default_rng(seed)
    n = lambda *s: g.standard_normal(s)  # noqa: E731
    kw = dict(x=n(B, L, D), gate=1 / (1 + np.exp(-n(B, L, D))) if mode == "decay" else n(B, L, D))
    if mode == "rate":
        kw["A"] = -g.uniform(0.05, 3.0, D)
        if in_gate:
            kw["in_gate"] = n(B, L, D)
            if bias:
                kw["in_bias"] = n(D)
    if mode != "decay" and bias:
        kw["gate_bias"] = n(D)
    kw["reset"] = (g.random((B, L)) < 0.25).astype(np.uint8)
    kw["h0"] = n(B, D)
    return kw


def test_sigmoid_mode_is_the_scan_with_one_state():
    """S6 with N = 1, A = -1, B = C = 1 and delta = softplus(gate) is the gated RNN of Theorem 1."""
    k = _inputs("sigmoid", L=40, bias=False)
    x, gate = k["x"], k["gate"]
    one = np.ones((2, 40, 1))
    y, h = oracle.selective_scan(x, np.log1p(np.exp(gate)), -np.ones((5, 1)), one, one, h0=k["h0"][:, :, None])
    H, _, _ = R.gated_scan("sigmoid", x, gate, h0=k["h0"])
    np.testing.assert_allclose(H, y, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(H[:, -1], h[:, :, 0], rtol=1e-12, atol=1e-13)


def test_constant_decay_is_a_geometric_sum():
    x = np.random.default_rng(1).standard_normal((1, 30, 1))
    H, _, _ = R.gated_scan("decay", x, np.full_like(x, 0.7))
    want = [sum(0.7 ** (t - s) * x[0, s, 0] for s in range(t + 1)) for t in range(30)]
    np.testing.assert_allclose(H[0, :, 0], want, rtol=1e-12)


def test_rate_mode_keeps_unit_variance():
    g = np.random.default_rng(2)
    x = g.standard_normal((1, 4000, 200))
    H, _, _ = R.gated_scan("rate", x, np.zeros_like(x), A=np.full(200, -0.2))
    assert abs(H[:, 500:].var() - 1.0) < 0.02


@pytest.mark.parametrize("mode", ["decay", "sigmoid", "rate"])
def test_packed_documents_equal_calls_of_their_own(mode):
    k = _inputs(mode, B=1, L=12)
    k["reset"] = np.zeros((1, 12), np.uint8)
    k["reset"][0, [4, 9]] = 1
    H, _, _ = R.gated_scan(mode, **k)
    for lo, hi in ((0, 4), (4, 9), (9, 12)):
        part = {n: v[:, lo:hi] if n in ("x", "gate", "in_gate") else v for n, v in k.items()}
        part["reset"], part["h0"] = None, k["h0"] if lo == 0 else None
        np.testing.assert_array_equal(H[:, lo:hi], R.gated_scan(mode, **part)[0])


@pytest.mark.parametrize("mode", ["decay", "sigmoid", "rate"])
def test_gradients_match_finite_differences(mode):
    k = _inputs(mode)
    g = np.random.default_rng(7)
    dy, dh = g.standard_normal(k["x"].shape), g.standard_normal(k["h0"].shape)

    def loss(kw):
        H, _, _ = R.gated_scan(mode, **kw)
        return (H * dy).sum() + (H[:, -1] * dh).sum()

    got = R.gated_scan_bwd(mode, dy=dy, dh_final=dh, **k)
    names = {"x": "dx", "gate": "dgate", "in_gate": "din_gate", "A": "dA", "gate_bias": "dgate_bias",
             "in_bias": "din_bias", "h0": "dh0"}
    assert set(got) == {names[n] for n in k if n in names}
    for n, grad in names.items():
        if n not in k:
            continue
        want = np.zeros_like(k[n])
        for idx in np.ndindex(*k[n].shape):
            e = 1e-6
            hi, lo = dict(k), dict(k)
            hi[n], lo[n] = k[n].copy(), k[n].copy()
            hi[n][idx] += e
            lo[n][idx] -= e
            want[idx] = (loss(hi) - loss(lo)) / (2 * e)
        np.testing.assert_allclose(got[grad][0], want, rtol=2e-6, atol=2e-7, err_msg=n)


def _t(a):
    return torch.tensor(a, dtype=torch.float64, requires_grad=True)


@pytest.mark.parametrize("post,scale,res", [(False, False, True), (True, True, True), (False, True, False)])
def test_add_norm_against_torch(post, scale, res):
    g = np.random.default_rng(3)
    n = lambda *s: g.standard_normal(s)  # noqa: E731
    k = dict(x=n(4, 6), w=n(6), residual=n(4, 6) if res else None, scale=n(6) if scale else None,
             post_w=n(6) if post else None)
    dy, dres = n(4, 6), n(4, 6)
    t = {m: None if v is None else _t(v) for m, v in k.items()}
    u = t["x"] if not post else torch.nn.functional.rms_norm(t["x"], (6,), t["post_w"], 1e-5)
    r = u if not scale else u * t["scale"]
    r = r if not res else r + t["residual"]
    y = torch.nn.functional.rms_norm(r, (6,), t["w"], 1e-5)
    got_y, got_r = R.add_rmsnorm(**k)
    np.testing.assert_allclose(got_y, y.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(got_r, r.detach().numpy(), rtol=1e-12)
    torch.autograd.backward([y, r], [torch.tensor(dy), torch.tensor(dres)])
    got = R.add_rmsnorm_bwd(k["x"], k["w"], k["residual"], dy, dres, k["scale"], k["post_w"])
    for m, v in t.items():
        if v is not None:
            np.testing.assert_allclose(got["d" + m], v.grad.numpy(), rtol=1e-10, atol=1e-12, err_msg=m)


@pytest.mark.parametrize("groups", [1, 3])
@pytest.mark.parametrize("gate_first", [True, False])
def test_gated_norm_against_torch(groups, gate_first):
    g = np.random.default_rng(4)
    x, z, dy = (g.standard_normal((4, 12)) for _ in range(3))
    w = g.standard_normal(12)
    t = [_t(v) for v in (x, z, w)]
    gate = torch.nn.functional.silu(t[1])
    v = (t[0] * gate if gate_first else t[0]).view(4, groups, -1)
    y = torch.nn.functional.rms_norm(v, (12 // groups,), None, 1e-5).view(4, 12) * t[2]
    y = y if gate_first else y * gate
    np.testing.assert_allclose(R.gated_rmsnorm(x, z, w, groups, gate_first), y.detach().numpy(), rtol=1e-12)
    y.backward(torch.tensor(dy))
    got = R.gated_rmsnorm_bwd(x, z, w, dy, groups, gate_first)
    for name, u in zip(("dx", "dz", "dw"), t):
        np.testing.assert_allclose(got[name], u.grad.numpy(), rtol=1e-10, atol=1e-12, err_msg=name)


def test_the_fp32_error_bound_holds_for_an_fp32_evaluation_in_torch():
    """The bound the GPU is held to, applied to a plain sequential fp32 evaluation on the CPU."""
    for mode in ("decay", "sigmoid", "rate"):
        k = _inputs(mode, B=1, L=300, D=40, seed=9)
        k = {n: v.astype(np.float32).astype(np.float64) if v.dtype != np.uint8 else v for n, v in k.items()}
        H, _, E = R.gated_scan(mode, **k)
        f = {n: torch.tensor(v, dtype=torch.float32) if v.dtype != np.uint8 else torch.tensor(v) for n, v in k.items()}
        g = f["gate"] + f["gate_bias"] if "gate_bias" in f else f["gate"]
        if mode == "decay":
            a, b = g, f["x"]
        elif mode == "sigmoid":
            a, b = torch.sigmoid(-g), torch.sigmoid(g) * f["x"]
        else:
            la = f["A"] * torch.sigmoid(g)
            a = torch.exp(la)
            b = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(f["in_gate"] + f["in_bias"]) * f["x"]
        h = f["h0"]
        for t in range(300):
            h = torch.where(f["reset"][:, t, None] != 0, 0.0, a[:, t] * h) + b[:, t]
            off = np.abs(h.double().numpy() - H[:, t])
            assert (off <= E[:, t]).all(), (mode, t, float((off / E[:, t]).max()))
