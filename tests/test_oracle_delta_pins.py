"""Pins of the fp64 definitions of oracle/delta.py: worked by hand, against differences, against torch's own
rounding to e4m3."""
import numpy as np
import pytest
import torch

from oracle import delta as R


def test_one_key_by_hand():
    """One channel each way, k = q = 1, no decay: S <- S + beta (v - S), an exponential average."""
    one = np.ones((1, 3, 1, 1))
    v = np.array([4.0, 8.0, 2.0]).reshape(1, 3, 1, 1)
    o, S = R.gated_delta(one, one, v, np.zeros((1, 3, 1)), np.full((1, 3, 1), 0.5), scale=1.0)
    assert np.allclose(o[0, :, 0, 0], [2.0, 5.0, 3.5]) and S[0, 0, 0, 0] == 3.5
    # half forgotten before each step: S' = S / 2
    o, _ = R.gated_delta(one, one, v, np.full((1, 3, 1), np.log(0.5)), np.full((1, 3, 1), 0.5), scale=2.0)
    assert np.allclose(o[0, :, 0, 0], 2 * np.array([2.0, 4.5, 2.125]))


def test_a_full_correction_replaces_the_value():
    """beta = 1 and a unit key: reading with that key gives the value just written, whatever was there."""
    rng = np.random.default_rng(0)
    q = rng.standard_normal((1, 5, 1, 6))
    v = rng.standard_normal((1, 5, 2, 3))
    h0 = rng.standard_normal((1, 2, 6, 3))
    o, _ = R.gated_delta(q, q, v, -rng.random((1, 5, 2)), np.ones((1, 5, 2)), scale=1.0, l2norm=True, h0=h0)
    assert np.allclose(o, v, atol=1e-5)  # (the 1e-6 under the root)


def test_a_reset_starts_anew():
    rng = np.random.default_rng(1)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    q, k, v, g, b = n(2, 9, 1, 4), n(2, 9, 1, 4), n(2, 9, 2, 3), -rng.random((2, 9, 2)), rng.random((2, 9, 2))
    reset = np.zeros((2, 9), np.uint8)
    reset[:, 4] = 1
    h0 = np.full((2, 2, 4, 3), np.inf)
    o, S = R.gated_delta(q, k, v, g, b, l2norm=True, reset=reset, h0=np.where(reset[:, :1, None, None] > 0, h0, 1.0))
    part = lambda t: t[:, 4:]  # noqa: E731
    o2, S2 = R.gated_delta(part(q), part(k), part(v), part(g), part(b), l2norm=True)
    assert np.array_equal(o[:, 4:], o2) and np.array_equal(S, S2)


@pytest.mark.parametrize("l2norm", [False, True])
def test_gradients_against_differences(l2norm):
    """Central differences of sum(o do) + sum(S dS) at h = 1e-5: their own error is about h^2 and 1e-16 / h."""
    rng = np.random.default_rng(2)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    x = dict(q=n(2, 6, 2, 3), k=0.5 * n(2, 6, 2, 3), v=n(2, 6, 4, 2), g=-rng.random((2, 6, 4)), beta=rng.random((2, 6, 4)),
             h0=n(2, 4, 3, 2))
    do, dS = n(2, 6, 4, 2), n(2, 4, 3, 2)
    reset = np.zeros((2, 6), np.uint8)
    reset[1, 3] = 1
    kw = dict(l2norm=l2norm, reset=reset)

    def loss(**y):
        o, S = R.gated_delta(**y, **kw)
        return (o * do).sum() + (S * dS).sum()

    got = R.gated_delta_bwd(**x, do=do, dh_final=dS, **kw)
    for name, t in x.items():
        for _ in range(12):
            at = tuple(rng.integers(0, d) for d in t.shape)
            up, down = t.copy(), t.copy()
            up[at] += 1e-5
            down[at] -= 1e-5
            want = (loss(**dict(x, **{name: up})) - loss(**dict(x, **{name: down}))) / 2e-5
            assert abs(got["d" + name][at] - want) < 1e-6 * (1 + abs(want)), (name, at)
    assert (got["dg"][1, 3] == 0).all()


def test_e4m3_rounds_as_torch_does():
    x = torch.cat([torch.linspace(-448, 448, 20001), torch.linspace(-0.02, 0.02, 4001),
                   torch.arange(-256, 257) / 2.0 ** 10, torch.arange(-100, 101) * 4.5])
    x = x[x.abs() <= 448]
    assert np.array_equal(R.e4m3(x.double().numpy()), x.to(torch.float8_e4m3fn).double().numpy())


def test_block_scales_and_product():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 300))
    x[2, 128:256] = 0
    s = R.block_scales(x, 1)
    assert s.shape == (5, 3) and s[2, 1] == np.float64(np.float32(2.0 ** -100 / 448))
    assert np.allclose(s[0], [np.abs(x[0, a:b]).max() / 448 for a, b in ((0, 128), (128, 256), (256, 300))])
    w = rng.standard_normal((130, 300))
    t = R.block_scales(w, 128)
    assert t.shape == (2, 3)
    xq, wq = R.e4m3(x / R.spread(s, 1, 5, 300)), R.e4m3(w / R.spread(t, 128, 130, 300))
    y, size = R.matmul_blocks(xq, s, wq, t)
    assert np.abs(y - x @ w.T).max() < 2.0 ** -3 * (np.abs(x) @ np.abs(w).T).max() and (size >= np.abs(y)).all()
