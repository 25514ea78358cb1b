"""Inputs and tolerances of the gated delta rule's tests.

Inputs are drawn on the CPU in fp32 and rounded to their type; the fp64 definitions (oracle/delta.py)
read the rounded values.  A result may be off by its fp32 bound, relative to the largest value of its
tensor, plus one rounding to its own type: half a step of bf16 is at most 2^-8 of the value, of fp32
2^-24."""
import numpy as np
import torch

from oracle import delta as R
from tests.recurrent_helpers import HALF_STEP, f64


def delta_case(B, L, Hk, H, K, V, dtype, seed, l2norm=True, doc=0, h0=True, beta=1.0, device="cuda", grow=0.0):
    """Keyword arguments of a gated_delta_fwd call."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    k = dict(q=n(B, L, Hk, K), k=n(B, L, Hk, K), v=n(B, L, H, V).to(dtype))
    if not l2norm:  # keys the rule is stable for all the same
        k["k"] = k["k"] / k["k"].norm(dim=-1, keepdim=True)
        k["q"] = k["q"] * 0.3
    k["q"], k["k"] = k["q"].to(dtype), k["k"].to(dtype)
    rate = torch.exp(-6 * torch.rand(H, generator=g))  # memories of 1 to 400 steps
    k["g"] = grow - rate * torch.nn.functional.softplus(n(B, L, H))
    k["beta"] = (beta * torch.sigmoid(n(B, L, H))).to(dtype)
    if doc:
        k["reset"] = (torch.rand(B, L, generator=g) < 1.0 / doc).to(torch.uint8)
    if h0:
        k["h0"] = 0.3 * n(B, H, K, V)
    k = {m: v.to(device) for m, v in k.items()}
    return dict(k, l2norm=l2norm)


def case64(k):
    return {m: f64(v) if isinstance(v, torch.Tensor) else v for m, v in k.items()}


def close(got, ref, rel, what, roundings=1):
    """|got - ref| <= rel max|ref| + half a step of got's type for each of `roundings` (two where ref was
    rounded to that type as well)."""
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    if not ref.size:
        return
    tol = rel * np.abs(ref).max() + roundings * HALF_STEP[got.dtype] * np.abs(ref) + 1e-37
    off = np.abs(g - ref)
    bad = ~(off <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(off), np.inf, off / tol)), off.shape)
        raise AssertionError("%s: %d of %d outside; worst at %s: got %r, want %r, tolerance %.3e"
                             % (what, bad.sum(), bad.size, i, g[i], ref[i], tol[i]))


def bound(k):
    L, K, V = k["q"].shape[1], k["q"].shape[-1], k["v"].shape[-1]
    return R.relative_bound(L, K, V)
