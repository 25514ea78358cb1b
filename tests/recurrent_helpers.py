"""Inputs and tolerances of the gated-recurrence and norm tests.

Inputs are drawn on the CPU in fp32 and rounded to the I/O type; the fp64 definitions
(oracle/recurrent.py) read the rounded values.  A result may differ from them by the fp32 error
bound of the formula plus one rounding to its own type, half a step: 2^-9 of the value's binade,
so at most 2^-8 relative to the value in bf16; 2^-24 in fp32.
"""
import numpy as np
import torch

from oracle.recurrent import U

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def check(got, ref, bound, what):
    """|got - ref| <= bound + half a step of got's type at |ref| + bound, element by element
    (1e-37: results below the normal range may be flushed to 0)."""
    half = HALF_STEP[got.dtype]
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    tol = bound + half * (np.abs(ref) + bound) + 1e-37
    off = np.abs(g - ref)
    bad = ~(off <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(off), np.inf, off / tol)), off.shape)
        raise AssertionError("%s: %d of %d outside; worst at %s: got %r, want %r, tolerance %.3e"
                             % (what, bad.sum(), bad.size, i, g[i], ref[i], tol[i]))


def scan_case(mode, B, L, D, dtype, seed, in_gate=True, bias=True, doc=0, h0=True, device="cuda"):
    """Keyword arguments of a gated_scan_fwd call."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    k = dict(x=n(B, L, D).to(dtype), mode=mode)
    if mode == "decay":
        k["gate"] = (2 * torch.rand(B, L, D, generator=g) - 1).abs().sqrt().to(dtype)
        k["gate"][:, :, ::3] *= -1  # decays of either sign
    else:
        k["gate"] = n(B, L, D).to(dtype)
    if mode == "rate":
        k["A"] = -torch.exp(-6 * torch.rand(D, generator=g))  # memories of 1 to 1000 steps
        if in_gate:
            k["in_gate"] = n(B, L, D).to(dtype)
            if bias:
                k["in_bias"] = n(D)
    if mode != "decay" and bias:
        k["gate_bias"] = n(D)
    if doc:
        k["reset"] = (torch.rand(B, L, generator=g) < 1.0 / doc).to(torch.uint8)
    if h0:
        k["h0"] = n(B, D)
    return {m: v.to(device) if isinstance(v, torch.Tensor) else v for m, v in k.items()}


def scan_case64(k):
    out = {m: f64(v) if isinstance(v, torch.Tensor) else v for m, v in k.items()}
    return out


def norm_bound(x, w, residual, scale, post_w, dy=None, dres=None, eps=1e-5):
    """Majorants of the boundary's results (the same formulas on absolute values) times the
    relative error an fp32 evaluation may collect: `depth` additions in a row for a mean over D
    (lanes of 8 or 64 share a row, so D / 8 at most for short rows and D / 64 + 16 beyond),
    halved by the square root, a few operations more, cubed at worst in a gradient, and the
    cancellation of residual + scale u (kappa) where a norm follows it."""
    D = x.shape[-1]
    depth = min(D, 64) / 8 + D / 64 + 16
    ax, aw = np.abs(x), np.abs(w)
    k = None if post_w is None else 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = ax if k is None else ax * k * np.abs(post_w)
    su = u if scale is None else u * np.abs(scale)
    rmaj = su if residual is None else np.abs(residual) + su
    us = x if k is None else x * k * post_w
    us = us if scale is None else us * scale
    r = us if residual is None else residual + us
    q = 1 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    kappa = np.sqrt((rmaj ** 2).mean(-1, keepdims=True)) * q + 1
    rel = (2 * depth + 40) * kappa * U
    b = {"res_out": rmaj * (depth + 10) * U, "y": rmaj * q * aw * rel}
    if dy is None:
        return b
    ady = np.abs(dy)
    dr = q * aw * ady + rmaj * q ** 3 * (ady * aw * rmaj).mean(-1, keepdims=True)
    if dres is not None:
        dr = dr + np.abs(dres)
    n = min(512 + x.shape[0] / 64, x.shape[0])  # rows added up in a row for a column sum
    s = lambda m: ((rel + n * U) * m).sum(0)  # noqa: E731
    b["dw"] = s(ady * rmaj * q)
    b["dresidual"] = rel * dr
    du = dr
    if scale is not None:
        b["dscale"] = s(dr * u)
        du = du * np.abs(scale)
    if k is not None:
        b["dpost_w"] = s(du * ax * k)
        du = du * np.abs(post_w)
        du = k * du + ax * k ** 3 * (du * ax).mean(-1, keepdims=True)
    b["dx"] = 2 * rel * du
    return b


def gnorm_bound(x, z, w, groups, gate_first, dy=None, eps=1e-5):
    """As norm_bound; the gate's logistic adds 3 |z| + 7 operations (oracle/recurrent.py)."""
    R, D = x.shape
    S = D // groups
    depth = min(S, 64) / 8 + S / 64 + 16
    s = np.where(z >= 0, 1, np.exp(-np.abs(z))) / (1 + np.exp(-np.abs(z)))
    g = np.abs(z) * s
    # |silu'| <= sig (1 + |z| (1 - sig)), and 1 - sig itself may be off by U where sig is near 1
    slope = s * (1 + np.abs(z) * (1 - s)) + np.abs(z) * s
    ax, aw = np.abs(x), np.abs(w)
    v = ax * g if gate_first else ax
    per = lambda t: t.reshape(R, groups, S).mean(-1, keepdims=True).repeat(S, -1).reshape(R, D)  # noqa: E731
    k = 1 / np.sqrt(per(v * v) + eps)
    rel = (2 * depth + 60 + 9 * np.abs(z).max()) * U
    b = {"y": v * k * aw * rel if gate_first else v * k * aw * g * rel}
    if dy is None:
        return b
    ady = np.abs(dy)
    inner = ady if gate_first else ady * g
    dv = k * inner * aw + v * k ** 3 * per(inner * aw * v)
    n = min(512 + R / 64, R)
    b["dw"] = ((rel + n * U) * inner * v * k).sum(0)
    b["dx"] = rel * (dv * g if gate_first else dv)
    b["dz"] = rel * (dv * ax * slope if gate_first else ady * v * k * aw * slope)
    return b
