"""fp64 definitions of the gated delta rule and of e4m3 with block scales (numpy, one step at a time),
for the test suite only.  Shares no code with the HIP library.

A bound on what an fp32 evaluation may be off by stands beside the gated delta rule: the maps a state
goes through do not lengthen it where the decays are at most 1 and beta |k|^2 lies in [0, 2], so an error
made in one chunk reaches the end no larger than it was made, and the chunks' errors add up.  In a chunk a
result goes through at most four products (K S, the inverse, the update, the output; as many backwards),
each a sum of at most K, V or 64 terms in two parts, every term rounded to a factor within 1 + 2^-24.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
CHUNK = 64
L2_EPS = 1e-6


def relative_bound(L, K, V):
    """What an fp32 result may be off by, relative to the largest value of its tensor."""
    return 4 * (max(K, V) + 2 * CHUNK) * -(-L // CHUNK) * U


def _unit(x, l2norm):
    r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) + L2_EPS) if l2norm else np.ones(x.shape[:-1] + (1,))
    return x * r, r


def _setup(q, k, v, g, scale, l2norm, reset):
    heads = v.shape[2] // q.shape[2]
    (qh, rq), (kh, rk) = _unit(q, l2norm), _unit(k, l2norm)
    spread = lambda t: np.repeat(t, heads, axis=2)  # noqa: E731
    a = np.exp(g)
    if reset is not None:
        a = np.where(reset[..., None] != 0, 0.0, a)
    return heads, spread(qh), spread(kh), rq, rk, a, q.shape[-1] ** -0.5 if scale is None else scale


def gated_delta(q, k, v, g, beta, scale=None, l2norm=False, reset=None, h0=None, keep=False):
    """(o, final state), and with `keep` the states before each step too."""
    heads, qh, kh, _, _, a, scale = _setup(q, k, v, g, scale, l2norm, reset)
    B, L, H, V = v.shape
    S = np.zeros((B, H, q.shape[-1], V)) if h0 is None else h0.copy()
    o, states = np.empty_like(v), []
    for t in range(L):
        if keep:
            states.append(S)
        S = np.where(a[:, t, :, None, None] != 0, a[:, t, :, None, None] * S, 0.0)
        e = v[:, t] - np.einsum("bhkv,bhk->bhv", S, kh[:, t])
        S = S + kh[:, t, :, :, None] * (beta[:, t, :, None] * e)[:, :, None]
        o[:, t] = scale * np.einsum("bhkv,bhk->bhv", S, qh[:, t])
    return (o, S, states) if keep else (o, S)


def gated_delta_bwd(q, k, v, g, beta, do, scale=None, l2norm=False, reset=None, h0=None, dh_final=None):
    """{name: gradient}."""
    _, final, states = gated_delta(q, k, v, g, beta, scale, l2norm, reset, h0, keep=True)
    heads, qh, kh, rq, rk, a, scale = _setup(q, k, v, g, scale, l2norm, reset)
    B, L, H, V = v.shape
    dq, dk = np.zeros_like(qh), np.zeros_like(kh)
    dv, dg, dbeta = np.zeros_like(v), np.zeros_like(g), np.zeros_like(beta)
    dS = np.zeros_like(final) if dh_final is None else dh_final.copy()
    for t in reversed(range(L)):
        at, kt, qt, bt = a[:, t, :, None, None], kh[:, t], qh[:, t], beta[:, t, :, None]
        old = np.where(at != 0, at * states[t], 0.0)
        e = v[:, t] - np.einsum("bhkv,bhk->bhv", old, kt)
        new = old + kt[..., None] * (bt * e)[:, :, None]
        dq[:, t] = scale * np.einsum("bhkv,bhv->bhk", new, do[:, t])
        dS = dS + scale * qt[..., None] * do[:, t][:, :, None]
        du = np.einsum("bhkv,bhk->bhv", dS, kt)
        dbeta[:, t] = (du * e).sum(-1)
        dv[:, t] = bt * du
        dk[:, t] = np.einsum("bhkv,bhv->bhk", dS, bt * e) - np.einsum("bhkv,bhv->bhk", old, bt * du)
        dS = dS - kt[..., None] * (bt * du)[:, :, None]
        dg[:, t] = (dS * old).sum((-1, -2))
        dS = np.where(at != 0, at * dS, 0.0)
    out = dict(dv=dv, dg=dg, dbeta=dbeta)
    for name, x, r, d in (("dq", q, rq, dq), ("dk", k, rk, dk)):
        d = d.reshape(B, L, q.shape[2], heads, -1).sum(3)
        out[name] = r * (d - x * r * (x * r * d).sum(-1, keepdims=True)) if l2norm else d
    if h0 is not None:
        out["dh0"] = dS
    return out


# ------------------------------------------------------------------------------- e4m3
def e4m3(x):
    """To the nearest of e4m3's values, ties to the one with the even last bit (|x| <= 448): from 2^-6 on
    three bits stand behind the leading one, below it the steps stay those of 2^-6."""
    x = np.asarray(x, np.float64)
    with np.errstate(divide="ignore"):
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.rint(x / step) * step


def block_scales(x, rows):
    """max(largest magnitude, 2^-100) / 448, rounded to fp32, per block of `rows` x 128."""
    M, D = x.shape
    out = np.empty((-(-M // rows), -(-D // 128)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = max(np.abs(x[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]).max(), 2.0 ** -100)
    return (out / 448).astype(np.float32).astype(np.float64)


def spread(scales, rows, M, D):
    """A block's scale at each of its elements."""
    return np.repeat(np.repeat(scales, rows, 0)[:M], 128, 1)[:, :D]


def matmul_blocks(xq, sx, wq, sw):
    """(x w^T, the same of magnitudes) of e4m3 values with block scales."""
    x, w = xq * spread(sx, 1, *xq.shape), wq * spread(sw, 128, *wq.shape)
    return x @ w.T, np.abs(x) @ np.abs(w).T
