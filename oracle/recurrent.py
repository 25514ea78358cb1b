"""fp64 definitions of the gated recurrence and the fused norms (numpy, one step or row at a
time), for the test suite only.  Shares no code with the HIP library.

Beside each result stands a bound on what an fp32 evaluation of the same formulas may be off by:
`u` = 2^-24 is half a unit in the last place of an fp32 value, so every operation perturbs its
result by a factor within 1 + c u with c = 1 for a correctly rounded operation and c = 2 for the
hardware's exponential, reciprocal, square root and reciprocal root (1 ulp).
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def sig(v):
    with np.errstate(over="ignore"):
        return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def gates(mode, x, gate, A=None, in_gate=None, gate_bias=None, in_bias=None):
    """a, b = w x, and the relative errors (in units of u) an fp32 evaluation may give a and w."""
    g = gate if gate_bias is None else gate + gate_bias
    if mode == "decay":
        return dict(a=gate, w=np.ones_like(x), ca=np.zeros_like(x), cw=np.zeros_like(x), x=x)
    # exp2 of -(gate + bias) log2 e: log2 e itself, the products and the sum move the argument by
    # 3 u of |gate| + |bias|; the exponential 2, the sum 1, the reciprocal 2 and one product 1 follow
    cs = 3 * (np.abs(gate) + (0 if gate_bias is None else np.abs(gate_bias))) + 6
    if mode == "sigmoid":
        return dict(a=sig(-g), w=sig(g), ca=cs, cw=cs, x=x, s=sig(g), c=sig(-g))
    r = sig(g)
    la = A * r
    # log a = A r: its relative error is cs + 1, then as above for the exponential
    ca = np.abs(la) * (cs + 4) + 2
    with np.errstate(invalid="ignore"):
        q = np.maximum(-np.expm1(2 * la), 0.0)
    # q = 1 - a^2: relative error of its argument (cs + 2) at worst as it is (|dq/q| <= |dw/w|);
    # the series adds 6 operations, the difference 1 - a^2 at most 3 / q with q > 0.11
    cq = cs + 2 + 28
    w = np.sqrt(q)
    cw = 0.5 * cq + 4
    i = np.ones_like(x)
    if in_gate is not None:
        gi = in_gate if in_bias is None else in_gate + in_bias
        i = sig(gi)
        cw = cw + 3 * (np.abs(in_gate) + (0 if in_bias is None else np.abs(in_bias))) + 7
    return dict(a=np.exp(la), w=w * i, ca=ca, cw=cw, x=x, r=r, beta=w, i=i, cs=cs, cq=cq)


def _run(a, b, first, cut, err_a, err_b, first_err):
    """h_t = a_t h_{t-1} + b_t along axis 1 from `first`, with a majorant of |h| and a bound of
    the error: every surviving term carries its decays' relative errors, one product and one sum
    per step (in whatever order they are formed), so 4 u a step beside the decay's own."""
    B, L, D = b.shape
    h, maj, err = first.copy(), np.abs(first), first_err.copy()
    H, M, E = (np.empty((B, L, D)) for _ in range(3))
    for t in range(L):
        keep = np.ones((B, 1)) if cut is None else 1.0 - cut[:, t, None]
        at = np.abs(a[:, t]) * keep
        err = at * (err + (err_a[:, t] + 4) * U * maj) + (err_b[:, t] + 4) * U * np.abs(b[:, t])
        maj = at * maj + np.abs(b[:, t])
        h = np.where(keep > 0, a[:, t] * h, 0.0) + b[:, t]
        H[:, t], M[:, t], E[:, t] = h, maj, err
    return H, M, E


def gated_scan(mode, x, gate, A=None, in_gate=None, gate_bias=None, in_bias=None, reset=None, h0=None):
    """(h, majorant of |h|, fp32 error bound), each (B, L, D)."""
    c = gates(mode, x, gate, A, in_gate, gate_bias, in_bias)
    B, L, D = x.shape
    first = np.zeros((B, D)) if h0 is None else h0
    cut = None if reset is None else (reset != 0).astype(np.float64)
    return _run(c["a"], c["w"] * x, first, cut, c["ca"], c["cw"] + 1, np.zeros((B, D)))


def gated_scan_bwd(mode, x, gate, dy, A=None, in_gate=None, gate_bias=None, in_bias=None, reset=None, h0=None,
                   dh_final=None):
    """{name: (gradient, fp32 error bound)}."""
    c = gates(mode, x, gate, A, in_gate, gate_bias, in_bias)
    B, L, D = x.shape
    a, w = c["a"], c["w"]
    first = np.zeros((B, D)) if h0 is None else h0
    cut = np.zeros((B, L)) if reset is None else (reset != 0).astype(np.float64)
    H, M, E = _run(a, w * x, first, cut, c["ca"], c["cw"] + 1, np.zeros((B, D)))
    prev = np.concatenate([first[:, None], H[:, :-1]], 1)
    pmaj = np.concatenate([np.abs(first)[:, None], M[:, :-1]], 1)
    perr = np.concatenate([np.zeros((B, 1, D)), E[:, :-1]], 1)
    # mu_t = a_t (dy_t + mu_{t+1}) backwards from dh_final, lambda_t = dy_t + mu_{t+1}
    mu = np.zeros((B, D)) if dh_final is None else dh_final
    mmaj, merr = np.abs(mu), np.zeros((B, D))
    lam, lmaj, lerr = (np.empty((B, L, D)) for _ in range(3))
    for t in range(L - 1, -1, -1):
        lam[:, t] = dy[:, t] + mu
        lmaj[:, t] = np.abs(dy[:, t]) + mmaj
        lerr[:, t] = merr + 2 * U * lmaj[:, t]
        keep = 1.0 - cut[:, t, None]
        mu = keep * a[:, t] * lam[:, t]
        merr = keep * np.abs(a[:, t]) * (lerr[:, t] + (c["ca"][:, t] + 4) * U * lmaj[:, t])
        mmaj = keep * np.abs(a[:, t]) * lmaj[:, t]
    keep = 1.0 - cut[:, :, None]
    da = keep * lam * prev
    damaj, daerr = keep * lmaj * pmaj, keep * (lerr * pmaj + lmaj * perr + 2 * U * lmaj * pmaj)
    out = {}
    if mode == "decay":
        out["dx"], out["dgate"] = (lam, lerr), (da, daerr)
        return _finish(out, None, h0, (mu, merr))
    if mode == "sigmoid":
        s, cc = c["s"], c["c"]
        out["dx"] = (lam * s, lerr * s + (c["cw"] + 2) * U * lmaj * s)
        v = (lam * x - da) * s * cc
        e = (lerr * np.abs(x) + daerr + (2 * c["cw"] + 6) * U * (lmaj * np.abs(x) + damaj)) * s * cc
        out["dgate"] = (v, e)
        sums = {} if gate_bias is None else {"dgate_bias": (v, e, (lmaj * np.abs(x) + damaj) * s * cc)}
        return _finish(out, sums, h0, (mu, merr))
    beta, i, r = c["beta"], c["i"], c["r"]
    rs = np.where(beta > 0, 1 / np.where(beta > 0, beta, 1), 0.0)
    out["dx"] = (lam * beta * i, (lerr + (c["cw"] + 4) * U * lmaj) * beta * i)
    sums = {}
    if in_gate is not None:
        m = lmaj * beta * np.abs(x) * i * (1 - i)
        v, e = lam * beta * x * i * (1 - i), lerr * beta * np.abs(x) * i * (1 - i) + (2 * c["cw"] + 6) * U * m
        out["din_gate"] = (v, e)
        if in_bias is not None:
            sums["din_bias"] = (v, e, m)
    dla = a * (da - lam * i * x * a * rs)
    k = a * rs * np.abs(x) * i
    maj = a * (damaj + lmaj * k)
    e = a * (daerr + lerr * k) + (3 * c["ca"] + 2 * c["cw"] + c["cq"] + 10) * U * maj
    out["dgate"] = (dla * A * r * (1 - r), (e + (2 * c["cs"] + 3) * U * maj) * np.abs(A) * r * (1 - r))
    sums["dA"] = (dla * r, (e + (c["cs"] + 1) * U * maj) * r, maj * r)
    if gate_bias is not None:
        sums["dgate_bias"] = out["dgate"] + (maj * np.abs(A) * r * (1 - r),)
    return _finish(out, sums, h0, (mu, merr))


def _finish(out, sums, h0, dh0):
    for k, (v, e, maj) in (sums or {}).items():
        # a sum of n terms in any order with at most 512 additions in a row
        n = min(512, v.shape[0] * v.shape[1])
        out[k] = (v.sum((0, 1)), e.sum((0, 1)) + n * U * maj.sum((0, 1)))
    if h0 is not None:
        out["dh0"] = dh0
    return out


def _rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def _norm_bwd(dyw, v, k):
    return k * dyw - v * k ** 3 * (dyw * v).mean(-1, keepdims=True)


def add_rmsnorm(x, w, residual=None, scale=None, post_w=None, eps=1e-5):
    u = x if post_w is None else x * _rms(x, eps) * post_w
    r = u if scale is None else scale * u
    if residual is not None:
        r = residual + r
    return r * _rms(r, eps) * w, r


def add_rmsnorm_bwd(x, w, residual, dy, dres=None, scale=None, post_w=None, eps=1e-5):
    k = None if post_w is None else _rms(x, eps)
    u = x if k is None else x * k * post_w
    _, r = add_rmsnorm(x, w, residual, scale, post_w, eps)
    q = _rms(r, eps)
    dr = _norm_bwd(dy * w, r, q)
    if dres is not None:
        dr = dr + dres
    out = {"dw": (dy * r * q).sum(0)}
    if residual is not None:
        out["dresidual"] = dr
    du = dr
    if scale is not None:
        out["dscale"] = (dr * u).sum(0)
        du = dr * scale
    if k is not None:
        out["dpost_w"] = (du * x * k).sum(0)
        du = _norm_bwd(du * post_w, x, k)
    out["dx"] = du
    return out


def gated_rmsnorm(x, z, w, groups=1, gate_first=True, eps=1e-5):
    R, D = x.shape
    g = z * sig(z)
    v = (x * g if gate_first else x).reshape(R, groups, D // groups)
    y = (v * _rms(v, eps)).reshape(R, D) * w
    return y if gate_first else y * g


def gated_rmsnorm_bwd(x, z, w, dy, groups=1, gate_first=True, eps=1e-5):
    R, D = x.shape
    s = sig(z)
    g, slope = z * s, s * (1 + z * (1 - s))
    cut = lambda t: t.reshape(R, groups, D // groups)  # noqa: E731
    v = cut(x * g if gate_first else x)
    k = _rms(v, eps)
    inner = dy if gate_first else dy * g
    n = (v * k).reshape(R, D)
    dv = _norm_bwd(cut(inner * w), v, k).reshape(R, D)
    dw = (inner * n).sum(0)
    if gate_first:
        return {"dx": dv * g, "dz": dv * x * slope, "dw": dw}
    return {"dx": dv, "dz": dy * n * w * slope, "dw": dw}
