"""Cases, plain forms and 64-bit definitions of the gated recurrence and the fused norms.

Three operators of a recurrent block:

  gated scan     h_t = a_t h_{t-1} + b_t per channel, with a_t and b_t from gates; forward,
                 forward + backward, and one decode token on a resident state
  add + RMSNorm  the boundary between two blocks: r = residual + scale u, y = RMSNorm(r) w,
                 u = x or its own (post-)norm; forward, and forward + backward
  gated RMSNorm  y = RMSNorm(x silu(z)) w over groups of channels, or RMSNorm(x) w silu(z);
                 forward, and forward + backward

`run` computes a case in elementary torch operations in 32 bits, or, where `own` is set, with
the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------------------------ cases
def _scan(name, op, mode, dtype, B, L, D, in_gate=False, bias=False, doc=0, h0=False):
    return dict(name=name, op=op, mode=mode, dtype=dtype, B=B, L=L, D=D, in_gate=in_gate, bias=bias,
                doc=doc, h0=h0)


def _norm(name, op, dtype, rows, D, res="bf16", post=False, scale=False):
    return dict(name=name, op=op, dtype=dtype, rows=rows, D=D, res=res, post=post, scale=scale)


def _gnorm(name, op, dtype, rows, D, groups=1, gate_first=True):
    return dict(name=name, op=op, dtype=dtype, rows=rows, D=D, groups=groups, gate_first=gate_first)


def listed():
    return [
        # one chat, one token: the width of a 130M-like layer; latency is all that counts
        _scan("step_one_sequence", "scan_step", "rate", "bf16", 1, 1, 1536, in_gate=True, bias=True),
        # decode of 256 sequences at the width of a 2.8B-like layer
        _scan("step_256_sequences", "scan_step", "rate", "bf16", 256, 1, 5120, in_gate=True, bias=True),
        # fine-tuning of an odd-sized fp32 model on packed documents, state carried between calls
        _scan("scan_odd_f32_packed", "scan_train", "decay", "f32", 3, 1237, 331, doc=200, h0=True),
        # prefill of the 130M-like layer's batch
        _scan("scan_layer", "scan_fwd", "rate", "bf16", 8, 2048, 1536, in_gate=True, bias=True),
        # one DNA-like sequence of a million tokens
        _scan("scan_1m_tokens", "scan_fwd", "rate", "bf16", 1, 1 << 20, 1024, in_gate=True, bias=True),
        # a training step of the 130M-like layer
        _scan("scan_layer_train", "scan_train", "rate", "bf16", 8, 2048, 1536, in_gate=True, bias=True),
        # a training step at the 2.8B-like width on packed documents
        _scan("scan_wide_train_packed", "scan_train", "sigmoid", "bf16", 4, 4096, 5120, bias=True, doc=700),
        # the norm ahead of a block when 256 sequences decode (d_model 2560)
        _norm("add_norm_decode", "norm_fwd", "bf16", 256, 2560),
        # a training step, 130M-like d_model, residual stream in fp32
        _norm("add_norm_train", "norm_train", "bf16", 16384, 768, res="f32"),
        # the same with a norm behind the block and a residual scale, 2.8B-like d_model
        _norm("add_norm_post_train", "norm_train", "bf16", 16384, 2560, post=True, scale=True),
        # the norm behind the SSD layer of the Mamba-2 130M-like model, prefill
        _gnorm("gated_norm_prefill", "gnorm_fwd", "bf16", 16384, 1536),
        # a training step at the 2.7B-like width, 8 groups
        _gnorm("gated_norm_train_groups", "gnorm_train", "bf16", 16384, 5120, groups=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_step", "scan_fwd", "scan_train", "scan_train", "norm_fwd", "norm_train",
                     "gnorm_fwd", "gnorm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("scan"):
        mode = rng.choice(["decay", "sigmoid", "rate"])
        D = _log(rng, 24, 5120)
        if rng.random() < 0.6:
            D = max(8, D // 8 * 8)
        B = _log(rng, 1, 256) if op == "scan_step" else _log(rng, 1, 16)
        L = 1 if op == "scan_step" else min(_log(rng, 3, 60000), max(3, (1 << 26) // (B * D)))
        return dict(op=op, mode=mode, dtype=dtype, B=B, L=L, D=D, in_gate=mode == "rate" and rng.random() < 0.7,
                    bias=mode != "decay" and rng.random() < 0.7,
                    doc=0 if op == "scan_step" else rng.choice([0, 0, _log(rng, 20, 2000)]),
                    h0=rng.random() < 0.4)
    D = _log(rng, 48, 8192)
    if rng.random() < 0.7:
        D = max(16, D // 16 * 16)
    rows = min(_log(rng, 1, 40000), (1 << 26) // D)
    if op.startswith("norm"):
        return dict(op=op, dtype=dtype, rows=rows, D=D, res="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                    post=rng.random() < 0.4, scale=rng.random() < 0.4)
    groups = rng.choice([g for g in (1, 2, 4, 8, 16) if D % g == 0 and D // g >= 16])
    return dict(op=op, dtype=dtype, rows=rows, D=D, groups=groups, gate_first=rng.random() < 0.6)


# ----------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    io = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    s = dict(case)
    if case["op"].startswith("scan"):
        B, L, D, mode = case["B"], case["L"], case["D"], case["mode"]
        shape = (B, D) if case["op"] == "scan_step" else (B, L, D)
        s["x"] = randn(*shape, dtype=io)
        if mode == "decay":
            s["gate"] = torch.sigmoid(randn(*shape, mean=2.0)).to(io)
        else:
            s["gate"] = randn(*shape, mean=-2.0 if mode == "sigmoid" else 0.0, dtype=io)
        s["ig"] = randn(*shape, dtype=io) if case["in_gate"] else None
        # rates so that the channels remember about 10 to 1000 steps
        s["A"] = None
        if mode == "rate":
            s["A"] = -0.2 * torch.exp(-math.log(100.0) * torch.rand(D, generator=g, device="cuda"))
        s["gb"] = randn(D, std=0.3) if case["bias"] else None
        s["ib"] = randn(D, std=0.3) if case["bias"] and case["in_gate"] else None
        s["reset"] = None
        if case["doc"]:
            s["reset"] = (torch.rand(B, L, generator=g, device="cuda") < 1.0 / case["doc"]).to(torch.uint8)
        s["h0"] = randn(B, D) if case["h0"] else None
        if case["op"] == "scan_step":
            s["state"] = randn(B, D)
        if case["op"] == "scan_train":
            s["dy"] = randn(*shape, dtype=io)
    else:
        rows, D = case["rows"], case["D"]
        s["x"] = randn(rows, D, dtype=io)
        s["w"] = randn(D, std=0.1, mean=1.0)
        if case["op"].startswith("gnorm"):
            s["z"] = randn(rows, D, dtype=io)
        else:
            s["residual"] = randn(rows, D, std=2.0, dtype=DTYPES[case["res"]])
            s["scale"] = randn(D, std=0.1, mean=0.5) if case["scale"] else None
            s["post_w"] = randn(D, std=0.1, mean=1.0) if case["post"] else None
        if case["op"].endswith("train"):
            s["dy"] = randn(rows, D, dtype=io)
            if case["op"] == "norm_train":
                s["dres"] = randn(rows, D, dtype=DTYPES[case["res"]])
    return s


def run(s):
    if own:
        return _own(s)
    return {"scan_step": _plain_step, "scan_fwd": _plain_scan, "scan_train": _plain_scan_train,
            "norm_fwd": _plain_norm, "norm_train": _plain_norm_train, "gnorm_fwd": _plain_gnorm,
            "gnorm_train": _plain_gnorm_train}[s["op"]](s)


# --------------------------------------------------------------------- the library's calls
def _own(s):
    import selective_state_space_59_amd as ssm
    op = s["op"]
    if op.startswith("scan"):
        kw = dict(mode=s["mode"], A=s["A"], in_gate=s["ig"], gate_bias=s["gb"], in_bias=s["ib"])
        if op == "scan_step":
            y = ssm.gated_scan_step(s["state"], s["x"], s["gate"], **kw)
            return y, s["state"]
        kw.update(reset=s["reset"], h0=s["h0"])
        if op == "scan_fwd":
            return ssm.gated_scan_fwd(s["x"], s["gate"], return_final_state=True, **kw)
        ck = torch.empty(ssm.gated_checkpoint_shape(*s["x"].shape), device=s["x"].device)
        y, hf = ssm.gated_scan_fwd(s["x"], s["gate"], return_final_state=True, checkpoints=ck, **kw)
        return y, hf, ssm.gated_scan_bwd(s["x"], s["gate"], s["dy"], checkpoints=ck, **kw)
    if op.startswith("norm"):
        y, r = ssm.add_rmsnorm_fwd(s["x"], s["w"], s["residual"], scale=s["scale"], post_w=s["post_w"], eps=EPS)
        if op == "norm_fwd":
            return y, r
        return y, r, ssm.add_rmsnorm_bwd(s["x"], s["w"], s["residual"], s["dy"], s["dres"], scale=s["scale"],
                                         post_w=s["post_w"], eps=EPS)
    y = ssm.gated_rmsnorm_fwd(s["x"], s["z"], s["w"], groups=s["groups"], gate_first=s["gate_first"], eps=EPS)
    if op == "gnorm_fwd":
        return y
    return y, ssm.gated_rmsnorm_bwd(s["x"], s["z"], s["w"], s["dy"], groups=s["groups"],
                                    gate_first=s["gate_first"], eps=EPS)


# -------------------------------------------------------------------------------- plain forms
def _f(t):
    return None if t is None else t.float()


def _coefficients(s):
    """a, b and what the gradients need of the gates, in fp32."""
    x, g = s["x"].float(), s["gate"].float()
    if s["gb"] is not None:
        g = g + s["gb"]
    if s["mode"] == "decay":
        return g, x, dict(x=x)
    if s["mode"] == "sigmoid":
        sg = torch.sigmoid(g)
        return torch.sigmoid(-g), sg * x, dict(x=x, s=sg)
    r = torch.sigmoid(g)
    la = s["A"] * r
    a = torch.exp(la)
    beta = torch.sqrt(-torch.expm1(2 * la))
    i = None
    if s["ig"] is not None:
        i = s["ig"].float()
        i = torch.sigmoid(i if s["ib"] is None else i + s["ib"])
    b = beta * x if i is None else beta * i * x
    return a, b, dict(x=x, r=r, a=a, beta=beta, i=i)


def _doubling(a, h):
    """h_t = a_t h_{t-1} + h_t along dim 1, in place, by doubling the reach of every step."""
    a, step, L = a.clone(), 1, h.shape[1]
    while step < L:
        more = a[:, step:] * h[:, :-step]
        grown = a[:, step:] * a[:, :-step]
        h[:, step:] += more
        a[:, step:] = grown
        step *= 2
    return h


def _plain_states(s):
    a, b, c = _coefficients(s)
    if s["reset"] is not None:
        a = torch.where(s["reset"].bool().unsqueeze(-1), 0.0, a)
    h = b.clone()
    if s["h0"] is not None:
        h[:, 0] += a[:, 0] * s["h0"]
    return a, _doubling(a, h), c


def _plain_step(s):
    a, b, _ = _coefficients(s)
    s["state"].copy_(a * s["state"] + b)
    return s["state"].to(s["x"].dtype), s["state"]


def _plain_scan(s):
    _, h, _ = _plain_states(s)
    return h.to(s["x"].dtype), h[:, -1].clone()


def _plain_scan_train(s):
    a, h, c = _plain_states(s)
    y, hf = h.to(s["x"].dtype), h[:, -1].clone()
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"].unsqueeze(1)
    before = torch.cat([first, h[:, :-1]], dim=1)
    # lambda_t = dy_t + a_{t+1} lambda_{t+1}, run backwards in time
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], dim=1)
    lam = _doubling(nxt.flip(1), s["dy"].float().flip(1)).flip(1)
    out, io = {}, s["x"].dtype
    if s["h0"] is not None:
        out["dh0"] = a[:, 0] * lam[:, 0]
    da = lam * before
    if s["reset"] is not None:
        da = torch.where(s["reset"].bool().unsqueeze(-1), 0.0, da)
    x = c["x"]
    if s["mode"] == "decay":
        out["dx"], out["dgate"] = lam.to(io), da.to(io)
        return y, hf, out
    if s["mode"] == "sigmoid":
        dg = (lam * x - da) * (c["s"] * torch.sigmoid(-s["gate"].float() if s["gb"] is None
                                                      else -(s["gate"].float() + s["gb"])))
        out["dx"] = (lam * c["s"]).to(io)
    else:
        ix = x if c["i"] is None else c["i"] * x
        # dL/d(log a): through the state, and through beta = sqrt(1 - a^2)
        dla = c["a"] * da - lam * ix * c["a"] * c["a"] / c["beta"]
        out["dA"] = (dla * c["r"]).sum((0, 1))
        dg = dla * s["A"] * c["r"] * (1 - c["r"])
        lb = lam * c["beta"]
        out["dx"] = (lb if c["i"] is None else lb * c["i"]).to(io)
        if c["i"] is not None:
            di = lb * x * c["i"] * (1 - c["i"])
            out["din_gate"] = di.to(io)
            if s["ib"] is not None:
                out["din_bias"] = di.sum((0, 1))
    out["dgate"] = dg.to(io)
    if s["gb"] is not None:
        out["dgate_bias"] = dg.sum((0, 1))
    return y, hf, out


def _rms(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _norm_grad(dy_w, v, k):
    """Gradient of v k(v) with k = rsqrt(mean v^2 + eps), for the upstream gradient dy_w."""
    return k * dy_w - v * (k ** 3) * (dy_w * v).mean(-1, keepdim=True)


def _plain_boundary(s):
    x = s["x"].float()
    k = None if s["post_w"] is None else _rms(x)
    u = x if k is None else x * k * s["post_w"]
    r = s["residual"].float() + (u if s["scale"] is None else s["scale"] * u)
    return x, k, u, r, _rms(r)


def _plain_norm(s):
    _, _, _, r, q = _plain_boundary(s)
    return (r * q * s["w"]).to(s["x"].dtype), r.to(s["residual"].dtype)


def _plain_norm_train(s):
    x, k, u, r, q = _plain_boundary(s)
    y, stream = (r * q * s["w"]).to(s["x"].dtype), r.to(s["residual"].dtype)
    dy = s["dy"].float()
    dr = s["dres"].float() + _norm_grad(dy * s["w"], r, q)
    out = {"dw": (dy * r * q).sum(0), "dresidual": dr.to(s["residual"].dtype)}
    du = dr
    if s["scale"] is not None:
        out["dscale"] = (dr * u).sum(0)
        du = dr * s["scale"]
    if k is not None:
        out["dpost_w"] = (du * x * k).sum(0)
        du = _norm_grad(du * s["post_w"], x, k)
    out["dx"] = du.to(s["x"].dtype)
    return y, stream, out


def _grouped(t, groups):
    return t.float().unflatten(-1, (groups, -1))


def _plain_gnorm(s):
    x, z, w = (_grouped(s[k], s["groups"]) for k in ("x", "z", "w"))
    gate = z * torch.sigmoid(z)
    v = x * gate if s["gate_first"] else x
    y = v * _rms(v) * w
    return (y if s["gate_first"] else y * gate).flatten(-2).to(s["x"].dtype)


def _plain_gnorm_train(s):
    y = _plain_gnorm(s)
    x, z, w, dy = (_grouped(s[k], s["groups"]) for k in ("x", "z", "w", "dy"))
    sg = torch.sigmoid(z)
    gate = z * sg
    slope = sg * (1 + z * (1 - sg))
    v = x * gate if s["gate_first"] else x
    k = _rms(v)
    inner = dy if s["gate_first"] else dy * gate
    dw = (inner * v * k).sum(0).flatten()
    dv = _norm_grad(inner * w, v, k)
    if s["gate_first"]:
        dx, dz = dv * gate, dv * x * slope
    else:
        dx, dz = dv, dy * v * k * w * slope
    io = s["x"].dtype
    return y, {"dx": dx.flatten(-2).to(io), "dz": dz.flatten(-2).to(io), "dw": dw}


# ------------------------------------------------------------------------------------- work
def work(case):
    e = {"bf16": 2, "f32": 4}
    io = e[case["dtype"]]
    if case["op"].startswith("scan"):
        n, bd, D = case["B"] * case["L"] * case["D"], case["B"] * case["D"], case["D"]
        ins = 3 if case["in_gate"] else 2
        vec = 4 * D * ((case["mode"] == "rate") + case["bias"] * (1 + case["in_gate"]))
        masks = case["B"] * case["L"] if case["doc"] else 0
        per = {"decay": 2, "sigmoid": 12, "rate": 30}[case["mode"]]
        if case["op"] == "scan_step":
            return {"bytes": n * io * (ins + 1) + 8 * bd + vec, "flops": n * per}
        fwd = n * io * (ins + 1) + 4 * bd * (1 + case["h0"]) + vec + masks
        if case["op"] == "scan_fwd":
            return {"bytes": fwd, "flops": n * per}
        # the pass returns y too; its backward reads dy and writes a gradient for each input
        return {"bytes": fwd + n * io * (1 + ins) + vec + 4 * bd * case["h0"], "flops": n * 4 * per}
    n, D = case["rows"] * case["D"], case["D"]
    train = case["op"].endswith("train")
    if case["op"].startswith("gnorm"):
        return {"bytes": n * io * (3 + 3 * train) + 4 * D * (1 + train), "flops": n * (10 + 25 * train)}
    res = e[case["res"]]
    vec = 4 * D * (1 + case["post"] + case["scale"])
    return {"bytes": n * (2 * io + 2 * res) + vec + train * (n * (2 * io + 2 * res) + vec),
            "flops": n * (6 + 20 * train)}


# ------------------------------------------------------------- the definitions in 64 bits
def _recur64(a, b, start):
    """States of h <- a h + b along dim 1 in fp64: blocks of steps side by side, one step at a
    time within each, then one block after the other."""
    B, L, D = b.shape
    T = max(1, int(math.sqrt(L)))
    n = -(-L // T)
    pad = n * T - L
    if pad:
        a = torch.cat([a, torch.ones(B, pad, D, dtype=a.dtype, device=a.device)], 1)
        b = torch.cat([b, torch.zeros(B, pad, D, dtype=b.dtype, device=b.device)], 1)
    a, h = a.reshape(B, n, T, D), b.reshape(B, n, T, D).clone()
    reach = a.clone()
    for t in range(1, T):
        h[:, :, t].addcmul_(a[:, :, t], h[:, :, t - 1])
        reach[:, :, t].mul_(reach[:, :, t - 1])
    enter = start
    for k in range(n):
        h[:, k].addcmul_(reach[:, k], enter.unsqueeze(1))
        enter = h[:, k, -1]
    return h.reshape(B, n * T, D)[:, :L]


def _exact_scan(s):
    wide = {k: s[k].double() for k in ("x", "gate", "ig", "A", "gb", "ib") if s[k] is not None}
    train = s["op"] == "scan_train"
    step = s["op"] == "scan_step"
    if step:
        for k in ("x", "gate", "ig"):
            if k in wide:
                wide[k] = wide[k].unsqueeze(1)
    if train:
        for v in wide.values():
            v.requires_grad_(True)
    logits = wide["gate"] + wide["gb"] if "gb" in wide else wide["gate"]
    if s["mode"] == "decay":
        a, b = logits, wide["x"]
    elif s["mode"] == "sigmoid":
        a, b = 1 / (1 + torch.exp(logits)), wide["x"] / (1 + torch.exp(-logits))
    else:
        lg = wide["A"] / (1 + torch.exp(-logits))
        a, b = torch.exp(lg), torch.sqrt(-torch.expm1(2 * lg)) * wide["x"]
        if "ig" in wide:
            b = b / (1 + torch.exp(-(wide["ig"] + wide["ib"] if "ib" in wide else wide["ig"])))
    keep = torch.ones((), dtype=torch.float64, device=a.device)
    if s["reset"] is not None:
        keep = 1.0 - s["reset"].double().unsqueeze(-1)
    start = torch.zeros_like(b[:, 0]).detach()
    if step:
        start = s["state"].double()
    elif s["h0"] is not None:
        start = s["h0"].double()
    with torch.no_grad():
        used = a * keep
        h = _recur64(used, b, start)
    if step:
        return h[:, 0], h[:, 0]
    if not train:
        return h, h[:, -1]
    with torch.no_grad():
        ahead = torch.cat([torch.zeros_like(used[:, :1]), used.flip(1)[:, :-1]], 1)
        lam = _recur64(ahead, s["dy"].double().flip(1), torch.zeros_like(start)).flip(1)
        da = torch.cat([start.unsqueeze(1), h[:, :-1]], 1).mul_(lam).mul_(keep)
        dh0 = used[:, 0] * lam[:, 0]
    names = {"x": "dx", "gate": "dgate", "ig": "din_gate", "A": "dA", "gb": "dgate_bias", "ib": "din_bias"}
    grads = torch.autograd.grad([a, b], list(wide.values()), [da, lam])
    out = {names[k]: v for k, v in zip(wide, grads)}
    if s["h0"] is not None:
        out["dh0"] = dh0
    return h, h[:, -1], out


def _exact_norms(s):
    v = {k: s[k].double() for k in ("x", "w", "z", "residual", "scale", "post_w") if s.get(k) is not None}
    train = s["op"].endswith("train")
    if train:
        for t in v.values():
            t.requires_grad_(True)

    def normed(t):
        return t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) / t.shape[-1] + EPS)

    if s["op"].startswith("gnorm"):
        cut = (s["rows"], s["groups"], s["D"] // s["groups"])
        gate = v["z"] / (1 + torch.exp(-v["z"]))
        if s["gate_first"]:
            y = normed((v["x"] * gate).reshape(cut)).reshape(s["rows"], s["D"]) * v["w"]
        else:
            y = normed(v["x"].reshape(cut)).reshape(s["rows"], s["D"]) * v["w"] * gate
        outs, ups = [y], [s.get("dy")]
    else:
        u = normed(v["x"]) * v["post_w"] if "post_w" in v else v["x"]
        r = v["residual"] + (u * v["scale"] if "scale" in v else u)
        y = normed(r) * v["w"]
        outs, ups = [y, r], [s.get("dy"), s.get("dres")]
    if not train:
        return outs[0] if len(outs) == 1 else tuple(outs)
    grads = torch.autograd.grad(outs, list(v.values()), [u.double() for u in ups])
    return tuple(o.detach() for o in outs) + ({"d" + k: g for k, g in zip(v, grads)},)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_scan(s) if case["op"].startswith("scan") else _exact_norms(s)
