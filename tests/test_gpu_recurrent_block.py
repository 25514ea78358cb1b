"""The gated recurrence and the fused norms as a model uses them together (needs an MI355X): a
residual block trained and decoded with them, the norm behind the SSD layer, and all of them
under HIP graph capture."""
import threading

import pytest
import torch

import oracle
import selective_state_space_59_amd as ssm
from oracle import recurrent as R
from selective_state_space_59_amd import workloads as W
from tests.gpu_helpers import TOL, assert_close, to64
from tests.recurrent_helpers import check, f64, gnorm_bound, scan_case, scan_case64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
DM, DI = 48, 96


def _weights(seed, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = dict(norm=1 + 0.1 * n(DM), scale=0.5 + 0.1 * n(DM), post=1 + 0.1 * n(DM), mix=1 + 0.1 * n(DI),
             w_x=n(DM, DI) * DM ** -0.5, w_g=n(DM, DI) * DM ** -0.5, w_i=n(DM, DI) * DM ** -0.5,
             w_z=n(DM, DI) * DM ** -0.5, w_o=n(DI, DM) * DI ** -0.5, A=-torch.exp(-4 * torch.rand(DI, generator=g)),
             gb=n(DI), ib=n(DI))
    return {k: v.to(DEV) for k, v in w.items()}


def _block(x, residual, w, reset, h0):
    """residual + scale * RMSNorm(x) -> norm -> projections -> recurrence -> gated norm -> out."""
    y, r = ssm.add_rmsnorm(x, w["norm"], residual, w["scale"], w["post"])
    h, hf = ssm.gated_scan((y @ w["w_x"]).contiguous(), y @ w["w_g"], "rate", A=w["A"], in_gate=y @ w["w_i"],
                           gate_bias=w["gb"], in_bias=w["ib"], reset=reset, h0=h0)
    return ssm.gated_rmsnorm(h, y @ w["w_z"], w["mix"], groups=4) @ w["w_o"], r, hf


def _block64(x, residual, w, reset, h0):
    """The same in elementary fp64 torch operations, one step at a time."""
    rms = lambda v: v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-5)  # noqa: E731
    r = residual + w["scale"] * (rms(x) * w["post"])
    y = rms(r) * w["norm"]
    la = w["A"] * torch.sigmoid(y @ w["w_g"] + w["gb"])
    b = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(y @ w["w_i"] + w["ib"]) * (y @ w["w_x"])
    a, h, hs = torch.exp(la) * (1.0 - reset.to(la.dtype)).unsqueeze(-1), h0, []
    for t in range(x.shape[1]):
        h = a[:, t] * h + b[:, t]
        hs.append(h)
    h = torch.stack(hs, 1)
    v = (h * torch.nn.functional.silu(y @ w["w_z"])).unflatten(-1, (4, -1))
    return (rms(v).flatten(-2) * w["mix"]) @ w["w_o"], r, hs[-1]


def test_two_blocks_train_like_their_definition():
    """Forward and every gradient through two blocks in fp32.  The bound is on the 2-norm: each of
    the twelve operators of the chain adds at most some 100 roundings of 2^-24, and its neighbours
    pass them on with factors of a few, so 12 * 100 * 5 * 2^-24 = 3.6e-4."""
    B, L = 2, 300
    g = torch.Generator().manual_seed(1)
    x, res = torch.randn(B, L, DM, generator=g).to(DEV), torch.randn(B, L, DM, generator=g).to(DEV)
    h0 = torch.randn(B, DI, generator=g).to(DEV)
    reset = (torch.rand(B, L, generator=g) < 0.01).to(torch.uint8).to(DEV)
    dy = torch.randn(B, L, DM, generator=g).to(DEV)
    results = []
    for cast, block in ((torch.Tensor.float, _block), (torch.Tensor.double, _block64)):
        leaf = lambda t: cast(t).detach().clone().requires_grad_()  # noqa: E731
        w1, w2 = ({k: leaf(v) for k, v in _weights(s).items()} for s in (2, 3))
        xi, ri, hi = leaf(x), leaf(res), leaf(h0)
        o1, r1, f1 = block(xi, ri, w1, reset, hi)
        o2, r2, f2 = block(o1, r1, w2, reset, hi)
        torch.autograd.backward([o2, r2, f2], [cast(dy), cast(dy), torch.ones_like(f2)])
        results.append([o2, r2, f1, f2] + [t.grad for t in (xi, ri, hi, *w1.values(), *w2.values())])
    for i, (a, b) in enumerate(zip(*results)):
        off = float((a.detach().double() - b.detach()).norm() / b.detach().norm())
        assert off <= 3.6e-4, (i, off)


def test_decoding_continues_a_prefill():
    """Tokens one at a time through the norms and the step, from a prefill's state, against one
    pass over all of them: the norms give the very same rows, the recurrence its own bound."""
    B, L, P = 3, 40, 33
    w = _weights(5)
    g = torch.Generator().manual_seed(6)
    x, res = torch.randn(B, L, DM, generator=g).to(DEV).to(BF), torch.randn(B, L, DM, generator=g).to(DEV)
    y, r = ssm.add_rmsnorm_fwd(x, w["norm"], res, scale=w["scale"], post_w=w["post"])
    proj = {k: (y.float() @ w["w_" + k]).to(BF) for k in "xgiz"}
    kw = dict(mode="rate", A=w["A"], gate_bias=w["gb"], in_bias=w["ib"])
    h, _ = ssm.gated_scan_fwd(proj["x"], proj["g"], in_gate=proj["i"], **kw)
    out = ssm.gated_rmsnorm_fwd(h, proj["z"], w["mix"], groups=4)
    part = lambda t, lo, hi: t[:, lo:hi].contiguous()  # noqa: E731
    _, state = ssm.gated_scan_fwd(part(proj["x"], 0, P), part(proj["g"], 0, P), in_gate=part(proj["i"], 0, P),
                                  return_final_state=True, **kw)
    k64 = scan_case64(dict(x=proj["x"], gate=proj["g"], in_gate=proj["i"], **kw))
    H, _, E = R.gated_scan(**k64)
    for t in range(P, L):
        yt, rt = ssm.add_rmsnorm_fwd(x[:, t].contiguous(), w["norm"], res[:, t].contiguous(), scale=w["scale"],
                                     post_w=w["post"])
        assert torch.equal(yt, y[:, t]) and torch.equal(rt, r[:, t])
        one = {k: v[:, t].contiguous() for k, v in proj.items()}
        ht = ssm.gated_scan_step(state, one["x"], one["g"], in_gate=one["i"], **kw)
        check(ht, H[:, t], E[:, t], "token %d" % t)
        got = ssm.gated_rmsnorm_fwd(ht, one["z"], w["mix"], groups=4)
        same = torch.equal(ht, h[:, t])  # (bf16: nearly always; a tie may round the other way)
        assert not same or torch.equal(got, out[:, t])


def test_the_norm_behind_the_ssd_layer():
    """A Mamba-2 layer with its gate in the norm: ssd_fwd without z, then the gated norm."""
    B, L, H, P, N = 2, 200, 4, 64, 64
    inp = W.make_ssd_inputs(B, L, H, P, 1, N, seed=7, device=DEV, gate=True)
    y = ssm.ssd_fwd(inp["x"], inp["delta"], inp["A"], inp["Bm"], inp["Cm"], Dskip=inp["Dskip"])
    w = 1 + 0.1 * torch.randn(H * P, generator=torch.Generator().manual_seed(8)).to(DEV)
    flat = lambda t: t.reshape(B, L, H * P)  # noqa: E731
    out = ssm.gated_rmsnorm_fwd(flat(y), flat(inp["z"]), w, groups=2)
    torch.cuda.synchronize()
    ref, _ = oracle.ssd(to64(inp["x"]), to64(inp["delta"]), to64(inp["A"]), to64(inp["Bm"]), to64(inp["Cm"]),
                        Dskip=to64(inp["Dskip"]))
    assert_close(to64(y), ref, TOL[BF], "ssd")
    rows = lambda t: f64(t).reshape(B * L, H * P)  # noqa: E731
    args = rows(flat(y)), rows(flat(inp["z"])), f64(w)
    check(out.reshape(B * L, H * P), R.gated_rmsnorm(*args, 2), gnorm_bound(*args, 2, True)["y"], "norm")


# ------------------------------------------------------------------------- graph capture
def _capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fn()
    return g, out


def _flat(v):
    if isinstance(v, torch.Tensor):
        return [v]
    if isinstance(v, dict):
        return [t for k in sorted(v) for t in _flat(v[k])]
    return [t for u in v if u is not None for t in _flat(u)]


def _calls():
    k = scan_case("rate", 2, 1300, 136, BF, seed=9, doc=200)
    dy = torch.randn(k["x"].shape, generator=torch.Generator().manual_seed(10)).to(DEV).to(BF)
    ck = torch.empty(ssm.gated_checkpoint_shape(2, 1300, 136), device=DEV)
    x, z = k["x"], k["gate"]
    w = torch.ones(136, device=DEV)
    return dict(
        forward=lambda: ssm.gated_scan_fwd(return_final_state=True, checkpoints=ck, **k),
        backward=lambda: ssm.gated_scan_bwd(dy=dy, **k),
        add_norm=lambda: (ssm.add_rmsnorm_fwd(x, w, z), ssm.add_rmsnorm_bwd(x, w, z, dy, dy)),
        gated_norm=lambda: (ssm.gated_rmsnorm_fwd(x, z, w, groups=2), ssm.gated_rmsnorm_bwd(x, z, w, dy, groups=2)))


@pytest.mark.parametrize("name", ["forward", "backward", "add_norm", "gated_norm"])
def test_replays_match_eager(name):
    call = _calls()[name]
    want = [t.clone() for t in _flat(call())]
    g, out = _capture(call)
    out = _flat(out)
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        call()  # eager work of the same kind between replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_step_replays_advance_the_state():
    k = scan_case("rate", 4, 1, 520, BF, seed=11)
    state = k.pop("h0")
    one = {m: v[:, 0].contiguous() if m in ("x", "gate", "in_gate") else v for m, v in k.items()}
    start, y = state.clone(), torch.empty_like(one["x"])
    g, _ = _capture(lambda: ssm.gated_scan_step(state, y=y, **one))
    state.copy_(start)
    ref = start.clone()
    for _ in range(4):
        want = ssm.gated_scan_step(ref, **one)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(state, ref) and torch.equal(y, want)


def test_two_graphs_replay_at_once():
    """Each capture holds a workspace of its own: two graphs replayed on two streams at the same
    time, and an eager call beside them, do not meet."""
    calls = _calls()
    want = {n: [t.clone() for t in _flat(calls[n]())] for n in ("forward", "backward")}
    graphs = {n: _capture(calls[n]) for n in want}
    streams = {n: torch.cuda.Stream() for n in want}
    for _ in range(4):
        torch.cuda.synchronize()
        for n, (g, _) in graphs.items():
            with torch.cuda.stream(streams[n]):
                g.replay()
        calls["backward"]()
        torch.cuda.synchronize()
        for n, (_, out) in graphs.items():
            for a, b in zip(_flat(out), want[n]):
                assert torch.equal(a, b), n


def test_a_captured_training_step():
    """Forward and backward of the differentiable op recorded in one graph, on leaves that no
    other autograd graph holds."""
    k = scan_case("rate", 2, 700, 72, BF, seed=12)
    leaves = [k["x"], k["gate"], k["A"]]
    for t in leaves:
        t.requires_grad_()
    dy = torch.randn(k["x"].shape, generator=torch.Generator().manual_seed(13)).to(DEV).to(BF)

    def step():
        y, _ = ssm.gated_scan(**k)
        return torch.autograd.grad(y, leaves, dy)

    want = [t.clone() for t in step()]
    g, out = _capture(step)
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_two_threads_on_one_stream():
    """Calls of two host threads alternate launch by launch on the stream they share; each gets
    the results it gets alone."""
    ks = [scan_case("rate", 1, 3000 + 500 * i, 96, F32, seed=91 + i, doc=400) for i in range(2)]
    gen = torch.Generator().manual_seed(9)
    rows = [torch.randn(4000 + i, 768, generator=gen).to(DEV) for i in range(2)]
    w = torch.randn(768, generator=gen).to(DEV)

    def calls(i):
        y, hf = ssm.gated_scan_fwd(return_final_state=True, **ks[i])
        g = ssm.gated_scan_bwd(dy=y, **ks[i])
        n = ssm.add_rmsnorm_bwd(rows[i], w, None, rows[i])
        return [y, hf, *g.values(), *n.values()]

    want = [calls(0), calls(1)]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(i):
        try:
            for _ in range(20):
                got[i].append(calls(i))
        except Exception as e:  # reported below, by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))
