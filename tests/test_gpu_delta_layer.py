"""The gated delta rule and the 8-bit projections as a model uses them together (needs an MI355X): a layer
trained like its definition, served in 8 bits, decoded behind a prefill, and all of it under graph capture,
on several streams and from several threads."""
import threading

import numpy as np
import pytest
import torch

import selective_state_space_59_amd as ssm
from oracle import delta as R
from tests.delta_helpers import bound, case64, close, delta_case
from tests.recurrent_helpers import f64
from tests.test_gpu_recurrent_block import _capture, _flat

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
DM, HK, H, K, V = 64, 2, 4, 16, 24


def _weights(seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    out = 2 * HK * K + 2 * H * V
    w = dict(norm=1 + 0.1 * n(DM), mix=1 + 0.1 * n(H * V), w_in=n(DM, out) * DM ** -0.5, w_b=n(DM, H) * DM ** -0.5,
             w_a=n(DM, H) * DM ** -0.5, A=-torch.exp(-3 * torch.rand(H, generator=g)), w_out=n(H * V, DM) * (H * V) ** -0.5)
    return {k: v.to(DEV) for k, v in w.items()}


def _cut(y, w):
    q, k, v, z = (y @ w["w_in"]).split([HK * K, HK * K, H * V, H * V], -1)
    g = w["A"] * torch.nn.functional.softplus(y @ w["w_a"])
    return q.unflatten(-1, (HK, K)), k.unflatten(-1, (HK, K)), v.unflatten(-1, (H, V)), z, g, torch.sigmoid(y @ w["w_b"])


def _layer(x, residual, w, reset, h0):
    y, r = ssm.add_rmsnorm(x, w["norm"], residual)
    q, k, v, z, g, beta = _cut(y, w)
    o, hf = ssm.gated_delta(q, k, v, g, beta, l2norm=True, reset=reset, h0=h0)
    return ssm.gated_rmsnorm(o.flatten(2), z.contiguous(), w["mix"], groups=H) @ w["w_out"], r, hf


def _layer64(x, residual, w, reset, h0):
    rms = lambda t: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-5)  # noqa: E731
    r = residual + x
    y = rms(r) * w["norm"]
    q, k, v, z, g, beta = _cut(y, w)
    unit = lambda t: (t * torch.rsqrt((t * t).sum(-1, keepdim=True) + 1e-6)).repeat_interleave(H // HK, 2)  # noqa: E731
    q, k, S, os = unit(q), unit(k), h0, []
    keep = 1.0 - reset.to(q.dtype)
    for t in range(x.shape[1]):
        S = (torch.exp(g[:, t]) * keep[:, t, None])[..., None, None] * S
        e = v[:, t] - (S * k[:, t, :, :, None]).sum(2)
        S = S + k[:, t, :, :, None] * (beta[:, t, :, None] * e)[:, :, None]
        os.append((S * q[:, t, :, :, None]).sum(2) * K ** -0.5)
    o = torch.stack(os, 1).flatten(2)
    u = (o * torch.nn.functional.silu(z)).unflatten(-1, (H, V))
    return (rms(u).flatten(2) * w["mix"]) @ w["w_out"], r, S


def test_two_layers_train_like_their_definition():
    """Forward and every gradient through two layers in fp32, against autograd through the definition in fp64,
    in the 2-norm: fourteen operators of some 100 roundings of 2^-24 each, passed on with factors of a few:
    14 * 100 * 5 * 2^-24 = 4.2e-4."""
    B, L = 2, 150
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    x, res, h0, dy = n(B, L, DM), n(B, L, DM), 0.3 * n(B, H, K, V), n(B, L, DM)
    reset = (torch.rand(B, L, generator=g) < 0.02).to(torch.uint8).to(DEV)
    results = []
    for cast, layer in ((torch.Tensor.float, _layer), (torch.Tensor.double, _layer64)):
        leaf = lambda t: cast(t).detach().clone().requires_grad_()  # noqa: E731
        w1, w2 = ({k: leaf(v) for k, v in _weights(s).items()} for s in (2, 3))
        xi, ri, hi = leaf(x), leaf(res), leaf(h0)
        o1, r1, f1 = layer(xi, ri, w1, reset, hi)
        o2, r2, f2 = layer(o1, r1, w2, reset, hi)
        torch.autograd.backward([o2, r2, f2], [cast(dy), cast(dy), torch.ones_like(f2)])
        results.append([o2, r2, f1, f2] + [t.grad for t in (xi, ri, hi, *w1.values(), *w2.values())])
    for i, (a, b) in enumerate(zip(*results)):
        off = float((a.detach().double() - b.detach()).norm() / b.detach().norm())
        assert off <= 4.2e-4, (i, off)


def test_gradients_of_a_few_inputs_only():
    k = delta_case(2, 100, 1, 2, 24, 16, BF, seed=2)
    do = torch.randn(k["v"].shape, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    want = ssm.gated_delta_bwd(do=do, **k)
    opts = dict(l2norm=k.pop("l2norm"))
    for name in ("v", "g", "h0"):
        leaves = {n: t.clone().requires_grad_(n == name) for n, t in k.items()}
        o, _ = ssm.gated_delta(**leaves, **opts)
        o.backward(do)
        assert torch.equal(leaves[name].grad, want["d" + name])
        assert all(t.grad is None for n, t in leaves.items() if n != name)


def test_a_changed_input_is_noticed():
    k = delta_case(1, 70, 1, 1, 16, 16, F32, seed=3)
    opts = dict(l2norm=k.pop("l2norm"))
    k["q"].requires_grad_()
    o, _ = ssm.gated_delta(**k, **opts)
    ssm.gated_delta_step(k["h0"], *(k[n].detach()[:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()


def test_decoding_continues_a_prefill():
    """Tokens one at a time from a prefill's state against the definition over all of them, in bf16."""
    B, L, P = 3, 100, 90
    k = delta_case(B, L, 2, 4, 40, 24, BF, seed=4, h0=False)
    ro, rs = R.gated_delta(**case64(k))
    part = lambda a, b: {n: k[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")}  # noqa: E731
    _, state = ssm.gated_delta_fwd(return_final_state=True, l2norm=True, **part(0, P))
    for t in range(P, L):
        o = ssm.gated_delta_step(state, l2norm=True, **{n: x[:, 0] for n, x in part(t, t + 1).items()})
        close(o, ro[:, t], bound(k), "token %d" % t)
    close(state, rs, bound(k), "state")


def test_served_in_8_bits():
    """norm -> e4m3 -> product -> delta rule -> gated norm -> e4m3 -> product.  Each stage against its own
    definition on what the stage before gave it, the layer's shape put together from them."""
    B, L = 2, 130
    g = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    w = _weights(6)
    w_in, s_in = ssm.quantize_fp8(w["w_in"].t().contiguous(), 128)
    w_out, s_out = ssm.quantize_fp8(w["w_out"].t().contiguous(), 128)
    x, res = n(B, L, DM).to(BF), n(B, L, DM)
    yq, ys, r = ssm.add_rmsnorm_fp8(x, w["norm"], res)
    proj = ssm.matmul_fp8(yq, ys, w_in, s_in)
    ref = R.matmul_blocks(f64(yq.float()).reshape(-1, DM), f64(ys).reshape(-1, 1), f64(w_in.float()), f64(s_in))
    # (the 8-bit instruction: what lies 2^14 below the largest of eight products is dropped)
    off = np.abs(f64(proj).reshape(ref[0].shape) - ref[0])
    assert (off <= 2.0 ** -8 * np.abs(ref[0]) + 8 * 2.0 ** -14 * ref[1]).all()
    q, k, v, z = proj.split([HK * K, HK * K, H * V, H * V], -1)
    y = yq.float() * ys
    gate, beta = -torch.nn.functional.softplus(y @ w["w_a"]), torch.sigmoid(y @ w["w_b"]).to(BF)
    args = q.unflatten(-1, (HK, K)), k.unflatten(-1, (HK, K)), v.unflatten(-1, (H, V)), gate, beta
    o, hf = ssm.gated_delta_fwd(*args, l2norm=True, return_final_state=True)
    ro, rs = R.gated_delta(*(f64(t) for t in args), l2norm=True)
    close(o, ro, R.relative_bound(L, K, V), "o")
    close(hf, rs, R.relative_bound(L, K, V), "h_final")
    mixed = ssm.gated_rmsnorm_fwd(o.flatten(2), z.contiguous(), w["mix"], groups=H)
    mq, ms = ssm.quantize_fp8(mixed)
    out = ssm.matmul_fp8(mq, ms, w_out, s_out, out_dtype=F32)
    ref = R.matmul_blocks(f64(mq.float()).reshape(-1, H * V), f64(ms).reshape(-1, 1), f64(w_out.float()), f64(s_out))
    assert out.shape == (B, L, DM)
    assert (np.abs(f64(out).reshape(ref[0].shape) - ref[0]) <= 2 * (H * V + 4) * 2.0 ** -24 * ref[1]).all()
    # one more token, all of it on the state in place
    t = x[:, -1].contiguous(), res[:, -1].contiguous()
    yq1, ys1, _ = ssm.add_rmsnorm_fp8(t[0], w["norm"], t[1])
    assert torch.equal(yq1.view(torch.uint8), yq[:, -1].contiguous().view(torch.uint8)) and torch.equal(ys1, ys[:, -1])
    p1 = ssm.matmul_fp8(yq1, ys1, w_in, s_in)
    q1, k1, v1, z1 = p1.split([HK * K, HK * K, H * V, H * V], -1)
    o1 = ssm.gated_delta_step(hf, q1.unflatten(-1, (HK, K)), k1.unflatten(-1, (HK, K)), v1.unflatten(-1, (H, V)),
                              gate[:, -1].contiguous(), beta[:, -1].contiguous(), l2norm=True)
    m1 = ssm.gated_rmsnorm_fwd(o1.flatten(1), z1.contiguous(), w["mix"], groups=H)
    out1 = ssm.matmul_fp8(*ssm.quantize_fp8(m1), w_out, s_out)
    assert out1.shape == (B, DM) and torch.isfinite(out1.float()).all()


# ------------------------------------------------------------------------- graph capture
def _calls():
    k = delta_case(2, 300, 2, 4, 72, 40, BF, seed=9, doc=100)
    do = torch.randn(k["v"].shape, generator=torch.Generator().manual_seed(10)).to(BF).to(DEV)
    ck = torch.empty(ssm.gated_delta_checkpoint_shape(2, 300, 4, 72, 40), device=DEV)
    x = torch.randn(300, 400, generator=torch.Generator().manual_seed(11)).to(DEV)
    w, ones = ssm.quantize_fp8(x[:130].contiguous(), 128), torch.ones(400, device=DEV)
    long, wide = delta_case(1, 2100, 1, 2, 40, 24, BF, seed=12, doc=900), delta_case(1, 3100, 1, 5, 16, 344, BF, seed=13)
    dlong = torch.randn(long["v"].shape, generator=torch.Generator().manual_seed(14)).to(BF).to(DEV)
    return dict(segments=lambda: ssm.gated_delta_fwd(return_final_state=True, **long),
                wide_segments=lambda: ssm.gated_delta_fwd(return_final_state=True, **wide),
                segments_backward=lambda: ssm.gated_delta_bwd(do=dlong, **long),
                forward=lambda: ssm.gated_delta_fwd(return_final_state=True, checkpoints=ck, **k),
                backward=lambda: ssm.gated_delta_bwd(do=do, **k),
                product=lambda: ssm.matmul_fp8(*ssm.quantize_fp8(x), *w),
                norm=lambda: ssm.add_rmsnorm_fp8(x, ones, x))


def _equal(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("name", ["forward", "backward", "segments", "wide_segments", "segments_backward", "product", "norm"])
def test_replays_match_eager(name):
    call = _calls()[name]
    want = [t.clone() for t in _flat(call())]
    g, out = _capture(call)
    out = _flat(out)
    for _ in range(3):
        for t in out:
            t.view(torch.uint8).fill_(255)
        call()  # eager work of the same kind between replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(_equal(a, b) for a, b in zip(out, want))


def test_step_replays_advance_the_state():
    k = delta_case(4, 1, 2, 4, 64, 72, BF, seed=11)
    one = {n: k[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")}
    state, o = k["h0"].clone(), torch.empty_like(one["v"])
    g, _ = _capture(lambda: ssm.gated_delta_step(state, o=o, **one))
    state.copy_(k["h0"])
    ref = k["h0"].clone()
    for _ in range(4):
        want = ssm.gated_delta_step(ref, **one)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(state, ref) and torch.equal(o, want)


def test_two_graphs_replay_at_once():
    """Each capture holds a workspace of its own."""
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
            assert all(_equal(a, b) for a, b in zip(_flat(out), want[n])), n


def test_a_captured_training_step():
    """Forward and backward of the differentiable op in one graph, on leaves no other autograd graph holds."""
    k = delta_case(2, 200, 1, 2, 24, 32, BF, seed=12)
    leaves = [k[n].requires_grad_() for n in ("q", "k", "v", "g", "beta", "h0")]
    do = torch.randn(k["v"].shape, generator=torch.Generator().manual_seed(13)).to(BF).to(DEV)

    def step():
        o, hf = ssm.gated_delta(**k)
        return torch.autograd.grad([o, hf], leaves, [do, torch.ones_like(hf)])

    want = [t.clone() for t in step()]
    g, out = _capture(step)
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_threads_and_other_streams():
    """Calls of two host threads on one stream, and on streams of their own, give what they give alone."""
    ks = [delta_case(1, 600 + 70 * i, 1, 2, 40, 24, F32, seed=91 + i) for i in range(2)]

    def calls(i):
        o, hf = ssm.gated_delta_fwd(return_final_state=True, **ks[i])
        return [o, hf, *ssm.gated_delta_bwd(do=o, **ks[i]).values()]

    want = [calls(0), calls(1)]
    torch.cuda.synchronize()
    for own_stream in (False, True):
        got, failed = [[], []], []

        def work(i):
            try:
                side = torch.cuda.Stream() if own_stream else torch.cuda.current_stream()
                with torch.cuda.stream(side):
                    for _ in range(10):
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


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("K_", [24, 96])
def test_many_heads(K_, dtype):
    """Enough heads that a workgroup takes 32 channels of one, the last of them half a workgroup's."""
    k = delta_case(17, 70, 8, 16, K_, 40, dtype, seed=14, doc=50)
    o, hf = ssm.gated_delta_fwd(return_final_state=True, **k)
    ro, rs = R.gated_delta(**case64(k))
    close(o, ro, bound(k), "o")
    close(hf, rs, bound(k), "h_final")
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    d = ssm.gated_delta_bwd(do=do, **k)
    for n, v in R.gated_delta_bwd(do=f64(do), **case64(k)).items():
        close(d[n], v, bound(k), n)
