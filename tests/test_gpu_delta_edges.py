"""The gated delta rule and the e4m3 calls where they can go wrong (needs an MI355X): frames around outputs,
parts of wider tensors, dropped states, keys that repeat, long memories, long sequences, offsets past 32
bits, what they refuse."""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_59_amd as ssm
from oracle import delta as R
from selective_state_space_59_amd import ssm as capi
from tests.delta_helpers import bound, case64, close, delta_case
from tests.recurrent_helpers import f64
from tests.test_gpu_recurrent_frames import Frames

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
IDS = dict(argvalues=[F32, BF], ids=["f32", "bf16"])


def _call(call, args, frames, size=None, **tensors):
    for k, t in tensors.items():
        if t is not None:
            setattr(args, k, t.data_ptr())
    L = ssm.lib()
    if size is not None:
        need = getattr(L, size)(ctypes.byref(args))
        assert need != ctypes.c_size_t(-1).value
        args.workspace = frames.take((max(need, 1),), torch.uint8, odd=False).data_ptr()
        args.workspace_bytes = need
    status = getattr(L, call)(ctypes.byref(args), torch.cuda.current_stream().cuda_stream)
    assert status == capi.SSM_OK, L.ssm_last_error_message().decode()
    frames.check(call)


def _take(frames, tensors, aligned=()):
    return {k: frames.take(tuple(t.shape), t.dtype, odd=k not in aligned) for k, t in tensors.items()}


def _same(got, want, what):
    for n, t in want.items():
        same = got[n].view(torch.uint8) == t.view(torch.uint8)
        assert same.all(), (what, n)


@pytest.mark.parametrize("dtype", **IDS)
def test_stores_of_the_chain_stay_inside(dtype):
    """Every output and a workspace of exactly the size asked for lie in marked memory."""
    for B, L, Hk, H, K, V in [(1, 1, 1, 1, 8, 8), (2, 65, 1, 2, 72, 24), (1, 64, 2, 2, 64, 72), (1, 130, 2, 6, 128, 136),
                               (32, 66, 2, 8, 72, 24), (16, 65, 8, 8, 128, 40),
                               (1, 2050, 1, 2, 72, 40)]:
        what = "%dx%d %d/%d heads %dx%d" % (B, L, Hk, H, K, V)
        print(what, flush=True)
        k = delta_case(B, L, Hk, H, K, V, dtype, seed=L, doc=20)
        sizes = dict(batch=B, seqlen=L, kheads=Hk, heads=H, kdim=K, vdim=V, io_dtype=capi._io_code(dtype), l2norm=1,
                     scale=K ** -0.5)
        ins = {m: v for m, v in k.items() if isinstance(v, torch.Tensor)}
        ck = torch.empty(ssm.gated_delta_checkpoint_shape(B, L, H, K, V), device=DEV)
        o, hf = ssm.gated_delta_fwd(return_final_state=True, checkpoints=ck, **k)
        want = dict(o=o, h_final=hf, checkpoints=ck)
        fr = Frames()
        out = _take(fr, want, aligned=("checkpoints",))
        _call("ssm_gated_delta_fwd", capi.GatedDeltaArgs(**sizes), fr, "ssm_gated_delta_workspace_size", **ins, **out)
        _same(out, want, what)
        do = torch.randn(o.shape, device=DEV).to(dtype)
        want = ssm.gated_delta_bwd(do=do, dh_final=hf, **k)
        for given in (ck, None):
            fr = Frames()
            out = _take(fr, want)
            _call("ssm_gated_delta_bwd", capi.GatedDeltaBwdArgs(**sizes), fr, "ssm_gated_delta_bwd_workspace_size", **ins,
                  **out, dout=do, dh_final=hf, checkpoints=given)
            _same(out, want, what)
        one = {m: ins[m][:, 0].contiguous() for m in ("q", "k", "v", "g", "beta", "reset")}
        state = k["h0"].clone()
        want = dict(o=ssm.gated_delta_step(state, l2norm=True, **one), state=state)
        fr = Frames()
        out = _take(fr, want, aligned=("state",))
        out["state"].copy_(k["h0"])
        del sizes["seqlen"]
        _call("ssm_gated_delta_step", capi.GatedDeltaStepArgs(**sizes), fr, **one, **out)
        _same(out, want, what)


@pytest.mark.parametrize("dtype", **IDS)
def test_stores_of_the_8_bit_calls_stay_inside(dtype):
    io = capi._io_code(dtype)
    for M, D in [(1, 16), (5, 144), (129, 272), (3, 2576), (2, 9008)]:
        x = torch.randn(M, D, device=DEV).to(dtype)
        for rows in (1, 128):
            want = dict(zip(("q", "scales"), ssm.quantize_fp8(x, rows)))
            fr = Frames()
            out = _take(fr, want, aligned=("q",))
            _call("ssm_quantize_fp8", capi.QuantizeFp8Args(rows=M, dim=D, block_rows=rows, io_dtype=io), fr, x=x, **out)
            _same(out, want, "%dx%d" % (M, D))
        w = torch.rand(D, device=DEV)
        want = dict(zip(("q", "scales", "res_out"), ssm.add_rmsnorm_fp8(x, w, x, scale=w, post_w=w)))
        fr = Frames()
        out = _take(fr, want, aligned=("q",))
        a = capi.AddNormFp8Args(norm=capi.AddNormArgs(rows=M, dim=D, io_dtype=io, res_dtype=io, eps=1e-5))
        for n, t in dict(x=x, residual=x, scale=w, post_w=w, w=w, res_out=out.pop("res_out")).items():
            setattr(a.norm, n, t.data_ptr())
        _call("ssm_add_rmsnorm_fp8", a, fr, **out)
        _same(out, {n: want[n] for n in out}, "norm %dx%d" % (M, D))
    for M, N, K in [(1, 1, 16), (15, 17, 144), (33, 31, 128), (65, 63, 272), (1200, 1301, 144), (4100, 4097, 32)]:
        xq, xs = ssm.quantize_fp8(torch.randn(M, K, device=DEV))
        wq, ws = ssm.quantize_fp8(torch.randn(N, K, device=DEV), 128)
        want = dict(y=ssm.matmul_fp8(xq, xs, wq, ws, out_dtype=dtype))
        fr = Frames()
        out = _take(fr, want)
        _call("ssm_matmul_fp8", capi.MatmulFp8Args(m=M, n=N, k=K, out_dtype=io), fr, xq=xq, x_scales=xs, wq=wq, w_scales=ws,
              **out)
        _same(out, want, "%dx%dx%d" % (M, N, K))


@pytest.mark.parametrize("dtype", **IDS)
def test_parts_of_wider_tensors(dtype):
    """q, k and v cut out of one projection's rows give the results of dense copies, to the bit: forward,
    backward, the autograd op and the step; a row that is one of several too."""
    B, L, Hk, H, K, V = 2, 100, 2, 4, 40, 24
    g = torch.Generator().manual_seed(3)
    wide = torch.randn(B, L, 2 * Hk * K + H * V + 16, generator=g).to(dtype).to(DEV)
    q, k, v, _ = wide.split([Hk * K, Hk * K, H * V, 16], -1)
    views = q.unflatten(-1, (Hk, K)), k.unflatten(-1, (Hk, K)), v.unflatten(-1, (H, V))
    dense = [t.contiguous() for t in views]
    gate = -torch.rand(B, L, H, generator=g).to(DEV)
    beta = torch.rand(B, L, H, generator=g).to(dtype).to(DEV)
    do = torch.randn(B, L, H, V, generator=g).to(dtype).to(DEV)
    for rows in (slice(0, 2), slice(1, 2)):
        a = [t[rows] for t in views], [t[rows].contiguous() for t in dense]
        outs = [ssm.gated_delta_fwd(*t, gate[rows].contiguous(), beta[rows].contiguous(), l2norm=True,
                                    return_final_state=True) for t in a]
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        grads = [ssm.gated_delta_bwd(*t, gate[rows].contiguous(), beta[rows].contiguous(), do[rows].contiguous(),
                                     l2norm=True) for t in a]
        for n in grads[0]:
            assert torch.equal(grads[0][n], grads[1][n]), n
    leaf = wide.clone().requires_grad_()
    parts = leaf.split([Hk * K, Hk * K, H * V, 16], -1)
    o, _ = ssm.gated_delta(parts[0].unflatten(-1, (Hk, K)), parts[1].unflatten(-1, (Hk, K)),
                           parts[2].unflatten(-1, (H, V)), gate, beta, l2norm=True)
    o.backward(do)
    d = ssm.gated_delta_bwd(*dense, gate, beta, do, l2norm=True)
    want = torch.cat([d["dq"].flatten(2), d["dk"].flatten(2), d["dv"].flatten(2), torch.zeros_like(wide[..., :16])], -1)
    assert torch.equal(leaf.grad, want)
    states = [torch.zeros(B, H, K, V, device=DEV) for _ in range(2)]
    os = [ssm.gated_delta_step(s, *(x[:, 5] for x in t), gate[:, 5].contiguous(), beta[:, 5].contiguous(), l2norm=True)
          for s, t in zip(states, (views, dense))]
    assert torch.equal(os[0], os[1]) and torch.equal(*states)


@pytest.mark.parametrize("dtype", **IDS)
def test_a_reset_drops_whatever_the_state_held(dtype):
    """An entering state of infinities and NaNs is not seen behind a reset: not by the outputs, not by the
    final state; the same for decays that round to 0."""
    k = delta_case(2, 150, 1, 2, 40, 24, dtype, seed=4)
    k["reset"] = torch.zeros(2, 150, dtype=torch.bool, device=DEV)
    k["reset"][0, 0] = True
    k["reset"][1, 70] = True
    k["g"][0, 100, 1] = float("-inf")
    k["g"][1, 90] = -200.0
    ref = R.gated_delta(**case64(k))
    bad = dict(k, h0=k["h0"].clone())
    bad["h0"][0] = float("nan")
    bad["h0"][1] = float("inf")
    o, hf = ssm.gated_delta_fwd(return_final_state=True, **bad)
    close(o[0], ref[0][0], bound(k), "o, reset at once")
    close(o[1, 70:], ref[0][1, 70:], bound(k), "o behind the reset")
    close(hf, ref[1], bound(k), "h_final")
    state = bad["h0"].clone()
    one = {n: k[n][:, 0].contiguous() for n in ("q", "k", "v", "beta")}
    got = ssm.gated_delta_step(state, g=torch.tensor([[float("-inf"), -150.0], [0.0, 0.0]], device=DEV),
                               reset=torch.tensor([0, 1], dtype=torch.uint8, device=DEV), l2norm=True, **one)
    assert torch.isfinite(state).all() and torch.isfinite(got.float()).all()
    # and the gradient of g is 0 where it makes a reset
    do = torch.randn(k["v"].shape, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    d = ssm.gated_delta_bwd(do=do, **k)
    assert d["dg"][1, 70].abs().max() == 0 and d["dg"][1, 90].abs().max() == 0 and d["dg"][0, 100, 1] == 0
    ref = R.gated_delta_bwd(do=f64(do), **case64(k))
    for n, v in ref.items():
        close(d[n], v, bound(k), n)


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("beta", [0.3, 1.0, 1.9])
def test_equal_keys(beta, dtype):
    """One key over and over: the triangular system is as far from the identity as it gets, its inverse's
    entries are beta (1 - beta)^n all the same."""
    k = delta_case(1, 200, 1, 2, 32, 16, dtype, seed=5)
    k["k"] = k["k"][:, :1].expand(1, 200, 1, 32).contiguous()
    k["beta"] = torch.full_like(k["beta"], beta)
    k["g"] = k["g"] * 1e-3
    o, hf = ssm.gated_delta_fwd(return_final_state=True, **k)
    ro, rs = R.gated_delta(**case64(k))
    close(o, ro, bound(k), "o")
    close(hf, rs, bound(k), "h_final")
    do = torch.randn(k["v"].shape, generator=torch.Generator().manual_seed(2)).to(dtype).to(DEV)
    d = ssm.gated_delta_bwd(do=do, **k)
    for n, v in R.gated_delta_bwd(do=f64(do), **case64(k)).items():
        close(d[n], v, bound(k), n)


@pytest.mark.parametrize("dtype", **IDS)
def test_beta_of_zero_and_no_decay(dtype):
    """beta = 0 writes nothing (its own gradient is not 0), g = 0 forgets nothing."""
    k = delta_case(2, 90, 1, 1, 16, 16, dtype, seed=6)
    k["beta"][:, ::3] = 0
    k["g"].zero_()
    do = torch.randn(k["v"].shape, generator=torch.Generator().manual_seed(3)).to(dtype).to(DEV)
    d = ssm.gated_delta_bwd(do=do, **k)
    ref = R.gated_delta_bwd(do=f64(do), **case64(k))
    assert np.abs(ref["dbeta"][:, ::3]).max() > 0.01
    for n, v in ref.items():
        close(d[n], v, bound(k), n)


def test_a_step_of_large_decay_keeps_the_others_exact():
    """Strong decays ahead of weak ones in a chunk: the running sum is large where the differences are small.
    The forward is linear in what follows, so the weak part has to come out as if it stood alone."""
    k = delta_case(1, 64, 1, 1, 32, 32, F32, seed=7, h0=False)
    k["g"][:, :30] = -100.0  # not yet a reset
    o, hf = ssm.gated_delta_fwd(return_final_state=True, **k)
    ro, rs = R.gated_delta(**case64(k))
    close(o, ro, R.relative_bound(64, 32, 32), "o")
    close(hf, rs, R.relative_bound(64, 32, 32), "h_final")


def test_growing_decays():
    k = delta_case(1, 150, 1, 2, 24, 16, F32, seed=8, grow=0.02)
    o, hf = ssm.gated_delta_fwd(return_final_state=True, **k)
    ro, rs = R.gated_delta(**case64(k))
    # an error made early grows as the state does: by e^{0.02 * 150} = 20 at most
    close(o, ro, 20 * bound(k), "o")
    close(hf, rs, 20 * bound(k), "h_final")


@pytest.mark.parametrize("chunks,cut", [(31, 13), (80, 35)])
def test_long_sequences_carry_their_state(chunks, cut):
    """Two halves with the state handed over give what one call does: the halves meet at a chunk's border, so
    to the bit where no call is split into segments (31 chunks).  A long call and its halves are split in other
    places; each is then within the bound of the definition, and within two of one another, and both were
    rounded."""
    L, cut = 64 * chunks, 64 * cut
    k = delta_case(1, L, 2, 2, 64, 64, BF, seed=9)
    o, hf = ssm.gated_delta_fwd(return_final_state=True, **k)
    part = lambda a, b: {n: t[:, a:b].contiguous() for n, t in k.items()  # noqa: E731
                         if isinstance(t, torch.Tensor) and n != "h0"}
    o1, h1 = ssm.gated_delta_fwd(return_final_state=True, l2norm=True, h0=k["h0"], **part(0, cut))
    o2, h2 = ssm.gated_delta_fwd(return_final_state=True, l2norm=True, h0=h1, **part(cut, L))
    if chunks == 31:
        assert torch.equal(torch.cat([o1, o2], 1), o) and torch.equal(h2, hf)
    close(torch.cat([o1, o2], 1), f64(o), 2 * bound(k), "o", roundings=2)
    close(h2, f64(hf), 2 * bound(k), "h_final")


def test_offsets_past_32_bits():
    """Tensors of more than 2^32 bytes: a long row of which only the end is compared (the state handed over),
    many states, a wide product's last rows."""
    L, cut = (1 << 24) + 200, 1 << 24
    g = torch.Generator("cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=BF)  # noqa: E731
    q, k, v = n(1, L, 1, 128), n(1, L, 1, 128), n(1, L, 1, 136)
    gate = torch.full((1, L, 1), -0.01, device=DEV)
    beta = torch.full((1, L, 1), 0.5, device=DEV, dtype=BF)
    assert v.numel() * 2 > 1 << 32
    o, hf = ssm.gated_delta_fwd(q, k, v, gate, beta, l2norm=True, return_final_state=True)
    tail = [t[:, cut - 6400:].contiguous() for t in (q, k, v, gate, beta)]
    o2, hf2 = ssm.gated_delta_fwd(*tail, l2norm=True, return_final_state=True)
    # 6400 steps at e^-0.01 each leave e^-64 of what was before; both sides' outputs are rounded to bf16, so
    # two equal values but for 1e-5 may come out a whole step apart
    close(o[:, cut:], f64(o2[:, 6400:]), 1e-5, "o", roundings=2)
    close(hf, f64(hf2), 1e-5, "h_final")
    del q, k, v, gate, beta, o, tail
    B, H, K, V = 300, 256, 128, 128
    state = torch.zeros(B, H, K, V, device=DEV)
    assert state.numel() > 1 << 30
    one = n(B, 1, K), n(B, 1, K), n(B, H, V), torch.zeros(B, H, device=DEV), torch.ones(B, H, device=DEV, dtype=BF)
    got = ssm.gated_delta_step(state, *one, l2norm=True)
    few = torch.zeros(1, H, K, V, device=DEV)
    want = ssm.gated_delta_step(few, *(t[-1:].contiguous() for t in one), l2norm=True)
    assert torch.equal(got[-1:], want) and torch.equal(state[-1:], few)
    del state, few
    M, N, K = (1 << 18) + 100, 8200, 32
    xq, xs = ssm.quantize_fp8(n(M, K))
    wq, ws = ssm.quantize_fp8(n(N, K), 128)
    y = ssm.matmul_fp8(xq, xs, wq, ws)
    assert y.numel() > 1 << 31
    assert torch.equal(y[-300:], ssm.matmul_fp8(xq[-300:], xs[-300:].contiguous(), wq, ws))


def test_empty_calls():
    e = lambda *s, d=BF: torch.empty(*s, device=DEV, dtype=d)  # noqa: E731
    h0 = torch.randn(2, 4, 16, 8, device=DEV)
    o, hf = ssm.gated_delta_fwd(e(2, 0, 2, 16), e(2, 0, 2, 16), e(2, 0, 4, 8), e(2, 0, 4, d=F32), e(2, 0, 4), h0=h0,
                                return_final_state=True)
    assert o.shape == (2, 0, 4, 8) and torch.equal(hf, h0)
    d = ssm.gated_delta_bwd(e(2, 0, 2, 16), e(2, 0, 2, 16), e(2, 0, 4, 8), e(2, 0, 4, d=F32), e(2, 0, 4), e(2, 0, 4, 8),
                            h0=h0, dh_final=h0)
    assert torch.equal(d["dh0"], h0) and d["dq"].shape == (2, 0, 2, 16)
    _, hf = ssm.gated_delta_fwd(e(2, 0, 2, 16), e(2, 0, 2, 16), e(2, 0, 4, 8), e(2, 0, 4, d=F32), e(2, 0, 4),
                                return_final_state=True)
    assert (hf == 0).all()
    assert ssm.gated_delta_step(e(0, 4, 16, 8, d=F32), e(0, 2, 16), e(0, 2, 16), e(0, 4, 8), e(0, 4, d=F32),
                                e(0, 4)).shape == (0, 4, 8)
    q, s = ssm.quantize_fp8(e(0, 160))
    assert q.shape == (0, 160) and s.shape == (0, 2)
    wq, ws = ssm.quantize_fp8(torch.randn(24, 160, device=DEV), 128)
    assert ssm.matmul_fp8(q, s, wq, ws).shape == (0, 24)


def test_refusals_in_python():
    k = delta_case(2, 10, 2, 4, 16, 24, BF, seed=1)
    args = [k[n] for n in ("q", "k", "v", "g", "beta")]
    swap = lambda i, t: args[:i] + [t] + args[i + 1:]  # noqa: E731
    wrong = [(0, args[0][..., 0]), (0, args[0].cpu()), (1, args[1].float()), (1, args[1][:, :5]), (1, None),
             (2, args[2][0]), (2, args[2].transpose(1, 2)), (3, args[3].to(BF)), (3, args[3][..., :2]), (4, args[4].float()),
             (2, args[2].expand(2, 10, 4, 24)[..., ::2]), (0, args[0].half()), (1, args[1].transpose(2, 3).contiguous().transpose(2, 3))]
    for i, t in wrong:
        with pytest.raises((ValueError, TypeError)):
            ssm.gated_delta_fwd(*swap(i, t))
    with pytest.raises(ValueError):
        ssm.gated_delta_fwd(*args, h0=torch.zeros(2, 4, 24, 16, device=DEV))
    with pytest.raises(ValueError):
        ssm.gated_delta_fwd(*args, checkpoints=torch.zeros(1, 2, 4, 16, 24, device=DEV))
    with pytest.raises(ssm.SSMError):
        ssm.gated_delta_fwd(*args, scale=float("nan"))
    with pytest.raises(ssm.SSMError):  # heads that do not share evenly
        ssm.gated_delta_fwd(args[0], args[1], *(t[:, :, :3].contiguous() for t in args[2:]))
    with pytest.raises(ssm.SSMError):
        ssm.gated_delta_fwd(*(t[..., :12].contiguous() for t in args[:2]), *args[2:])
    with pytest.raises(ssm.SSMError, match="16-byte"):
        big = torch.zeros(2, 10, 2 * 16 + 4, device=DEV, dtype=BF)
        ssm.gated_delta_fwd(big[..., 4:].unflatten(-1, (2, 16)), *args[1:])
    state = torch.zeros(2, 4, 16, 24, device=DEV)
    one = [t[:, 0].contiguous() for t in args]
    for i, t in [(0, one[0][:1]), (2, one[2][:, :2]), (3, one[3].double()), (1, one[1][..., :8])]:
        with pytest.raises((ValueError, TypeError)):
            ssm.gated_delta_step(state, *one[:i], t, *one[i + 1:])
    with pytest.raises((ValueError, TypeError)):
        ssm.gated_delta_step(state.to(BF), *one)
    x = torch.randn(4, 160, device=DEV)
    with pytest.raises(ValueError):
        ssm.quantize_fp8(x, 1.5)
    with pytest.raises(ValueError):
        ssm.quantize_fp8(x[None], 128)
    with pytest.raises(ssm.SSMError):
        ssm.quantize_fp8(x[:, :24].contiguous())
    q, s = ssm.quantize_fp8(x)
    wq, ws = ssm.quantize_fp8(torch.randn(130, 160, device=DEV), 128)
    for bad in [(q.float(), s, wq, ws), (q, s[:, :1], wq, ws), (q, s, wq, ws[:1]), (q, s, wq[:, :128], ws), (q, ws, wq, s)]:
        with pytest.raises((ValueError, TypeError)):
            ssm.matmul_fp8(*bad)
    with pytest.raises(TypeError):
        ssm.matmul_fp8(q, s, wq, ws, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        ssm.matmul_fp8(q, s, wq, ws, y=torch.empty(4, 131, device=DEV))
