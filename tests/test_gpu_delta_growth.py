"""Decays above 1 in the gated delta rule (needs an MI355X).  A chunk computed at once subtracts numbers as
large as its largest product of decays, which a state that keys write over again and again never reaches;
stepping does not.  The forward, the backward and the decode step have to agree all the same.

With keys of one channel (k the unit vector of channel J, q a multiple of it) each value channel is a
recurrence of numbers,
  s' = a s,  e = v - s',  s = s' + beta e,  o = scale c s,
whose errors shrink by m = a |1 - beta| a step.  With `top` the largest |v| and |s'|, fp32 steps make at most
5 u (e^g: 2 units in the last place, its product) + 1 (e) + 1 (beta e) + 1 (s) roundings of numbers up to
2 top each, so a state is off by at most r = 16 u top / (1 - m) in all, and so is e; backwards the same
holds of the state's gradient.  A gradient that is a sum of products is then off by the factors' errors,
the sum's own roundings (V + 8 terms) and the rounding to its type."""

import numpy as np
import pytest
import torch

import selective_state_space_59_amd as ssm
from oracle import delta as R
from selective_state_space_59_amd import ssm as capi
from tests.delta_helpers import bound, case64, close, delta_case
from tests.recurrent_helpers import check, f64
from tests.test_gpu_delta_edges import _call, _same, _take
from tests.test_gpu_recurrent_block import _capture, _flat
from tests.test_gpu_recurrent_frames import Frames

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
IDS = dict(argvalues=[F32, BF], ids=["f32", "bf16"])
U, J, Q = 2.0 ** -24, 3, 0.5


def _case(B, L, Hk, H, K, V, dtype, g, beta, seed, doc=0):
    """One key channel; head 1 of each row forgets, the others' log decays are `g` (a number, or one a step)."""
    n = torch.Generator().manual_seed(seed)
    k = torch.zeros(B, L, Hk, K)
    k[..., J] = 1
    gates = torch.empty(B, L, H)
    gates[:] = torch.as_tensor(g, dtype=F32).reshape(-1, 1)
    if H > 1:
        gates[:, :, 1] = -0.05
    h0 = torch.zeros(B, H, K, V)
    h0[:, :, J] = torch.randn(B, H, V, generator=n)
    c = dict(q=(Q * k).to(dtype), k=k.to(dtype), v=torch.randn(B, L, H, V, generator=n).to(dtype), g=gates,
             beta=torch.full((B, L, H), beta).to(dtype), h0=h0)
    if doc:
        c["reset"] = (torch.rand(B, L, generator=n) < 1.0 / doc).to(torch.uint8)
    return {m: t.to(DEV) for m, t in c.items()}


def _numbers(k, do, dhf):
    """What the recurrence of numbers gives, forwards and backwards: {name: (value, size of the sum)}."""
    v, g, b, d = f64(k["v"]), f64(k["g"]), f64(k["beta"])[..., None], f64(do)
    B, L, H, V = v.shape
    K, share = k["q"].shape[-1], H // k["q"].shape[2]
    scale = K ** -0.5
    a = np.exp(g)
    if "reset" in k:
        a = np.where(f64(k["reset"])[..., None] != 0, 0.0, a)
    s = f64(k["h0"])[:, :, J]
    old, err, new = (np.empty_like(v) for _ in range(3))
    for t in range(L):
        old[:, t] = a[:, t, :, None] * s
        err[:, t] = v[:, t] - old[:, t]
        new[:, t] = s = old[:, t] + b[:, t] * err[:, t]
    ds = f64(dhf)[:, :, J].copy()
    du, after = np.empty_like(v), np.empty_like(v)
    for t in reversed(range(L)):
        du[:, t] = ds = ds + scale * Q * d[:, t]
        after[:, t] = ds = ds - b[:, t] * ds
        ds = a[:, t, :, None] * ds
    top, back = max(np.abs(v).max(), np.abs(old).max(), np.abs(new).max()), np.abs(du).max()
    m = (a * np.abs(1 - b[..., 0])).max()
    assert m < 0.6
    rs, rd = 16 * U * top / (1 - m), 16 * U * max(back, np.abs(ds).max()) / (1 - m)
    one = lambda x: (x, np.abs(x))  # noqa: E731

    def product(*pairs):  # sums over the value channels of products of two numbers, off by rs and rd each
        off = [rs * np.abs(y) + ry * np.abs(x) + (V + 8) * U * np.abs(x * y) for x, y, ry in pairs]
        return sum(sign * (x * y) for sign, (x, y, _) in zip((1, -1), pairs)).sum(-1), sum(off).sum(-1)

    def channel(pair):  # of channel J, summed over the heads that share it
        out = []
        for x in pair:
            full = np.zeros((B, L, k["q"].shape[2], K))
            full[..., J] = x.reshape(B, L, -1, share).sum(-1)
            out.append(full)
        return tuple(out)

    def state(x, off):
        out = np.zeros((B, H, K, V)), np.zeros((B, H, K, V))
        out[0][:, :, J], out[1][:, :, J] = x, off
        return out

    dq = product((new, scale * d, 0.0))
    dk = product((b * err, du, rd), (old, b * du, rd))
    db, dg = product((err, du, rd)), product((old, after, rd))
    return dict(o=(scale * Q * new, 2 * rs + 0 * new), h_final=state(s, rs), dv=(b * du, rd + 0 * du), dq=channel(dq),
                dk=channel(dk), dbeta=db, dg=dg, dh0=state(ds, rd))


def _compare(got, want, what):
    for n, (x, off) in want.items():
        check(got[n], x, off, "%s %s" % (what, n))


CASES = [(0.1, 0.9), (0.3, 1.0), (2.0, 1.0)]


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("g,beta", CASES)
@pytest.mark.parametrize("shape,doc", [((2, 150, 1, 2, 16, 24), 0), ((1, 64, 2, 2, 128, 8), 0), ((2, 333, 1, 3, 72, 40), 60)],
                         ids=["shared", "chunk", "documents"])
def test_keys_of_one_channel(shape, doc, g, beta, dtype):
    """Products of decays of e^6 to e^666, states no larger than the values."""
    B, L, Hk, H, K, V = shape
    k = _case(*shape, dtype, g, beta, seed=L, doc=doc)
    n = torch.Generator().manual_seed(7)
    do = torch.randn(B, L, H, V, generator=n).to(dtype).to(DEV)
    dhf = torch.zeros(B, H, K, V)
    dhf[:, :, J] = torch.randn(B, H, V, generator=n)
    dhf = dhf.to(DEV)
    want = _numbers(k, do, dhf)
    ck = torch.full(ssm.gated_delta_checkpoint_shape(B, L, H, K, V), float("nan"), device=DEV)
    o, hf = ssm.gated_delta_fwd(return_final_state=True, checkpoints=ck, **k)
    _compare(dict(o=o, h_final=hf), {m: want.pop(m) for m in ("o", "h_final")}, "forward")
    assert torch.isfinite(ck).all()
    for given in (ck, None):
        d = ssm.gated_delta_bwd(do=do, dh_final=dhf, checkpoints=given, **k)
        _compare(d, want, "backward, checkpoints %s" % (given is not None))
    # the decode step, from the same state
    state, parts = k["h0"].clone(), ("q", "k", "v", "g", "beta", "reset")
    outs = [ssm.gated_delta_step(state, **{m: k[m][:, t].contiguous() for m in parts if m in k}) for t in range(L)]
    step = _numbers(k, do, dhf)
    _compare(dict(o=torch.stack(outs, 1), h_final=state), {m: step[m] for m in ("o", "h_final")}, "step")


@pytest.mark.parametrize("dtype", **IDS)
def test_a_growing_stretch_of_a_sequence_in_segments(dtype):
    """64 growing steps across a chunk's border in the middle of 40 chunks; the heads beside them as without."""
    B, L, Hk, H, K, V = 1, 2560, 1, 3, 64, 24
    g = torch.full((L,), -0.05)
    g[1300:1364] = 0.5
    k = _case(B, L, Hk, H, K, V, dtype, g, 1.0, seed=3)
    do = torch.randn(B, L, H, V, generator=torch.Generator().manual_seed(8)).to(dtype).to(DEV)
    dhf = torch.zeros(B, H, K, V, device=DEV)
    want = _numbers(k, do, dhf)
    o, hf = ssm.gated_delta_fwd(return_final_state=True, **k)
    d = ssm.gated_delta_bwd(do=do, dh_final=dhf, **k)
    _compare(dict(d, o=o, h_final=hf), want, "segments")
    calm = dict(k, g=torch.full_like(k["g"], -0.05))
    o2, hf2 = ssm.gated_delta_fwd(return_final_state=True, **calm)
    assert torch.equal(o[:, :, 1], o2[:, :, 1]) and torch.equal(hf[:, 1], hf2[:, 1])


@pytest.mark.parametrize("dtype", **IDS)
def test_slow_growth_through_many_chunks(dtype):
    """Decays that multiply to e^0.77 a chunk and e^30 over the sequence, in segments: the chunks are computed at
    once, where an error grows by less than e, and the keys leave a tenth of it to the next step."""
    B, L, Hk, H, K, V = 1, 2560, 1, 2, 16, 24
    k = _case(B, L, Hk, H, K, V, dtype, 0.012, 0.9, seed=6)
    do = torch.randn(B, L, H, V, generator=torch.Generator().manual_seed(8)).to(dtype).to(DEV)
    dhf = torch.zeros(B, H, K, V, device=DEV)
    want = _numbers(k, do, dhf)
    o, hf = ssm.gated_delta_fwd(return_final_state=True, **k)
    d = dict(ssm.gated_delta_bwd(do=do, dh_final=dhf, **k), o=o, h_final=hf)
    for n, (x, _) in want.items():
        close(d[n], x, 2 * np.e * R.relative_bound(64, K, V), n)


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("l2norm", [True, False])
def test_random_keys(l2norm, dtype):
    """Keys of 8 channels, the state growing slowly: errors reach the end through the products of the steps'
    maps, `amp` the largest norm of one."""
    B, L, Hk, H, K, V = 2, 150, 2, 4, 8, 16
    k = delta_case(B, L, Hk, H, K, V, dtype, seed=5, l2norm=l2norm, doc=50)
    k["g"] = torch.full_like(k["g"], 0.05)
    k["g"][:, :, 1] = -0.2
    k64 = case64(k)
    amp = 1.0
    kk = k64["k"] / np.sqrt((k64["k"] ** 2).sum(-1, keepdims=True) + 1e-6) if l2norm else k64["k"]
    for b in range(B):
        for h in range(H):
            maps = np.empty((0, K, K))
            for t in range(L):
                x = kk[b, t, h * Hk // H]
                a = 0.0 if k64["reset"][b, t] else np.exp(k64["g"][b, t, h])
                maps = np.concatenate([maps, np.eye(K)[None]]) if t else np.eye(K)[None]
                maps = a * ((np.eye(K) - k64["beta"][b, t, h] * np.outer(x, x)) @ maps)
                amp = max(amp, np.linalg.norm(maps, 2, axis=(1, 2)).max())
    assert amp < 30
    o, hf = ssm.gated_delta_fwd(return_final_state=True, **k)
    ro, rs = R.gated_delta(**k64)
    close(o, ro, amp * bound(k), "o")
    close(hf, rs, amp * bound(k), "h_final")
    do = torch.randn(B, L, H, V, generator=torch.Generator().manual_seed(2)).to(dtype).to(DEV)
    d = ssm.gated_delta_bwd(do=do, dh_final=hf, **k)
    for n, v in R.gated_delta_bwd(do=f64(do), dh_final=f64(hf), **k64).items():
        close(d[n], v, amp * bound(k), n)


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("shape", [(2, 65, 1, 2, 72, 24), (1, 1, 1, 1, 8, 8), (1, 130, 2, 6, 128, 136)],
                         ids=lambda s: "x".join(map(str, s)))
def test_stores_stay_inside(shape, dtype):
    """Every output and a workspace of exactly the size asked for lie in marked memory."""
    B, L, Hk, H, K, V = shape
    k = _case(*shape, dtype, 1.5, 1.0, seed=L, doc=20)
    sizes = dict(batch=B, seqlen=L, kheads=Hk, heads=H, kdim=K, vdim=V, io_dtype=capi._io_code(dtype), l2norm=0,
                 scale=K ** -0.5)
    ck = torch.empty(ssm.gated_delta_checkpoint_shape(B, L, H, K, V), device=DEV)
    o, hf = ssm.gated_delta_fwd(return_final_state=True, checkpoints=ck, **k)
    want = dict(o=o, h_final=hf, checkpoints=ck)
    fr = Frames()
    out = _take(fr, want, aligned=("checkpoints",))
    _call("ssm_gated_delta_fwd", capi.GatedDeltaArgs(**sizes), fr, "ssm_gated_delta_workspace_size", **k, **out)
    _same(out, want, "forward")
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    want = ssm.gated_delta_bwd(do=do, dh_final=hf, **k)
    for given in (ck, None):
        fr = Frames()
        out = _take(fr, want)
        _call("ssm_gated_delta_bwd", capi.GatedDeltaBwdArgs(**sizes), fr, "ssm_gated_delta_bwd_workspace_size", **k,
              **out, dout=do, dh_final=hf, checkpoints=given)
        _same(out, want, "backward")


def test_a_captured_call_whose_decays_begin_to_grow():
    """Which heads grow is found anew in each replay."""
    B, L, Hk, H, K, V = 1, 150, 1, 2, 16, 24
    k = _case(B, L, Hk, H, K, V, BF, -0.1, 1.0, seed=9)
    do = torch.randn(B, L, H, V, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    gates = [k["g"].clone(), torch.where(k["g"] == k["g"][0, 0, 0], 0.4, k["g"])]

    def call():
        o, hf = ssm.gated_delta_fwd(return_final_state=True, **k)
        return o, hf, ssm.gated_delta_bwd(do=do, **k)

    want = []
    for g in gates:
        k["g"].copy_(g)
        want.append([t.clone() for t in _flat(call())])
    k["g"].copy_(gates[0])
    graph, out = _capture(call)
    for i in (0, 1, 0, 1, 1, 0):
        k["g"].copy_(gates[i])
        call()  # eager work between replays
        torch.cuda.synchronize()
        for t in _flat(out):
            t.view(torch.uint8).fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(_flat(out), want[i]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
