"""States carried through many tiles: sequences without resets whose channels forget slowly, so that
every tile's results depend on the whole chain before it (needs an MI355X).

With memories of thousands of steps a state that is lost, doubled or taken from a wrong tile, channel
or row is off by the state itself; the bounds allow some 1e-3 of it."""
import pytest
import torch

import selective_state_space_59_amd as ssm
from oracle import recurrent as R
from tests.recurrent_helpers import check, f64, scan_case, scan_case64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def slow_case(mode, B, L, D, dtype, seed):
    """Decays between about 0.9995 and 0.99999."""
    k = scan_case(mode, B, L, D, dtype, seed=seed, bias=mode == "rate", in_gate=mode == "rate")
    g = torch.Generator().manual_seed(seed + 1)
    if mode == "decay":
        k["gate"] = (1 - 5e-4 * torch.rand(B, L, D, generator=g)).to(dtype).to(DEV)
    elif mode == "sigmoid":
        k["gate"] = (-8 - 3 * torch.rand(B, L, D, generator=g)).to(dtype).to(DEV)
    else:
        k["A"] = (-5e-4 * torch.rand(D, generator=g) - 2e-5).to(DEV)
    return k


@pytest.mark.parametrize("mode,dtype", [("decay", F32), ("sigmoid", F32), ("sigmoid", BF), ("rate", F32), ("rate", BF)],
                         ids=["decay_f32", "sigmoid_f32", "sigmoid_bf16", "rate_f32", "rate_bf16"])
@pytest.mark.parametrize("B,L,D", [(2, 5000, 72), (1, 2816, 200), (2, 20000, 70), (3, 16640, 24)])
def test_slow_channels(mode, dtype, B, L, D):
    """More tiles than one look back takes, and chains of 64 tiles and more (65, 79; backward 130,
    157), whose number is not a multiple of 8, over several channel blocks and rows."""
    k = slow_case(mode, B, L, D, dtype, seed=L + D)
    what = "%s %s B=%d L=%d D=%d" % (mode, dtype, B, L, D)
    print(what, flush=True)
    ck = torch.full(ssm.gated_checkpoint_shape(B, L, D), float("nan"), device=DEV)
    y, hf = ssm.gated_scan_fwd(return_final_state=True, checkpoints=ck, **k)
    torch.cuda.synchronize()
    k64 = scan_case64(k)
    H, _, E = R.gated_scan(**k64)
    check(y, H, E, what + " y")
    check(hf, H[:, -1], E[:, -1], what + " h_final")
    for j in range(1, ck.shape[0]):
        check(ck[j], H[:, 128 * j - 1], E[:, 128 * j - 1], "%s checkpoint %d" % (what, j))
    g = torch.Generator().manual_seed(7)
    dy = torch.randn(B, L, D, generator=g).to(dtype).to(DEV)
    dh = torch.randn(B, D, generator=g).to(DEV)
    got = ssm.gated_scan_bwd(dy=dy, dh_final=dh, checkpoints=ck, **k)
    torch.cuda.synchronize()
    for n, (v, e) in R.gated_scan_bwd(dy=f64(dy), dh_final=f64(dh), **k64).items():
        check(got[n], v, e, "%s %s" % (what, n))


def test_two_streams_every_time():
    """Chains on two streams at once: every result of every turn, final states and gradients
    included, is the one of a call alone."""
    k1, k2 = slow_case("rate", 1, 6000, 128, BF, 3), slow_case("sigmoid", 1, 7000, 96, F32, 4)

    def call(k):
        y, hf = ssm.gated_scan_fwd(return_final_state=True, **k)
        return [y, hf, *ssm.gated_scan_bwd(dy=y, dh_final=hf, **k).values()]

    want = [call(k1), call(k2)]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(4):
        for i, (s, k) in enumerate(zip(streams, (k1, k2))):
            with torch.cuda.stream(s):
                got[i].append(call(k))
    torch.cuda.synchronize()
    for i in range(2):
        for turn, run in enumerate(got[i]):
            assert all(torch.equal(a, b) for a, b in zip(run, want[i])), (i, turn)


def test_decoded_rows_pass_the_norm_like_prefilled_ones():
    """Tokens of a prefill and of the decode step through the gated norm: a row that is the same ahead
    of it is the same behind it, and such rows there are (the two evaluations differ by some 1e-7
    of a value, so one value in thousands rounds to another bf16)."""
    B, L, P, D = 3, 40, 33, 96
    k = scan_case("rate", B, L, D, BF, seed=21)
    z, w = torch.randn(B, L, D, device=DEV).to(BF), torch.ones(D, device=DEV)
    h, _ = ssm.gated_scan_fwd(**k)
    out = ssm.gated_rmsnorm_fwd(h, z, w, groups=4)
    cut = lambda lo, hi: {m: v[:, lo:hi].contiguous() if m in ("x", "gate", "in_gate") else v  # noqa: E731
                          for m, v in k.items()}
    _, state = ssm.gated_scan_fwd(return_final_state=True, **cut(0, P))
    same = 0
    for t in range(P, L):
        zt = z[:, t].contiguous()
        assert torch.equal(ssm.gated_rmsnorm_fwd(h[:, t].contiguous(), zt, w, groups=4), out[:, t])
        one = {m: v[:, 0] if m in ("x", "gate", "in_gate") else v for m, v in cut(t, t + 1).items() if m != "h0"}
        ht = ssm.gated_scan_step(state, **{m: v.contiguous() if isinstance(v, torch.Tensor) else v
                                           for m, v in one.items()})
        got = ssm.gated_rmsnorm_fwd(ht, zt, w, groups=4)
        for b in range(B):
            if torch.equal(ht[b], h[b, t]):
                same += 1
                assert torch.equal(got[b], out[b, t])
    assert same > 0
