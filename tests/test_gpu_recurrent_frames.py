"""Stores of the gated recurrence and the fused norms stay inside their tensors (needs an MI355X):
every output and a workspace of exactly the size asked for lie in buffers whose other bytes keep
their value, and every element of an output is written.  Widths below, at and past a lane's
channels (4 in fp32, 8 in bf16; groups of 8 in the norms), a block's, a wave's and a workgroup's."""
import ctypes

import pytest
import torch

import selective_state_space_59_amd as ssm
from selective_state_space_59_amd import ssm as capi
from tests.recurrent_helpers import scan_case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
IDS = dict(argvalues=[F32, BF], ids=["f32", "bf16"])
PAD, MARK = 512, 0xA5


class Frames:
    """Tensors of their own buffer each, PAD marked bytes ahead and behind; `odd`: one element
    further in, so that a wide store has no alignment to rely on."""

    def __init__(self):
        self.all = []

    def take(self, shape, dtype, odd=True):
        size = torch.empty(0, dtype=dtype).element_size()
        n = size
        for s in shape:
            n *= s
        lo = PAD + (size if odd else 0)
        buf = torch.full((lo + n + PAD,), MARK, dtype=torch.uint8, device=DEV)
        buf[lo:lo + n] = 0xFF  # NaNs: an element that is not written shows
        self.all.append((buf, lo, n))
        return buf[lo:lo + n].view(dtype).view(shape)

    def like(self, tensors):
        return {k: self.take(tuple(t.shape), t.dtype) for k, t in tensors.items()}

    def check(self, what):
        torch.cuda.synchronize()
        for i, (buf, lo, n) in enumerate(self.all):
            assert (buf[:lo] == MARK).all() and (buf[lo + n:] == MARK).all(), "%s: around output %d" % (what, i)


def _run(call, args, frames, size=None, **tensors):
    """The C entry point `call`, with a workspace of exactly what `size` asks for."""
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


def _same(got, want, what):
    for n, t in want.items():
        assert torch.equal(got[n], t), (what, n)


SCAN_DIMS = {F32: (1, 3, 4, 5, 31, 32, 33), BF: (1, 7, 8, 9, 63, 64, 65)}


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("mode", ["decay", "sigmoid", "rate"])
@pytest.mark.parametrize("B,L", [(2, 5), (1, 200), (2, 257)])
def test_scan_and_its_backward(mode, B, L, dtype):
    for D in SCAN_DIMS[dtype]:
        what = "%s B=%d L=%d D=%d" % (mode, B, L, D)
        print(what, flush=True)
        k = scan_case(mode, B, L, D, dtype, seed=D, doc=40)
        ins = {m: v for m, v in k.items() if isinstance(v, torch.Tensor)}
        sizes = dict(batch=B, seqlen=L, dim=D, io_dtype=capi._io_code(dtype), mode=capi.GATE_MODES[mode])
        ck = torch.empty(ssm.gated_checkpoint_shape(B, L, D), device=DEV)
        y, hf = ssm.gated_scan_fwd(return_final_state=True, checkpoints=ck, **k)
        want = dict(y=y, h_final=hf, checkpoints=ck)
        fr = Frames()
        out = fr.like(want)
        _run("ssm_gated_scan_fwd", capi.GatedScanArgs(**sizes), fr, "ssm_gated_scan_workspace_size", **ins, **out)
        _same(out, want, what)
        dy = torch.randn(B, L, D, device=DEV).to(dtype)
        want = ssm.gated_scan_bwd(dy=dy, dh_final=hf, **k)
        for given in (ck, None):  # and the backward's own checkpoints in its workspace
            fr = Frames()
            out = fr.like(want)
            _run("ssm_gated_scan_bwd", capi.GatedScanBwdArgs(**sizes), fr, "ssm_gated_scan_bwd_workspace_size", **ins,
                 **out, dy=dy, dh_final=hf, checkpoints=given)
            _same(out, want, what)


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("mode", ["decay", "sigmoid", "rate"])
def test_step(mode, dtype):
    for B, D in ((1, 1), (3, 3), (2, 4), (5, 5), (2, 67), (1, 1025)):
        k = scan_case(mode, B, 1, D, dtype, seed=D, doc=2)
        start = k.pop("h0")
        one = {m: v[:, 0].contiguous() if m in ("x", "gate", "in_gate", "reset") else v for m, v in k.items()}
        ref = start.clone()
        want = dict(y=ssm.gated_scan_step(ref, **one), state=ref)
        fr = Frames()
        out = fr.like(want)
        out["state"].copy_(start)
        ins = {m: v for m, v in one.items() if isinstance(v, torch.Tensor)}
        a = capi.GatedStepArgs(batch=B, dim=D, io_dtype=capi._io_code(dtype), mode=capi.GATE_MODES[mode])
        _run("ssm_gated_scan_step", a, fr, **ins, **out)
        _same(out, want, "%s B=%d D=%d" % (mode, B, D))


NORM_WIDTHS = (1, 7, 8, 9, 64, 65, 257, 513, 769, 1025, 2049, 4097, 8193)


@pytest.mark.parametrize("res", **IDS)
@pytest.mark.parametrize("io", **IDS)
@pytest.mark.parametrize("options", [False, True], ids=["plain", "post_scale"])
def test_add_norm(options, io, res):
    for D in NORM_WIDTHS:
        rows = 3 if D > 300 else 41
        what = "%d x %d" % (rows, D)
        print(what, flush=True)
        r = lambda *s: torch.randn(*s, device=DEV)  # noqa: E731
        ins = dict(x=r(rows, D).to(io), w=r(D), residual=r(rows, D).to(res))
        if options:
            ins.update(scale=r(D), post_w=r(D))
        dy, dres = r(rows, D).to(io), r(rows, D).to(res)
        sizes = dict(rows=rows, dim=D, io_dtype=capi._io_code(io), res_dtype=capi._io_code(res), eps=1e-5)
        y, s = ssm.add_rmsnorm_fwd(**ins)
        fr = Frames()
        out = fr.like(dict(y=y, res_out=s))
        _run("ssm_add_rmsnorm_fwd", capi.AddNormArgs(**sizes), fr, **ins, **out)
        _same(out, dict(y=y, res_out=s), what)
        want = ssm.add_rmsnorm_bwd(dy=dy, dres_out=dres, **ins)
        fr = Frames()
        out = fr.like(want)
        _run("ssm_add_rmsnorm_bwd", capi.AddNormBwdArgs(**sizes), fr, "ssm_add_rmsnorm_bwd_workspace_size", **ins,
             **out, dy=dy, dres_out=dres)
        _same(out, want, what)


@pytest.mark.parametrize("io", **IDS)
@pytest.mark.parametrize("gate_first", [True, False], ids=["gate_first", "norm_first"])
def test_gated_norm(gate_first, io):
    for S in NORM_WIDTHS:
        for groups in (1, 3, 5):
            rows, D = (3 if S > 300 else 41), S * groups
            what = "%d x %d in %d" % (rows, D, groups)
            print(what, flush=True)
            r = lambda *s: torch.randn(*s, device=DEV)  # noqa: E731
            ins = dict(x=r(rows, D).to(io), z=r(rows, D).to(io), w=r(D))
            dy = r(rows, D).to(io)
            sizes = dict(rows=rows, dim=D, groups=groups, io_dtype=capi._io_code(io), gate_first=int(gate_first),
                         eps=1e-5)
            want = dict(y=ssm.gated_rmsnorm_fwd(**ins, groups=groups, gate_first=gate_first))
            fr = Frames()
            out = fr.like(want)
            _run("ssm_gated_rmsnorm_fwd", capi.GatedNormArgs(**sizes), fr, **ins, **out)
            _same(out, want, what)
            want = ssm.gated_rmsnorm_bwd(**ins, dy=dy, groups=groups, gate_first=gate_first)
            fr = Frames()
            out = fr.like(want)
            _run("ssm_gated_rmsnorm_bwd", capi.GatedNormBwdArgs(**sizes), fr, "ssm_gated_rmsnorm_bwd_workspace_size",
                 **ins, **out, dy=dy)
            _same(out, want, what)
