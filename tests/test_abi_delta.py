"""Host-side argument checks of the gated delta rule and the e4m3 calls (no GPU needed; see test_abi.py:
placeholder addresses, checks that finish before any HIP call)."""
import ctypes
import os
import subprocess

import pytest
import torch

from selective_state_space_59_amd import ssm

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder device addresses must not reach a real GPU")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, DTYPE, UNSUP, ALIAS, WS, ALIGN = (ssm.SSM_ERR_NULL_ARG, ssm.SSM_ERR_BAD_SHAPE, ssm.SSM_ERR_BAD_DTYPE,
                                               ssm.SSM_ERR_UNSUPPORTED, ssm.SSM_ERR_ALIAS, ssm.SSM_ERR_WORKSPACE,
                                               ssm.SSM_ERR_ALIGN)


def addr(i, off=0):
    return 0x7F0000000000 + i * (1 << 32) + off


STRUCTS = {"ssm_gated_delta_args_t": ssm.GatedDeltaArgs, "ssm_gated_delta_bwd_args_t": ssm.GatedDeltaBwdArgs,
           "ssm_gated_delta_step_args_t": ssm.GatedDeltaStepArgs, "ssm_quantize_fp8_args_t": ssm.QuantizeFp8Args,
           "ssm_add_norm_fp8_args_t": ssm.AddNormFp8Args, "ssm_matmul_fp8_args_t": ssm.MatmulFp8Args}


def test_ctypes_structs_match_c_layout(tmp_path):
    lines = ['printf("%s %%zu", sizeof(%s));' % (t, t) + "".join(
        ' printf(" %%zu", offsetof(%s, %s));' % (t, f) for f, _ in c._fields_) + ' printf("\\n");'
        for t, c in STRUCTS.items()]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ssm.h"\nint main(void) {\n%s\nreturn 0; }\n'
                   % "\n".join(lines))
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    for line in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines():
        t, size, *offs = line.split()
        c = STRUCTS[t]
        assert int(size) == ctypes.sizeof(c), t
        assert [int(o) for o in offs] == [getattr(c, f).offset for f, _ in c._fields_], t


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "ssm.h")).read()
    assert "#define SSM_DELTA_CHUNK %d\n" % ssm.DELTA_CHUNK in text
    assert "#define SSM_FP8_BLOCK %d\n" % ssm.FP8_BLOCK in text


def _run(name, cls, base, kw):
    a = cls(**base)
    for k, v in kw.items():
        setattr(a, k, v)
    return getattr(ssm.lib(), name)(ctypes.byref(a), None)


SIZES = dict(batch=2, seqlen=300, kheads=2, heads=4, kdim=64, vdim=72, io_dtype=ssm.SSM_BF16, l2norm=1, scale=0.1)
IN = dict(q=addr(0), k=addr(1), v=addr(2), g=addr(3), beta=addr(4), reset=addr(5), h0=addr(6))
FWD = dict(SIZES, **IN, o=addr(7), h_final=addr(8), checkpoints=addr(9), workspace=addr(10), workspace_bytes=1 << 31)
COMMON = [(dict(io_dtype=2), DTYPE), (dict(batch=-1), SHAPE), (dict(seqlen=-1), SHAPE), (dict(kheads=0), SHAPE),
          (dict(heads=0), SHAPE), (dict(heads=5), SHAPE), (dict(kdim=0), SHAPE), (dict(vdim=0), SHAPE),
          (dict(kdim=12), UNSUP), (dict(kdim=136), UNSUP), (dict(vdim=20), UNSUP), (dict(vdim=1032), UNSUP),
          (dict(l2norm=2), UNSUP), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
          (dict(batch=65536), UNSUP), (dict(kheads=65536, heads=65536, kdim=8, vdim=8), UNSUP),
          (dict(seqlen=1 << 30), UNSUP), (dict(heads=1 << 15, vdim=512), UNSUP),
          (dict(batch=60000, heads=4000, vdim=72), UNSUP),
          (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(g=None), NULL), (dict(beta=None), NULL),
          (dict(q=addr(0, 8)), ALIGN), (dict(k=addr(1, 2)), ALIGN), (dict(v=addr(2, 1)), ALIGN),
          (dict(g=addr(3, 2)), ALIGN), (dict(beta=addr(4, 1)), ALIGN), (dict(h0=addr(6, 2)), ALIGN),
          (dict(checkpoints=addr(9, 8)), ALIGN),
          (dict(q_token=132), ALIGN), (dict(q_token=-128), SHAPE), (dict(v_token=-1), SHAPE),
          (dict(k_token=1 << 24), SHAPE), (dict(k_token=128, k_batch=1 << 41), SHAPE), (dict(k_token=128, k_batch=12), ALIGN),
          (dict(workspace=None), WS), (dict(workspace_bytes=1000), WS), (dict(workspace=addr(10, 128)), WS),
          (dict(workspace=addr(0)), ALIAS)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(o=None), NULL), (dict(o=addr(7, 1)), ALIGN), (dict(h_final=addr(8, 2)), ALIGN), (dict(o=addr(2)), ALIAS),
    (dict(o=addr(0, 512)), ALIAS), (dict(h_final=addr(6)), ALIAS), (dict(h_final=addr(9, 64)), ALIAS),
    (dict(checkpoints=addr(1, 16)), ALIAS), (dict(o=addr(10, 4096)), ALIAS),
    # the gaps of a wider tensor count as its own
    (dict(v_token=1024, v_batch=300 * 1024, o=addr(2, 1024)), ALIAS)])
def test_forward(kw, status):
    assert _run("ssm_gated_delta_fwd", ssm.GatedDeltaArgs, FWD, kw) == status, ssm.lib().ssm_last_error_message()


BWD = dict(SIZES, **IN, dout=addr(7), dh_final=addr(8), checkpoints=addr(9), workspace=addr(10),
           workspace_bytes=1 << 31, dq=addr(11), dk=addr(12), dv=addr(13), dg=addr(14), dbeta=addr(15), dh0=addr(16))


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dout=None), NULL), (dict(dq=None), NULL), (dict(dk=None), NULL), (dict(dv=None), NULL), (dict(dg=None), NULL),
    (dict(dbeta=None), NULL), (dict(dq=addr(11, 1)), ALIGN), (dict(dg=addr(14, 2)), ALIGN), (dict(dq=addr(0)), ALIAS),
    (dict(dq=addr(12)), ALIAS), (dict(dv=addr(7)), ALIAS), (dict(dh0=addr(8)), ALIAS), (dict(dbeta=addr(4)), ALIAS),
    (dict(dh0=addr(9, 256)), ALIAS)])
def test_backward(kw, status):
    assert _run("ssm_gated_delta_bwd", ssm.GatedDeltaBwdArgs, BWD, kw) == status, ssm.lib().ssm_last_error_message()


STEP = dict(batch=3, kheads=2, heads=4, kdim=64, vdim=72, io_dtype=ssm.SSM_BF16, l2norm=1, scale=0.1, state=addr(0),
            q=addr(1), k=addr(2), v=addr(3), g=addr(4), beta=addr(5), reset=addr(6), o=addr(7))


@pytest.mark.parametrize("kw,status", [
    (dict(io_dtype=5), DTYPE), (dict(batch=-1), SHAPE), (dict(heads=3), SHAPE), (dict(kdim=4), UNSUP),
    (dict(vdim=12), UNSUP), (dict(l2norm=-1), UNSUP), (dict(state=None), NULL), (dict(q=None), NULL), (dict(o=None), NULL),
    (dict(state=addr(0, 4)), ALIGN), (dict(q=addr(1, 1)), ALIGN), (dict(g=addr(4, 2)), ALIGN), (dict(o=addr(0, 64)), ALIAS),
    (dict(o=addr(3)), ALIAS), (dict(state=addr(5)), ALIAS), (dict(q_batch=-8), SHAPE), (dict(v_batch=1 << 24), SHAPE)])
def test_step(kw, status):
    assert _run("ssm_gated_delta_step", ssm.GatedDeltaStepArgs, STEP, kw) == status, ssm.lib().ssm_last_error_message()


QUANT = dict(rows=100, dim=272, block_rows=1, io_dtype=ssm.SSM_BF16, x=addr(0), q=addr(1), scales=addr(2))


@pytest.mark.parametrize("kw,status", [
    (dict(io_dtype=2), DTYPE), (dict(rows=-1), SHAPE), (dict(dim=0), SHAPE), (dict(dim=264), UNSUP),
    (dict(dim=(1 << 20) + 16), UNSUP), (dict(block_rows=2), UNSUP), (dict(block_rows=0), UNSUP), (dict(x=None), NULL),
    (dict(q=None), NULL), (dict(scales=None), NULL), (dict(x=addr(0, 1)), ALIGN), (dict(q=addr(1, 8)), ALIGN),
    (dict(scales=addr(2, 2)), ALIGN), (dict(q=addr(0, 16)), ALIAS), (dict(scales=addr(1, 64)), ALIAS),
    (dict(rows=1 << 28, dim=16), UNSUP), (dict(rows=1 << 60), UNSUP)])
def test_quantize(kw, status):
    assert _run("ssm_quantize_fp8", ssm.QuantizeFp8Args, QUANT, kw) == status, ssm.lib().ssm_last_error_message()


NORM = dict(rows=100, dim=272, io_dtype=ssm.SSM_BF16, res_dtype=ssm.SSM_F32, x=addr(0), residual=addr(1), scale=addr(2),
            post_w=addr(3), w=addr(4), res_out=addr(5), eps=1e-5)


@pytest.mark.parametrize("norm,kw,status", [
    (dict(io_dtype=2), {}, DTYPE), (dict(res_dtype=-1), {}, DTYPE), (dict(rows=-1), {}, SHAPE), (dict(dim=0), {}, SHAPE),
    (dict(dim=264), {}, UNSUP), (dict(eps=0.0), {}, SHAPE), (dict(y=addr(9)), {}, SHAPE), (dict(x=None), {}, NULL),
    (dict(w=None), {}, NULL), ({}, dict(q=None), NULL), ({}, dict(scales=None), NULL), ({}, dict(q=addr(6, 4)), ALIGN),
    (dict(w=addr(4, 2)), {}, ALIGN), (dict(residual=addr(1, 2)), {}, ALIGN), ({}, dict(q=addr(0)), ALIAS),
    ({}, dict(scales=addr(5, 4)), ALIAS), (dict(res_out=addr(0)), {}, ALIAS), (dict(res_out=addr(1, 4)), {}, ALIAS)])
def test_norm(norm, kw, status):
    base = dict(norm=ssm.AddNormArgs(**dict(NORM, **norm)), q=addr(6), scales=addr(7))
    assert _run("ssm_add_rmsnorm_fp8", ssm.AddNormFp8Args, base, kw) == status, ssm.lib().ssm_last_error_message()


MATMUL = dict(m=100, n=200, k=272, out_dtype=ssm.SSM_BF16, xq=addr(0), x_scales=addr(1), wq=addr(2), w_scales=addr(3),
              y=addr(4))


@pytest.mark.parametrize("kw,status", [
    (dict(out_dtype=2), DTYPE), (dict(m=-1), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE), (dict(k=264), UNSUP),
    (dict(k=(1 << 20) + 16), UNSUP), (dict(n=1 << 24), UNSUP), (dict(m=1 << 31), UNSUP), (dict(m=1 << 30, n=1 << 12), UNSUP),
    (dict(xq=None), NULL), (dict(x_scales=None), NULL), (dict(wq=None), NULL), (dict(w_scales=None), NULL),
    (dict(y=None), NULL), (dict(xq=addr(0, 8)), ALIGN), (dict(wq=addr(2, 4)), ALIGN), (dict(w_scales=addr(3, 2)), ALIGN),
    (dict(y=addr(4, 1)), ALIGN), (dict(y=addr(0, 16)), ALIAS), (dict(y=addr(1)), ALIAS), (dict(y=addr(2, 64)), ALIAS),
    (dict(y=addr(3)), ALIAS)])
def test_matmul(kw, status):
    assert _run("ssm_matmul_fp8", ssm.MatmulFp8Args, MATMUL, kw) == status, ssm.lib().ssm_last_error_message()


def test_empty_calls_ask_for_nothing():
    """Nothing to do: no pointers, no workspace, no HIP call."""
    L = ssm.lib()
    for kw in (dict(batch=0), dict(seqlen=0)):
        sizes = dict(SIZES, **kw)
        a = ssm.GatedDeltaArgs(**sizes)
        assert L.ssm_gated_delta_workspace_size(ctypes.byref(a)) == 0
        b = ssm.GatedDeltaBwdArgs(**sizes)
        assert L.ssm_gated_delta_bwd_workspace_size(ctypes.byref(b)) == 0
        assert L.ssm_gated_delta_fwd(ctypes.byref(a), None) == ssm.SSM_OK
        assert L.ssm_gated_delta_bwd(ctypes.byref(b), None) == ssm.SSM_OK
    none = {k: v for k, v in SIZES.items() if k != "seqlen"}
    assert _run("ssm_gated_delta_step", ssm.GatedDeltaStepArgs, none, dict(batch=0)) == ssm.SSM_OK
    assert _run("ssm_quantize_fp8", ssm.QuantizeFp8Args, QUANT, dict(rows=0, x=None, q=None)) == ssm.SSM_OK
    assert _run("ssm_matmul_fp8", ssm.MatmulFp8Args, MATMUL, dict(m=0, xq=None, y=None)) == ssm.SSM_OK


def test_workspace_sizes():
    L = ssm.lib()
    size = lambda cls, fn, **kw: getattr(L, fn)(ctypes.byref(cls(**dict(SIZES, **kw))))  # noqa: E731
    bad = ctypes.c_size_t(-1).value
    assert size(ssm.GatedDeltaArgs, "ssm_gated_delta_workspace_size", kdim=12) == bad
    assert size(ssm.GatedDeltaBwdArgs, "ssm_gated_delta_bwd_workspace_size", io_dtype=9) == bad
    with_ck = size(ssm.GatedDeltaBwdArgs, "ssm_gated_delta_bwd_workspace_size", checkpoints=addr(0))
    without = size(ssm.GatedDeltaBwdArgs, "ssm_gated_delta_bwd_workspace_size")
    assert 0 < with_ck and without - with_ck == 5 * 2 * 4 * (64 + 64) * 72 * 4
