"""Host-side argument checks of the gated recurrence and the fused norms (no GPU needed; see
test_abi.py: placeholder addresses, checks that finish before any HIP call)."""
import ctypes
import os
import subprocess

import pytest
import torch

from selective_state_space_59_amd import ssm

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="placeholder device addresses must not reach a real GPU")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, DTYPE, UNSUP, ALIAS, WS, HIP, ALIGN = (ssm.SSM_ERR_NULL_ARG, ssm.SSM_ERR_BAD_SHAPE,
                                                    ssm.SSM_ERR_BAD_DTYPE, ssm.SSM_ERR_UNSUPPORTED,
                                                    ssm.SSM_ERR_ALIAS, ssm.SSM_ERR_WORKSPACE, ssm.SSM_ERR_HIP,
                                                    ssm.SSM_ERR_ALIGN)


def addr(i, off=0):
    return 0x7F0000000000 + i * (1 << 32) + off


STRUCTS = {"ssm_gated_scan_args_t": ssm.GatedScanArgs, "ssm_gated_scan_bwd_args_t": ssm.GatedScanBwdArgs,
           "ssm_gated_step_args_t": ssm.GatedStepArgs, "ssm_add_norm_args_t": ssm.AddNormArgs,
           "ssm_add_norm_bwd_args_t": ssm.AddNormBwdArgs, "ssm_gated_norm_args_t": ssm.GatedNormArgs,
           "ssm_gated_norm_bwd_args_t": ssm.GatedNormBwdArgs}


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
    assert "#define SSM_GATED_BLOCK %d " % ssm.GATED_BLOCK in text
    for name, code in ssm.GATE_MODES.items():
        assert "SSM_GATE_%s = %d" % (name.upper(), code) in text


def _make(cls, base, kw):
    a = cls(**base)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _run(name, a):
    return getattr(ssm.lib(), name)(ctypes.byref(a), None)


SCAN = dict(batch=2, seqlen=300, dim=64, io_dtype=ssm.SSM_BF16, mode=2, x=addr(0), gate=addr(1), in_gate=addr(2),
            A=addr(3), gate_bias=addr(4), in_bias=addr(5), reset=addr(6), h0=addr(7), y=addr(8), h_final=addr(9),
            checkpoints=addr(10), workspace=addr(11), workspace_bytes=1 << 31)
GATES = [
    (dict(io_dtype=2), DTYPE), (dict(batch=-1), SHAPE), (dict(seqlen=-1), SHAPE), (dict(dim=0), SHAPE),
    (dict(dim=(1 << 20) + 1), UNSUP), (dict(mode=3), UNSUP), (dict(mode=-1), UNSUP), (dict(seqlen=1 << 60), SHAPE),
    (dict(batch=1 << 24, seqlen=1), UNSUP), (dict(mode=0), SHAPE), (dict(mode=1), SHAPE),
    (dict(mode=0, A=None, in_gate=None, in_bias=None), SHAPE), (dict(in_gate=None), SHAPE),
    (dict(x=None), NULL), (dict(gate=None), NULL), (dict(A=None), NULL), (dict(x=addr(0, 1)), ALIGN),
    (dict(gate_bias=addr(4, 2)), ALIGN)]


@pytest.mark.parametrize("kw,status", GATES + [
    (dict(y=None), NULL), (dict(h0=addr(7, 1)), ALIGN), (dict(y=addr(0)), ALIAS), (dict(y=addr(1, 64)), ALIAS),
    (dict(h_final=addr(7)), ALIAS), (dict(h_final=addr(10, 4)), ALIAS), (dict(checkpoints=addr(2, 4)), ALIAS),
    (dict(reset=addr(8, 3)), ALIAS)])
def test_scan_refusals(kw, status):
    assert _run("ssm_gated_scan_fwd", _make(ssm.GatedScanArgs, SCAN, kw)) == status
    assert ssm.lib().ssm_last_error_message().decode() != ""


def test_scan_passes_its_checks():
    for kw in ({}, dict(mode=1, A=None, in_gate=None, in_bias=None),
               dict(mode=0, A=None, in_gate=None, in_bias=None, gate_bias=None),
               dict(in_gate=None, in_bias=None, gate_bias=None, reset=None, h0=None, h_final=None, checkpoints=None)):
        assert _run("ssm_gated_scan_fwd", _make(ssm.GatedScanArgs, SCAN, kw)) == HIP  # no device here
    assert _run("ssm_gated_scan_fwd", _make(ssm.GatedScanArgs, SCAN, dict(batch=0))) == ssm.SSM_OK
    assert _run("ssm_gated_scan_fwd", _make(ssm.GatedScanArgs, SCAN, dict(seqlen=0, h_final=None))) == ssm.SSM_OK
    for f in ("ssm_gated_scan_fwd", "ssm_gated_scan_bwd", "ssm_gated_scan_step", "ssm_add_rmsnorm_fwd",
              "ssm_add_rmsnorm_bwd", "ssm_gated_rmsnorm_fwd", "ssm_gated_rmsnorm_bwd"):
        assert getattr(ssm.lib(), f)(None, None) == NULL


BWD = dict(batch=2, seqlen=300, dim=64, io_dtype=ssm.SSM_BF16, mode=2, x=addr(0), gate=addr(1), in_gate=addr(2),
           A=addr(3), gate_bias=addr(4), in_bias=addr(5), reset=addr(6), h0=addr(7), dy=addr(8), dh_final=addr(9),
           checkpoints=addr(10), dx=addr(11), dgate=addr(12), din_gate=addr(13), dA=addr(14), dgate_bias=addr(15),
           din_bias=addr(16), dh0=addr(17), workspace=addr(18), workspace_bytes=1 << 31)


@pytest.mark.parametrize("kw,status", GATES + [
    (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(dgate=None), NULL), (dict(din_gate=None), NULL),
    (dict(dA=None), NULL), (dict(mode=1, A=None, in_gate=None, in_bias=None), SHAPE),
    (dict(in_gate=None, in_bias=None), SHAPE), (dict(dx=addr(8)), ALIAS), (dict(dgate=addr(11, 64)), ALIAS),
    (dict(dh0=addr(9)), ALIAS), (dict(dA=addr(3)), ALIAS), (dict(workspace=addr(18, 8)), WS),
    (dict(workspace_bytes=16), WS), (dict(workspace=None), WS), (dict(workspace=addr(8)), ALIAS),
    (dict(workspace=addr(11)), ALIAS)])
def test_scan_backward_refusals(kw, status):
    a = _make(ssm.GatedScanBwdArgs, BWD, kw)
    assert _run("ssm_gated_scan_bwd", a) == status
    assert ssm.lib().ssm_last_error_message().decode() != ""


def test_workspace_sizes():
    L = ssm.lib()
    big = ctypes.c_size_t(-1).value
    assert L.ssm_gated_scan_workspace_size(None) == big
    assert L.ssm_gated_scan_workspace_size(ctypes.byref(_make(ssm.GatedScanArgs, SCAN, dict(dim=0)))) == big
    assert L.ssm_gated_scan_workspace_size(ctypes.byref(_make(ssm.GatedScanArgs, SCAN, dict(batch=0)))) == 0
    sizes_only = _make(ssm.GatedScanArgs, {}, dict(batch=2, seqlen=300, dim=64, io_dtype=1, mode=2))
    assert (L.ssm_gated_scan_workspace_size(ctypes.byref(sizes_only))
            == L.ssm_gated_scan_workspace_size(ctypes.byref(_make(ssm.GatedScanArgs, SCAN, {}))))
    w = L.ssm_gated_scan_bwd_workspace_size
    with_ck = w(ctypes.byref(_make(ssm.GatedScanBwdArgs, BWD, {})))
    assert 0 < with_ck < w(ctypes.byref(_make(ssm.GatedScanBwdArgs, BWD, dict(checkpoints=None)))) < big
    assert _run("ssm_gated_scan_bwd", _make(ssm.GatedScanBwdArgs, BWD, dict(workspace_bytes=with_ck - 1))) == WS
    assert _run("ssm_gated_scan_bwd", _make(ssm.GatedScanBwdArgs, BWD, dict(workspace_bytes=with_ck))) == HIP


def test_grid_limit():
    """B ceil(L / 128) ceil(D / 32) < 2^23: one more would be 2^32 threads in a launch."""
    size = lambda **kw: ssm.lib().ssm_gated_scan_workspace_size(  # noqa: E731
        ctypes.byref(_make(ssm.GatedScanArgs, dict(io_dtype=1, mode=2), kw)))
    none = ctypes.c_size_t(-1).value
    for B, L, D in ((1 << 23, 1, 1), (1 << 23, 128, 32), (1 << 22, 129, 24), (1 << 21, 200, 33), (1, 1 << 30, 1)):
        assert size(batch=B, seqlen=L, dim=D) == none, (B, L, D)
        if L == 1:
            assert _run("ssm_gated_scan_step", _make(ssm.GatedStepArgs, STEP, dict(batch=B, dim=D))) == UNSUP
    for B, L, D in (((1 << 23) - 1, 1, 1), ((1 << 23) - 1, 128, 32), ((1 << 22) - 1, 129, 24), (1, (1 << 30) - 128, 1),
                    (127, 1, 1 << 20), ((1 << 23) - 1, 0, 32)):
        assert size(batch=B, seqlen=L, dim=D) != none, (B, L, D)


STEP = dict(batch=2, dim=64, io_dtype=ssm.SSM_BF16, mode=2, state=addr(0), x=addr(1), gate=addr(2), in_gate=addr(3),
            A=addr(4), gate_bias=addr(5), in_bias=addr(6), reset=addr(7), y=addr(8))


@pytest.mark.parametrize("kw,status", [(k, s) for k, s in GATES if "seqlen" not in k] + [
    (dict(state=None), NULL), (dict(y=None), NULL), (dict(y=addr(0)), ALIAS), (dict(y=addr(1)), ALIAS),
    (dict(state=addr(2, 4)), ALIAS), (dict(state=addr(0, 2)), ALIGN), ({}, HIP), (dict(batch=0, x=None), ssm.SSM_OK)])
def test_step_refusals(kw, status):
    assert _run("ssm_gated_scan_step", _make(ssm.GatedStepArgs, STEP, kw)) == status


NORM = dict(rows=5, dim=64, io_dtype=1, res_dtype=0, x=addr(0), residual=addr(1), scale=addr(2), post_w=addr(3),
            w=addr(4), res_out=addr(5), y=addr(6), eps=1e-5)
SIZES = [(dict(rows=-1), SHAPE), (dict(dim=0), SHAPE), (dict(dim=1 << 21), UNSUP), (dict(io_dtype=9), DTYPE),
         (dict(eps=0.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
         (dict(rows=1 << 60), SHAPE)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(res_dtype=3), DTYPE), (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL),
    (dict(x=addr(0, 1)), ALIGN), (dict(residual=addr(1, 2)), ALIGN), (dict(scale=addr(2, 1)), ALIGN),
    (dict(y=addr(0)), ALIAS), (dict(res_out=addr(0)), ALIAS), (dict(res_out=addr(1, 4)), ALIAS),
    (dict(y=addr(5)), ALIAS), (dict(res_out=addr(1)), HIP), (dict(res_out=None, residual=None), HIP), ({}, HIP),
    (dict(rows=0, x=None), ssm.SSM_OK)])
def test_add_norm_refusals(kw, status):
    assert _run("ssm_add_rmsnorm_fwd", _make(ssm.AddNormArgs, NORM, kw)) == status


NBWD = dict(rows=5, dim=64, io_dtype=1, res_dtype=0, x=addr(0), residual=addr(1), scale=addr(2), post_w=addr(3),
            w=addr(4), dy=addr(5), dres_out=addr(6), dx=addr(7), dresidual=addr(8), dw=addr(9), dscale=addr(10),
            dpost_w=addr(11), workspace=addr(12), workspace_bytes=1 << 31, eps=1e-5)


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(res_dtype=3), DTYPE), (dict(x=None), NULL), (dict(dy=None), NULL), (dict(dx=None), NULL),
    (dict(dw=None), NULL), (dict(residual=None), SHAPE), (dict(scale=None), SHAPE), (dict(post_w=None), SHAPE),
    (dict(dx=addr(5)), ALIAS), (dict(dresidual=addr(6)), HIP), (dict(dresidual=addr(6, 4)), ALIAS),
    (dict(dw=addr(4)), ALIAS), (dict(workspace=None), WS), (dict(workspace=addr(12, 4)), WS),
    (dict(workspace_bytes=8), WS), (dict(workspace=addr(7)), ALIAS), ({}, HIP)])
def test_add_norm_backward_refusals(kw, status):
    assert _run("ssm_add_rmsnorm_bwd", _make(ssm.AddNormBwdArgs, NBWD, kw)) == status


GN = dict(rows=5, dim=64, groups=4, io_dtype=1, gate_first=1, x=addr(0), z=addr(1), w=addr(2), y=addr(3), eps=1e-5)


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(groups=0), SHAPE), (dict(groups=3), SHAPE), (dict(gate_first=2), UNSUP), (dict(z=None), NULL),
    (dict(y=None), NULL), (dict(z=addr(1, 1)), ALIGN), (dict(y=addr(0, 2)), ALIAS), (dict(y=addr(2)), ALIAS),
    (dict(y=addr(0)), HIP), (dict(y=addr(1)), HIP), ({}, HIP), (dict(rows=0, z=None), ssm.SSM_OK)])
def test_gated_norm_refusals(kw, status):
    assert _run("ssm_gated_rmsnorm_fwd", _make(ssm.GatedNormArgs, GN, kw)) == status


GNB = dict(rows=5, dim=64, groups=4, io_dtype=1, gate_first=1, x=addr(0), z=addr(1), w=addr(2), dy=addr(3),
           dx=addr(4), dz=addr(5), dw=addr(6), workspace=addr(7), workspace_bytes=1 << 31, eps=1e-5)


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(groups=7), SHAPE), (dict(dz=None), NULL), (dict(dw=None), NULL), (dict(dx=addr(0)), ALIAS),
    (dict(dz=addr(4)), ALIAS), (dict(dw=addr(6, 2)), ALIGN), (dict(workspace=None), WS),
    (dict(workspace_bytes=0), WS), ({}, HIP)])
def test_gated_norm_backward_refusals(kw, status):
    assert _run("ssm_gated_rmsnorm_bwd", _make(ssm.GatedNormBwdArgs, GNB, kw)) == status
