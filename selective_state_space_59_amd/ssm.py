"""Python binding of the C-ABI library libssm_hip.so (argument marshalling only).

Every function here checks tensor devices, dtypes, shapes and contiguity,
allocates the outputs it is not given, and passes raw device pointers plus
torch's current HIP stream to the library.  All arithmetic runs in the HIP
kernels; if the library is missing this module raises instead of computing
anything itself.

Names and semantics mirror include/ssm.h.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssm_hip.so")

SSM_OK = 0
SSM_ERR_NULL_ARG = 1
SSM_ERR_BAD_SHAPE = 2
SSM_ERR_BAD_DTYPE = 3
SSM_ERR_UNSUPPORTED = 4
SSM_ERR_ALIAS = 5
SSM_ERR_WORKSPACE = 6
SSM_ERR_HIP = 7
SSM_ERR_ALIGN = 8
SSM_F32 = 0
SSM_BF16 = 1
MAX_DSTATE = 16
MAX_CONV_K = 4

EXPORTED_SYMBOLS = ("ssm_selective_scan_workspace_size", "ssm_selective_scan_fwd",
                    "ssm_causal_conv1d_silu", "ssm_state_update", "ssm_status_string",
                    "ssm_last_error_message", "ssm_abi_version",
                    "ssm_selective_scan_bwd_workspace_size", "ssm_selective_scan_bwd",
                    "ssm_block_plan_create", "ssm_block_workspace_size", "ssm_block_fwd",
                    "ssm_block_plan_destroy", "ssm_ssd_fwd", "ssm_ssd_workspace_size",
                    "ssm_ssd_step", "ssm_selective_scan_fwd_noalloc",
                    "ssm_gated_scan_workspace_size", "ssm_gated_scan_fwd",
                    "ssm_gated_scan_bwd_workspace_size", "ssm_gated_scan_bwd", "ssm_gated_scan_step",
                    "ssm_add_rmsnorm_fwd", "ssm_add_rmsnorm_bwd_workspace_size", "ssm_add_rmsnorm_bwd",
                    "ssm_gated_rmsnorm_fwd", "ssm_gated_rmsnorm_bwd_workspace_size",
                    "ssm_gated_rmsnorm_bwd")
NOALLOC_SCRATCH_BYTES = 32 << 20

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32


class ScanArgs(ctypes.Structure):
    """Mirror of ssm_scan_args_t."""
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("dim", _I64), ("dstate", _I64),
                ("io_dtype", _I32), ("delta_softplus", _I32), ("conv_k", _I64),
                ("x", _P), ("delta", _P), ("Bm", _P), ("Cm", _P), ("z", _P),
                ("A", _P), ("Dskip", _P), ("delta_bias", _P), ("conv_w", _P), ("conv_b", _P),
                ("h0", _P), ("y", _P), ("h_final", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t),
                ("conv_state_in", _P), ("conv_state_out", _P), ("checkpoints", _P)]


class StateUpdateArgs(ctypes.Structure):
    """Mirror of ssm_state_update_args_t."""
    _fields_ = [("batch", _I64), ("dim", _I64), ("dstate", _I64),
                ("io_dtype", _I32), ("delta_softplus", _I32),
                ("state", _P), ("x", _P), ("delta", _P), ("z", _P), ("Bm", _P), ("Cm", _P),
                ("A", _P), ("Dskip", _P), ("delta_bias", _P), ("y", _P),
                ("conv_k", _I64), ("conv_w", _P), ("conv_b", _P), ("conv_state", _P)]


class ScanBwdArgs(ctypes.Structure):
    """Mirror of ssm_scan_bwd_args_t."""
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("dim", _I64), ("dstate", _I64),
                ("io_dtype", _I32), ("delta_softplus", _I32), ("conv_k", _I64),
                ("x", _P), ("delta", _P), ("Bm", _P), ("Cm", _P), ("z", _P),
                ("A", _P), ("Dskip", _P), ("delta_bias", _P), ("conv_w", _P), ("conv_b", _P),
                ("h0", _P), ("dy", _P), ("dh_final", _P),
                ("dx", _P), ("ddelta", _P), ("dz", _P), ("dA", _P), ("dBm", _P), ("dCm", _P),
                ("dDskip", _P), ("ddelta_bias", _P), ("dconv_w", _P), ("dconv_b", _P),
                ("dh0", _P), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t),
                ("conv_state_in", _P), ("dconv_state_in", _P), ("checkpoints", _P)]


class BlockDims(ctypes.Structure):
    """Mirror of ssm_block_dims_t."""
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("d_model", _I64), ("d_inner", _I64),
                ("dstate", _I64), ("dt_rank", _I64), ("conv_k", _I64)]


class BlockWeights(ctypes.Structure):
    """Mirror of ssm_block_weights_t."""
    _fields_ = [("norm_w", _P), ("w_in", _P), ("conv_w", _P), ("conv_b", _P), ("w_x", _P),
                ("w_dt", _P), ("dt_bias", _P), ("A", _P), ("Dskip", _P), ("w_out", _P),
                ("norm_eps", ctypes.c_float)]


class SsdArgs(ctypes.Structure):
    """Mirror of ssm_ssd_args_t."""
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("nheads", _I64), ("headdim", _I64),
                ("ngroups", _I64), ("dstate", _I64), ("io_dtype", _I32), ("delta_softplus", _I32),
                ("x", _P), ("delta", _P), ("A", _P), ("Bm", _P), ("Cm", _P), ("Dskip", _P),
                ("z", _P), ("delta_bias", _P), ("h0", _P), ("y", _P), ("h_final", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class SsdStepArgs(ctypes.Structure):
    """Mirror of ssm_ssd_step_args_t."""
    _fields_ = [("batch", _I64), ("nheads", _I64), ("headdim", _I64), ("ngroups", _I64),
                ("dstate", _I64), ("io_dtype", _I32), ("delta_softplus", _I32), ("state", _P),
                ("x", _P), ("delta", _P), ("A", _P), ("Bm", _P), ("Cm", _P), ("Dskip", _P),
                ("z", _P), ("delta_bias", _P), ("y", _P)]


class GatedScanArgs(ctypes.Structure):
    """Mirror of ssm_gated_scan_args_t."""
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("dim", _I64), ("io_dtype", _I32), ("mode", _I32),
                ("x", _P), ("gate", _P), ("in_gate", _P), ("A", _P), ("gate_bias", _P), ("in_bias", _P),
                ("reset", _P), ("h0", _P), ("y", _P), ("h_final", _P), ("checkpoints", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class GatedScanBwdArgs(ctypes.Structure):
    """Mirror of ssm_gated_scan_bwd_args_t."""
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("dim", _I64), ("io_dtype", _I32), ("mode", _I32),
                ("x", _P), ("gate", _P), ("in_gate", _P), ("A", _P), ("gate_bias", _P), ("in_bias", _P),
                ("reset", _P), ("h0", _P), ("dy", _P), ("dh_final", _P), ("checkpoints", _P),
                ("dx", _P), ("dgate", _P), ("din_gate", _P), ("dA", _P), ("dgate_bias", _P),
                ("din_bias", _P), ("dh0", _P), ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


class GatedStepArgs(ctypes.Structure):
    """Mirror of ssm_gated_step_args_t."""
    _fields_ = [("batch", _I64), ("dim", _I64), ("io_dtype", _I32), ("mode", _I32), ("state", _P),
                ("x", _P), ("gate", _P), ("in_gate", _P), ("A", _P), ("gate_bias", _P), ("in_bias", _P),
                ("reset", _P), ("y", _P)]


class AddNormArgs(ctypes.Structure):
    """Mirror of ssm_add_norm_args_t."""
    _fields_ = [("rows", _I64), ("dim", _I64), ("io_dtype", _I32), ("res_dtype", _I32), ("x", _P),
                ("residual", _P), ("scale", _P), ("post_w", _P), ("w", _P), ("res_out", _P), ("y", _P),
                ("eps", ctypes.c_float)]


class AddNormBwdArgs(ctypes.Structure):
    """Mirror of ssm_add_norm_bwd_args_t."""
    _fields_ = [("rows", _I64), ("dim", _I64), ("io_dtype", _I32), ("res_dtype", _I32), ("x", _P),
                ("residual", _P), ("scale", _P), ("post_w", _P), ("w", _P), ("dy", _P), ("dres_out", _P),
                ("dx", _P), ("dresidual", _P), ("dw", _P), ("dscale", _P), ("dpost_w", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t), ("eps", ctypes.c_float)]


class GatedNormArgs(ctypes.Structure):
    """Mirror of ssm_gated_norm_args_t."""
    _fields_ = [("rows", _I64), ("dim", _I64), ("groups", _I64), ("io_dtype", _I32), ("gate_first", _I32),
                ("x", _P), ("z", _P), ("w", _P), ("y", _P), ("eps", ctypes.c_float)]


class GatedNormBwdArgs(ctypes.Structure):
    """Mirror of ssm_gated_norm_bwd_args_t."""
    _fields_ = [("rows", _I64), ("dim", _I64), ("groups", _I64), ("io_dtype", _I32), ("gate_first", _I32),
                ("x", _P), ("z", _P), ("w", _P), ("dy", _P), ("dx", _P), ("dz", _P), ("dw", _P),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t), ("eps", ctypes.c_float)]


class SSMError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libssm_hip.so (built by selective_state_space_59_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libssm_hip.so is not built; run "
                               "`python -m selective_state_space_59_amd.build` first")
        L = ctypes.CDLL(LIB_PATH)
        L.ssm_selective_scan_workspace_size.argtypes = [ctypes.POINTER(ScanArgs)]
        L.ssm_selective_scan_workspace_size.restype = ctypes.c_size_t
        L.ssm_selective_scan_fwd.argtypes = [ctypes.POINTER(ScanArgs), _P]
        L.ssm_selective_scan_fwd.restype = ctypes.c_int
        L.ssm_selective_scan_fwd_noalloc.argtypes = [ctypes.POINTER(ScanArgs), _P]
        L.ssm_selective_scan_fwd_noalloc.restype = ctypes.c_int
        L.ssm_causal_conv1d_silu.argtypes = [_I64, _I64, _I64, _I64, _I32, _P, _P, _P, _P, _P]
        L.ssm_causal_conv1d_silu.restype = ctypes.c_int
        L.ssm_state_update.argtypes = [ctypes.POINTER(StateUpdateArgs), _P]
        L.ssm_state_update.restype = ctypes.c_int
        L.ssm_status_string.argtypes = [ctypes.c_int]
        L.ssm_status_string.restype = ctypes.c_char_p
        L.ssm_last_error_message.argtypes = []
        L.ssm_last_error_message.restype = ctypes.c_char_p
        L.ssm_abi_version.argtypes = []
        L.ssm_abi_version.restype = ctypes.c_int
        L.ssm_selective_scan_bwd_workspace_size.argtypes = [ctypes.POINTER(ScanBwdArgs)]
        L.ssm_selective_scan_bwd_workspace_size.restype = ctypes.c_size_t
        L.ssm_selective_scan_bwd.argtypes = [ctypes.POINTER(ScanBwdArgs), _P]
        L.ssm_selective_scan_bwd.restype = ctypes.c_int
        L.ssm_block_plan_create.argtypes = [ctypes.POINTER(BlockDims), ctypes.POINTER(_P)]
        L.ssm_block_plan_create.restype = ctypes.c_int
        L.ssm_block_workspace_size.argtypes = [_P]
        L.ssm_block_workspace_size.restype = ctypes.c_size_t
        L.ssm_block_fwd.argtypes = [_P, ctypes.POINTER(BlockWeights), _P, _P, _P, ctypes.c_size_t, _P]
        L.ssm_block_fwd.restype = ctypes.c_int
        L.ssm_block_plan_destroy.argtypes = [_P]
        L.ssm_block_plan_destroy.restype = None
        L.ssm_ssd_fwd.argtypes = [ctypes.POINTER(SsdArgs), _P]
        L.ssm_ssd_fwd.restype = ctypes.c_int
        L.ssm_ssd_workspace_size.argtypes = [ctypes.POINTER(SsdArgs)]
        L.ssm_ssd_step.argtypes = [ctypes.POINTER(SsdStepArgs), _P]
        L.ssm_ssd_step.restype = ctypes.c_int
        L.ssm_ssd_workspace_size.restype = ctypes.c_size_t
        for name, args in (("gated_scan_fwd", GatedScanArgs), ("gated_scan_bwd", GatedScanBwdArgs),
                           ("gated_scan_step", GatedStepArgs), ("add_rmsnorm_fwd", AddNormArgs),
                           ("add_rmsnorm_bwd", AddNormBwdArgs), ("gated_rmsnorm_fwd", GatedNormArgs),
                           ("gated_rmsnorm_bwd", GatedNormBwdArgs)):
            f = getattr(L, "ssm_" + name)
            f.argtypes, f.restype = [ctypes.POINTER(args), _P], ctypes.c_int
        for name, args in (("gated_scan", GatedScanArgs), ("gated_scan_bwd", GatedScanBwdArgs),
                           ("add_rmsnorm_bwd", AddNormBwdArgs), ("gated_rmsnorm_bwd", GatedNormBwdArgs)):
            f = getattr(L, "ssm_%s_workspace_size" % name)
            f.argtypes, f.restype = [ctypes.POINTER(args)], ctypes.c_size_t
        _lib = L
    return _lib


def abi_version() -> int:
    return lib().ssm_abi_version()


def status_string(status: int) -> str:
    return lib().ssm_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != SSM_OK:
        msg = lib().ssm_last_error_message().decode()
        raise SSMError(status, "%s failed: %s (%s)" % (what, status_string(status), msg))


def _io_code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return SSM_BF16
    if dtype == torch.float32:
        return SSM_F32
    raise TypeError("I/O tensors must be bfloat16 or float32, got %s" % dtype)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _req(t, name, shape, dtype, device):
    if t is None:
        raise ValueError("%s is required" % name)
    return _opt(t, name, shape, dtype, device)


def _opt(t, name, shape, dtype, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _changed(*tensors):
    """Count the given tensors as changed in place.  Autograd does not see the library's writes: a
    call marks the tensors it was given to write into (those it allocates are new), so that a
    backward which saved one of them raises."""
    for t in tensors:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _scan_args(x, delta, A, Bm, Cm, Dskip, z, delta_bias, delta_softplus, conv_w, conv_b, h0,
               y, h_final, conv_state_in=None, conv_state_out=None, checkpoints=None):
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a (B, L, D) tensor")
    if x.device.type != "cuda":
        raise ValueError("x must be on a GPU")
    dev = x.device
    Bsz, L, D = x.shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a (D, N) float32 tensor")
    N = A.shape[1]
    io = x.dtype
    _req(x, "x", (Bsz, L, D), io, dev)
    _req(delta, "delta", (Bsz, L, D), io, dev)
    _req(A, "A", (D, N), torch.float32, dev)
    _req(Bm, "Bm", (Bsz, L, N), io, dev)
    _req(Cm, "Cm", (Bsz, L, N), io, dev)
    _opt(z, "z", (Bsz, L, D), io, dev)
    _opt(Dskip, "Dskip", (D,), torch.float32, dev)
    _opt(delta_bias, "delta_bias", (D,), torch.float32, dev)
    K = 0
    if conv_w is not None:
        if conv_w.dim() != 2:
            raise ValueError("conv_w must be (D, K)")
        K = conv_w.shape[1]
        _req(conv_w, "conv_w", (D, K), torch.float32, dev)
    _opt(conv_b, "conv_b", (D,), torch.float32, dev)
    _opt(h0, "h0", (Bsz, D, N), torch.float32, dev)
    _req(y, "y", (Bsz, L, D), io, dev)
    _opt(h_final, "h_final", (Bsz, D, N), torch.float32, dev)
    if (conv_state_in is not None or conv_state_out is not None) and K == 0:
        raise ValueError("a conv state needs conv_w")
    _opt(conv_state_in, "conv_state_in", (Bsz, max(K - 1, 0), D), io, dev)
    _opt(conv_state_out, "conv_state_out", (Bsz, max(K - 1, 0), D), io, dev)
    _opt(checkpoints, "checkpoints", checkpoint_shape(Bsz, L, D), torch.float32, dev)
    a = ScanArgs(batch=Bsz, seqlen=L, dim=D, dstate=N, io_dtype=_io_code(io),
                 delta_softplus=int(bool(delta_softplus)), conv_k=K,
                 x=_ptr(x), delta=_ptr(delta), Bm=_ptr(Bm), Cm=_ptr(Cm), z=_ptr(z), A=_ptr(A),
                 Dskip=_ptr(Dskip), delta_bias=_ptr(delta_bias), conv_w=_ptr(conv_w),
                 conv_b=_ptr(conv_b), h0=_ptr(h0), y=_ptr(y), h_final=_ptr(h_final),
                 workspace=None, workspace_bytes=0, conv_state_in=_ptr(conv_state_in),
                 conv_state_out=_ptr(conv_state_out), checkpoints=_ptr(checkpoints))
    return a, dev


SCAN_BLOCK = 16  # SSM_SCAN_BLOCK
MAX_DSTATE = 16  # SSM_MAX_DSTATE


def checkpoint_shape(batch: int, seqlen: int, dim: int) -> tuple:
    """Shape of the fp32 checkpoint tensor a forward writes for the backward: the state
    entering every SCAN_BLOCK-step block, (ceil(L / SCAN_BLOCK), B, D, MAX_DSTATE)."""
    return ((seqlen + SCAN_BLOCK - 1) // SCAN_BLOCK, batch, dim, MAX_DSTATE)


_ws_cache = {}


def _workspace(dev: torch.device, nbytes: int) -> torch.Tensor:
    """Cached scratch tensor per device and stream (grown on demand).  Calls on one stream
    run in order and share it; calls on different streams get different ones.

    A call made while the current stream is being captured into a HIP graph gets a fresh
    tensor of its own instead: every capture without an explicit stream runs on the same
    side stream, and two graphs that recorded one cached buffer would race on it when
    replayed at the same time.  The graph's memory pool keeps that tensor alive."""
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    key = (dev.type, dev.index, torch.cuda.current_stream(dev).cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
        _ws_cache[key] = buf
    return buf


def selective_scan_workspace_size(x, delta, A, Bm, Cm, Dskip=None, z=None, delta_bias=None,
                                  delta_softplus=False, conv_w=None, conv_b=None, h0=None,
                                  return_final_state=False) -> int:
    y = torch.empty_like(x)
    hf = (torch.empty(x.shape[0], x.shape[2], A.shape[1], device=x.device, dtype=torch.float32)
          if return_final_state else None)
    a, _ = _scan_args(x, delta, A, Bm, Cm, Dskip, z, delta_bias, delta_softplus, conv_w, conv_b,
                      h0, y, hf)
    n = lib().ssm_selective_scan_workspace_size(ctypes.byref(a))
    if n == ctypes.c_size_t(-1).value:
        raise SSMError(SSM_ERR_BAD_SHAPE, "invalid sizes")
    return int(n)


def selective_scan_fwd(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor,
                       Cm: torch.Tensor, Dskip: Optional[torch.Tensor] = None,
                       z: Optional[torch.Tensor] = None,
                       delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
                       conv_w: Optional[torch.Tensor] = None,
                       conv_b: Optional[torch.Tensor] = None,
                       h0: Optional[torch.Tensor] = None, return_final_state: bool = False,
                       y: Optional[torch.Tensor] = None,
                       h_final: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       conv_state_in: Optional[torch.Tensor] = None,
                       conv_state_out: Optional[torch.Tensor] = None,
                       return_conv_state: bool = False,
                       checkpoints: Optional[torch.Tensor] = None):
    """ssm_selective_scan_fwd.  Returns (y, h_final or None), or with
    return_conv_state (or a conv_state_out given) (y, h_final or None,
    conv_state_out); conv states are (B, K-1, D) in x's dtype.  A float32 tensor
    `checkpoints` of checkpoint_shape(B, L, D) also receives the state entering every
    SCAN_BLOCK-step block, for selective_scan_bwd(checkpoints=...)."""
    given = (y, h_final, conv_state_out, checkpoints)
    if y is None:
        y = torch.empty_like(x)
    if return_final_state and h_final is None:
        h_final = torch.empty(x.shape[0], x.shape[2], A.shape[1], device=x.device,
                              dtype=torch.float32)
    want_cs = return_conv_state or conv_state_out is not None
    if return_conv_state and conv_state_out is None:
        if conv_w is None:
            raise ValueError("a conv state needs conv_w")
        conv_state_out = torch.empty(x.shape[0], max(conv_w.shape[1] - 1, 0), x.shape[2],
                                     device=x.device, dtype=x.dtype)
    a, dev = _scan_args(x, delta, A, Bm, Cm, Dskip, z, delta_bias, delta_softplus, conv_w,
                        conv_b, h0, y, h_final, conv_state_in, conv_state_out, checkpoints)
    need = lib().ssm_selective_scan_workspace_size(ctypes.byref(a))
    if need == ctypes.c_size_t(-1).value:
        _check(lib().ssm_selective_scan_fwd(ctypes.byref(a), None), "ssm_selective_scan_fwd")
    if need > 0:
        ws = workspace if workspace is not None else _workspace(dev, need)
        if ws.device != dev or ws.numel() * ws.element_size() < need:
            raise ValueError("workspace must be a device tensor of >= %d bytes" % need)
        a.workspace = ws.data_ptr()
        a.workspace_bytes = ws.numel() * ws.element_size()
    _check(lib().ssm_selective_scan_fwd(ctypes.byref(a), _stream(dev)), "ssm_selective_scan_fwd")
    _changed(*given)
    return (y, h_final, conv_state_out) if want_cs else (y, h_final)


def selective_scan_fwd_noalloc(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor,
                               Bm: torch.Tensor, Cm: torch.Tensor,
                               Dskip: Optional[torch.Tensor] = None,
                               z: Optional[torch.Tensor] = None,
                               delta_bias: Optional[torch.Tensor] = None,
                               delta_softplus: bool = False,
                               conv_w: Optional[torch.Tensor] = None,
                               conv_b: Optional[torch.Tensor] = None,
                               h0: Optional[torch.Tensor] = None,
                               y: Optional[torch.Tensor] = None,
                               h_final: Optional[torch.Tensor] = None,
                               conv_state_in: Optional[torch.Tensor] = None,
                               conv_state_out: Optional[torch.Tensor] = None,
                               checkpoints: Optional[torch.Tensor] = None):
    """ssm_selective_scan_fwd_noalloc: the scan with its workspace in the library's
    scratch array on the device (no workspace tensor).  The outputs y, h_final,
    conv_state_out and checkpoints must be given when wanted (nothing is allocated here
    either).  Returns (y, h_final)."""
    if y is None:
        raise ValueError("y is required (the no-allocation scan allocates nothing)")
    a, dev = _scan_args(x, delta, A, Bm, Cm, Dskip, z, delta_bias, delta_softplus, conv_w,
                        conv_b, h0, y, h_final, conv_state_in, conv_state_out, checkpoints)
    _check(lib().ssm_selective_scan_fwd_noalloc(ctypes.byref(a), _stream(dev)),
           "ssm_selective_scan_fwd_noalloc")
    _changed(y, h_final, conv_state_out, checkpoints)
    return y, h_final


def selective_scan_args(x, delta, A, Bm, Cm, Dskip=None, z=None, delta_bias=None,
                        delta_softplus=False, conv_w=None, conv_b=None, h0=None, y=None,
                        h_final=None, conv_state_in=None, conv_state_out=None, checkpoints=None):
    """The checked ssm_scan_args_t of a selective_scan_fwd call with a workspace of its own,
    for callers that launch the same scan repeatedly through lib().ssm_selective_scan_fwd.
    Returns (args, y, workspace or None); y is allocated when not given.  The tensors must
    outlive the struct."""
    if y is None:
        y = torch.empty_like(x)
    a, dev = _scan_args(x, delta, A, Bm, Cm, Dskip, z, delta_bias, delta_softplus, conv_w,
                        conv_b, h0, y, h_final, conv_state_in, conv_state_out, checkpoints)
    need = lib().ssm_selective_scan_workspace_size(ctypes.byref(a))
    if need == ctypes.c_size_t(-1).value:
        _check(lib().ssm_selective_scan_fwd(ctypes.byref(a), None), "ssm_selective_scan_fwd")
    ws = None
    if need > 0:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        a.workspace = ws.data_ptr()
        a.workspace_bytes = need
    return a, y, ws


def causal_conv1d_silu(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ssm_causal_conv1d_silu on x (B, L, D) with weights w (D, K)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3 or x.device.type != "cuda":
        raise ValueError("x must be a (B, L, D) GPU tensor")
    dev = x.device
    Bsz, L, D = x.shape
    if w.dim() != 2:
        raise ValueError("w must be (D, K)")
    K = w.shape[1]
    _req(x, "x", (Bsz, L, D), x.dtype, dev)
    _req(w, "w", (D, K), torch.float32, dev)
    _opt(bias, "bias", (D,), torch.float32, dev)
    given = out
    if out is None:
        out = torch.empty_like(x)
    _req(out, "out", (Bsz, L, D), x.dtype, dev)
    _check(lib().ssm_causal_conv1d_silu(Bsz, L, D, K, _io_code(x.dtype), _ptr(x), _ptr(w),
                                        _ptr(bias), _ptr(out), _stream(dev)),
           "ssm_causal_conv1d_silu")
    _changed(given)
    return out


def state_update(state: torch.Tensor, x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor,
                 Bm: torch.Tensor, Cm: torch.Tensor, Dskip: Optional[torch.Tensor] = None,
                 z: Optional[torch.Tensor] = None, delta_bias: Optional[torch.Tensor] = None,
                 delta_softplus: bool = False, y: Optional[torch.Tensor] = None,
                 conv_w: Optional[torch.Tensor] = None, conv_b: Optional[torch.Tensor] = None,
                 conv_state: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ssm_state_update: advances `state` (B, D, N) -- and with conv_w the conv
    window `conv_state` (B, K-1, D) -- in place and returns y (B, D)."""
    a, out = state_update_args(state, x, delta, A, Bm, Cm, Dskip, z, delta_bias, delta_softplus, y,
                               conv_w, conv_b, conv_state)
    _check(lib().ssm_state_update(ctypes.byref(a), _stream(state.device)), "ssm_state_update")
    _changed(state, y, conv_state)
    return out


def state_update_args(state, x, delta, A, Bm, Cm, Dskip=None, z=None, delta_bias=None,
                      delta_softplus=False, y=None, conv_w=None, conv_b=None, conv_state=None):
    """The checked ssm_state_update_args_t of a state_update call, and its y (allocated
    when not given), for callers that launch the same step repeatedly through
    lib().ssm_state_update.  The tensors must outlive the struct."""
    if not isinstance(state, torch.Tensor) or state.dim() != 3 or state.device.type != "cuda":
        raise ValueError("state must be a (B, D, N) float32 GPU tensor")
    dev = state.device
    Bsz, D, N = state.shape
    io = x.dtype
    _req(state, "state", (Bsz, D, N), torch.float32, dev)
    _req(x, "x", (Bsz, D), io, dev)
    _req(delta, "delta", (Bsz, D), io, dev)
    _opt(z, "z", (Bsz, D), io, dev)
    _req(Bm, "Bm", (Bsz, N), io, dev)
    _req(Cm, "Cm", (Bsz, N), io, dev)
    _req(A, "A", (D, N), torch.float32, dev)
    _opt(Dskip, "Dskip", (D,), torch.float32, dev)
    _opt(delta_bias, "delta_bias", (D,), torch.float32, dev)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", (Bsz, D), io, dev)
    K = 0
    if conv_w is not None:
        if conv_w.dim() != 2:
            raise ValueError("conv_w must be (D, K)")
        K = conv_w.shape[1]
        _req(conv_w, "conv_w", (D, K), torch.float32, dev)
        if K > 1:
            _req(conv_state, "conv_state", (Bsz, K - 1, D), io, dev)
    elif conv_b is not None or conv_state is not None:
        raise ValueError("conv_b/conv_state need conv_w")
    _opt(conv_b, "conv_b", (D,), torch.float32, dev)
    a = StateUpdateArgs(batch=Bsz, dim=D, dstate=N, io_dtype=_io_code(io),
                        delta_softplus=int(bool(delta_softplus)), state=_ptr(state), x=_ptr(x),
                        delta=_ptr(delta), z=_ptr(z), Bm=_ptr(Bm), Cm=_ptr(Cm), A=_ptr(A),
                        Dskip=_ptr(Dskip), delta_bias=_ptr(delta_bias), y=_ptr(y), conv_k=K,
                        conv_w=_ptr(conv_w), conv_b=_ptr(conv_b),
                        conv_state=_ptr(conv_state) if K > 1 else None)
    return a, y


def selective_scan_bwd(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor,
                       Cm: torch.Tensor, dy: torch.Tensor, Dskip: Optional[torch.Tensor] = None,
                       z: Optional[torch.Tensor] = None,
                       delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
                       h0: Optional[torch.Tensor] = None,
                       dh_final: Optional[torch.Tensor] = None,
                       conv_w: Optional[torch.Tensor] = None,
                       conv_b: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       conv_state_in: Optional[torch.Tensor] = None,
                       checkpoints: Optional[torch.Tensor] = None) -> dict:
    """ssm_selective_scan_bwd: gradients of the scan (1 <= N <= 16).  `checkpoints` are
    the ones a selective_scan_fwd call with the same inputs wrote (else the backward
    recomputes them).

    Returns a dict with dx, ddelta (x's dtype), dA, dBm, dCm (float32) and, for the
    optional inputs given, dz, dDskip, ddelta_bias, dh0, dconv_w, dconv_b and
    dconv_state_in (x's dtype, the gradient of the conv state entering the sequence)."""
    a, dev = _scan_args(x, delta, A, Bm, Cm, Dskip, z, delta_bias, delta_softplus, conv_w, conv_b,
                        h0, torch.empty_like(x), None, conv_state_in=conv_state_in,
                        checkpoints=checkpoints)
    Bsz, L, D = x.shape
    N = A.shape[1]
    io = x.dtype
    _req(dy, "dy", (Bsz, L, D), io, dev)
    _opt(dh_final, "dh_final", (Bsz, D, N), torch.float32, dev)
    f32 = dict(device=dev, dtype=torch.float32)
    out = dict(dx=torch.empty_like(x), ddelta=torch.empty_like(x), dA=torch.empty(D, N, **f32),
               dBm=torch.empty(Bsz, L, N, **f32), dCm=torch.empty(Bsz, L, N, **f32))
    if z is not None:
        out["dz"] = torch.empty_like(x)
    if Dskip is not None:
        out["dDskip"] = torch.empty(D, **f32)
    if delta_softplus:
        out["ddelta_bias"] = torch.empty(D, **f32)
    if h0 is not None:
        out["dh0"] = torch.empty(Bsz, D, N, **f32)
    if conv_w is not None:
        out["dconv_w"] = torch.empty(D, a.conv_k, **f32)
        out["dconv_b"] = torch.empty(D, **f32)
    if conv_state_in is not None:
        out["dconv_state_in"] = torch.empty_like(conv_state_in)
    g = lambda k: _ptr(out.get(k))
    b = ScanBwdArgs(batch=Bsz, seqlen=L, dim=D, dstate=N, io_dtype=a.io_dtype,
                    delta_softplus=a.delta_softplus, conv_k=a.conv_k, x=a.x, delta=a.delta, Bm=a.Bm,
                    Cm=a.Cm, z=a.z, A=a.A, Dskip=a.Dskip, delta_bias=a.delta_bias, h0=a.h0,
                    conv_w=a.conv_w, conv_b=a.conv_b, dconv_w=g("dconv_w"), dconv_b=g("dconv_b"),
                    dy=_ptr(dy), dh_final=_ptr(dh_final), dx=g("dx"), ddelta=g("ddelta"),
                    dz=g("dz"), dA=g("dA"), dBm=g("dBm"), dCm=g("dCm"), dDskip=g("dDskip"),
                    ddelta_bias=g("ddelta_bias"), dh0=g("dh0"), conv_state_in=a.conv_state_in,
                    dconv_state_in=g("dconv_state_in"), checkpoints=_ptr(checkpoints))
    need = lib().ssm_selective_scan_bwd_workspace_size(ctypes.byref(b))
    if need == ctypes.c_size_t(-1).value:
        _check(lib().ssm_selective_scan_bwd(ctypes.byref(b), None), "ssm_selective_scan_bwd")
    if need > 0:
        ws = workspace if workspace is not None else _workspace(dev, need)
        if ws.device != dev or ws.numel() * ws.element_size() < need:
            raise ValueError("workspace must be a device tensor of >= %d bytes" % need)
        b.workspace = ws.data_ptr()
        b.workspace_bytes = ws.numel() * ws.element_size()
    _check(lib().ssm_selective_scan_bwd(ctypes.byref(b), _stream(dev)), "ssm_selective_scan_bwd")
    return out


class _SelectiveScanFn(torch.autograd.Function):
    """selective_scan as a torch autograd function: the forward writes the block
    checkpoints, the backward reads them (ssm_selective_scan_fwd / _bwd)."""

    @staticmethod
    def forward(ctx, x, delta, A, Bm, Cm, Dskip, z, delta_bias, h0, conv_w, conv_b, delta_softplus):
        ck = torch.empty(checkpoint_shape(x.shape[0], x.shape[1], x.shape[2]), device=x.device,
                         dtype=torch.float32)
        y, hf = selective_scan_fwd(x, delta, A, Bm, Cm, Dskip=Dskip, z=z, delta_bias=delta_bias,
                                   delta_softplus=delta_softplus, conv_w=conv_w, conv_b=conv_b, h0=h0,
                                   return_final_state=True, checkpoints=ck)
        ctx.save_for_backward(x, delta, A, Bm, Cm, Dskip, z, delta_bias, h0, conv_w, conv_b, ck)
        ctx.delta_softplus = delta_softplus
        return y, hf

    @staticmethod
    def backward(ctx, dy, dh_final):
        x, delta, A, Bm, Cm, Dskip, z, delta_bias, h0, conv_w, conv_b, ck = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros_like(x)
        g = selective_scan_bwd(x, delta, A, Bm, Cm, dy.contiguous(), Dskip=Dskip, z=z,
                               delta_bias=delta_bias, delta_softplus=ctx.delta_softplus, h0=h0,
                               dh_final=None if dh_final is None else dh_final.contiguous(),
                               conv_w=conv_w, conv_b=conv_b, checkpoints=ck)
        given = lambda t, k: g.get(k) if t is not None else None
        return (g["dx"], g["ddelta"], g["dA"], g["dBm"], g["dCm"], given(Dskip, "dDskip"), given(z, "dz"),
                given(delta_bias, "ddelta_bias"), given(h0, "dh0"), given(conv_w, "dconv_w"),
                given(conv_b, "dconv_b"), None)


def selective_scan(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor,
                   Cm: torch.Tensor, Dskip: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, delta_bias: Optional[torch.Tensor] = None,
                   delta_softplus: bool = False, h0: Optional[torch.Tensor] = None,
                   conv_w: Optional[torch.Tensor] = None, conv_b: Optional[torch.Tensor] = None):
    """The scan as a differentiable torch op (1 <= N <= 16): returns (y, h_final), and
    backward() runs ssm_selective_scan_bwd from the checkpoints the forward kept.  The
    gradients of B and C are computed in fp32 and cast to their dtype by autograd."""
    return _SelectiveScanFn.apply(x, delta, A, Bm, Cm, Dskip, z, delta_bias, h0, conv_w, conv_b,
                                  bool(delta_softplus))


class BlockPlan:
    """A plan of ssm_block_fwd for fixed sizes (owns the library's plan handle)."""

    def __init__(self, batch: int, seqlen: int, d_model: int, d_inner: int, dstate: int,
                 dt_rank: int, conv_k: int):
        self.dims = BlockDims(batch=batch, seqlen=seqlen, d_model=d_model, d_inner=d_inner,
                              dstate=dstate, dt_rank=dt_rank, conv_k=conv_k)
        self._h = _P()
        self._lib = lib()
        _check(self._lib.ssm_block_plan_create(ctypes.byref(self.dims), ctypes.byref(self._h)),
               "ssm_block_plan_create")
        self.workspace_bytes = int(self._lib.ssm_block_workspace_size(self._h))

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            self._lib.ssm_block_plan_destroy(self._h)
            self._h = _P()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_plan_cache = {}


def mamba_block_fwd(h: torch.Tensor, norm_w: torch.Tensor, w_in: torch.Tensor, conv_w: torch.Tensor,
                    conv_b: Optional[torch.Tensor], w_x: torch.Tensor, w_dt: torch.Tensor,
                    dt_bias: torch.Tensor, A: torch.Tensor, Dskip: Optional[torch.Tensor],
                    w_out: torch.Tensor, eps: float = 1e-5, out: Optional[torch.Tensor] = None,
                    plan: Optional[BlockPlan] = None, workspace: Optional[torch.Tensor] = None):
    """One Mamba block with its pre-norm residual (ssm_block_fwd): h (B, L, d_model) bf16 ->
    h + out_proj(S6(...) * silu(z)).  Weight shapes as in ssm_block_weights_t; `out` may be h."""
    if not isinstance(h, torch.Tensor) or h.dim() != 3 or h.device.type != "cuda":
        raise ValueError("h must be a (B, L, d_model) GPU tensor")
    dev = h.device
    Bsz, L, dm = h.shape
    if A.dim() != 2 or w_dt.dim() != 2 or conv_w.dim() != 2:
        raise ValueError("A, w_dt and conv_w must be 2-D")
    D, N = A.shape
    R = w_dt.shape[1]
    K = conv_w.shape[1]
    bf, f32 = torch.bfloat16, torch.float32
    _req(h, "h", (Bsz, L, dm), bf, dev)
    _req(norm_w, "norm_w", (dm,), f32, dev)
    _req(w_in, "w_in", (2 * D, dm), bf, dev)
    _req(conv_w, "conv_w", (D, K), f32, dev)
    _opt(conv_b, "conv_b", (D,), f32, dev)
    _req(w_x, "w_x", (R + 2 * N, D), bf, dev)
    _req(w_dt, "w_dt", (D, R), bf, dev)
    _req(dt_bias, "dt_bias", (D,), f32, dev)
    _req(A, "A", (D, N), f32, dev)
    _opt(Dskip, "Dskip", (D,), f32, dev)
    _req(w_out, "w_out", (dm, D), bf, dev)
    given = out
    if out is None:
        out = torch.empty_like(h)
    _req(out, "out", (Bsz, L, dm), bf, dev)
    if plan is None:
        key = (dev.index, Bsz, L, dm, D, N, R, K)
        plan = _plan_cache.get(key)
        if plan is None:
            with torch.cuda.device(dev):
                plan = BlockPlan(Bsz, L, dm, D, N, R, K)
            _plan_cache[key] = plan
    d = plan.dims
    if (d.batch, d.seqlen, d.d_model, d.d_inner, d.dstate, d.dt_rank, d.conv_k) != (Bsz, L, dm, D, N, R, K):
        raise ValueError("the plan was made for other sizes")
    if workspace is None:
        workspace = _workspace(dev, plan.workspace_bytes)
    wts = BlockWeights(norm_w=_ptr(norm_w), w_in=_ptr(w_in), conv_w=_ptr(conv_w), conv_b=_ptr(conv_b),
                       w_x=_ptr(w_x), w_dt=_ptr(w_dt), dt_bias=_ptr(dt_bias), A=_ptr(A),
                       Dskip=_ptr(Dskip), w_out=_ptr(w_out), norm_eps=float(eps))
    _check(lib().ssm_block_fwd(plan.handle, ctypes.byref(wts), _ptr(h), _ptr(out), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(dev)),
           "ssm_block_fwd")
    _changed(given)
    return out


def ssd_fwd(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, Cm: torch.Tensor,
            Dskip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
            delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
            h0: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
            h_final: Optional[torch.Tensor] = None, return_final_state: bool = False):
    """ssm_ssd_fwd: the SSD (Mamba-2) layer.  x, z: (B, L, H, P) and delta: (B, L, H), bf16
    (chunked on the matrix cores) or fp32 (the recurrent form); A, Dskip, delta_bias: (H,)
    fp32; Bm, Cm: (B, L, G, N) in x's dtype; h0, h_final: (B, H, P, N) fp32.
    Returns y, or (y, h_final) with return_final_state or h_final given."""
    if not isinstance(x, torch.Tensor) or x.dim() != 4 or x.device.type != "cuda":
        raise ValueError("x must be a (B, L, H, P) GPU tensor")
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != 4:
        raise ValueError("Bm must be (B, L, G, N)")
    dev = x.device
    Bsz, L, H, P = x.shape
    G, N = Bm.shape[2], Bm.shape[3]
    bf, f32 = x.dtype, torch.float32
    _io_code(bf)
    _req(x, "x", (Bsz, L, H, P), bf, dev)
    _req(delta, "delta", (Bsz, L, H), bf, dev)
    _req(A, "A", (H,), f32, dev)
    _req(Bm, "Bm", (Bsz, L, G, N), bf, dev)
    _req(Cm, "Cm", (Bsz, L, G, N), bf, dev)
    _opt(Dskip, "Dskip", (H,), f32, dev)
    _opt(z, "z", (Bsz, L, H, P), bf, dev)
    _opt(delta_bias, "delta_bias", (H,), f32, dev)
    _opt(h0, "h0", (Bsz, H, P, N), f32, dev)
    given = (y, h_final)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", (Bsz, L, H, P), bf, dev)
    if h_final is None and return_final_state:
        h_final = torch.empty(Bsz, H, P, N, device=dev, dtype=f32)
    _opt(h_final, "h_final", (Bsz, H, P, N), f32, dev)
    a = SsdArgs(batch=Bsz, seqlen=L, nheads=H, headdim=P, ngroups=G, dstate=N, io_dtype=_io_code(bf),
                delta_softplus=int(bool(delta_softplus)), x=_ptr(x), delta=_ptr(delta), A=_ptr(A),
                Bm=_ptr(Bm), Cm=_ptr(Cm), Dskip=_ptr(Dskip), z=_ptr(z), delta_bias=_ptr(delta_bias),
                h0=_ptr(h0), y=_ptr(y), h_final=_ptr(h_final), workspace=None, workspace_bytes=0)
    need = lib().ssm_ssd_workspace_size(ctypes.byref(a))
    if need == ctypes.c_size_t(-1).value:
        _check(lib().ssm_ssd_fwd(ctypes.byref(a), _stream(dev)), "ssm_ssd_fwd")  # reports the error
    if need:
        ws = _workspace(dev, need)
        a.workspace = ws.data_ptr()
        a.workspace_bytes = ws.numel()
    _check(lib().ssm_ssd_fwd(ctypes.byref(a), _stream(dev)), "ssm_ssd_fwd")
    _changed(*given)
    return (y, h_final) if h_final is not None else y


def ssd_step(state: torch.Tensor, x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor,
             Bm: torch.Tensor, Cm: torch.Tensor, Dskip: Optional[torch.Tensor] = None,
             z: Optional[torch.Tensor] = None, delta_bias: Optional[torch.Tensor] = None,
             delta_softplus: bool = False, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ssm_ssd_step: one decode step of the SSD layer; advances `state` (B, H, P, N) fp32 in
    place.  x, z: (B, H, P) bf16; delta: (B, H) bf16; A, Dskip, delta_bias: (H,) fp32;
    Bm, Cm: (B, G, N) bf16.  Returns y (B, H, P) bf16."""
    a, out = ssd_step_args(state, x, delta, A, Bm, Cm, Dskip, z, delta_bias, delta_softplus, y)
    _check(lib().ssm_ssd_step(ctypes.byref(a), _stream(state.device)), "ssm_ssd_step")
    _changed(state, y)
    return out


def ssd_step_args(state, x, delta, A, Bm, Cm, Dskip=None, z=None, delta_bias=None,
                  delta_softplus=False, y=None):
    """The checked ssm_ssd_step_args_t of an ssd_step call, and its y (allocated when not
    given), for callers that launch the same step repeatedly through lib().ssm_ssd_step.
    The tensors must outlive the struct."""
    if not isinstance(state, torch.Tensor) or state.dim() != 4 or state.device.type != "cuda":
        raise ValueError("state must be a (B, H, P, N) GPU tensor")
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != 3:
        raise ValueError("Bm must be (B, G, N)")
    dev = state.device
    Bsz, H, P, N = state.shape
    G = Bm.shape[1]
    bf, f32 = torch.bfloat16, torch.float32
    _req(state, "state", (Bsz, H, P, N), f32, dev)
    _req(x, "x", (Bsz, H, P), bf, dev)
    _req(delta, "delta", (Bsz, H), bf, dev)
    _req(A, "A", (H,), f32, dev)
    _req(Bm, "Bm", (Bsz, G, N), bf, dev)
    _req(Cm, "Cm", (Bsz, G, N), bf, dev)
    _opt(Dskip, "Dskip", (H,), f32, dev)
    _opt(z, "z", (Bsz, H, P), bf, dev)
    _opt(delta_bias, "delta_bias", (H,), f32, dev)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", (Bsz, H, P), bf, dev)
    a = SsdStepArgs(batch=Bsz, nheads=H, headdim=P, ngroups=G, dstate=N, io_dtype=SSM_BF16,
                    delta_softplus=int(bool(delta_softplus)), state=_ptr(state), x=_ptr(x),
                    delta=_ptr(delta), A=_ptr(A), Bm=_ptr(Bm), Cm=_ptr(Cm), Dskip=_ptr(Dskip),
                    z=_ptr(z), delta_bias=_ptr(delta_bias), y=_ptr(y))
    return a, y


# ------------------------------------------------------------------ gated linear recurrence
GATE_MODES = {"decay": 0, "sigmoid": 1, "rate": 2}  # ssm_gate_mode_t
GATED_BLOCK = 128  # SSM_GATED_BLOCK
_NO_SIZE = ctypes.c_size_t(-1).value


def gated_checkpoint_shape(batch: int, seqlen: int, dim: int) -> tuple:
    """Shape of the fp32 checkpoint tensor of gated_scan_fwd: the state entering every
    GATED_BLOCK-step block, (ceil(L / GATED_BLOCK), B, D)."""
    return ((seqlen + GATED_BLOCK - 1) // GATED_BLOCK, batch, dim)


# The calls below serve single decode tokens, where the marshalling itself is what a step costs:
# an argument that is as expected passes one expression, and only one that is not goes to the
# checks that name what is wrong.
_raw_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream(i).cuda_stream


def _arg(t, name, shape, dtype, device):
    """Address of an optional tensor argument (None: not given)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device.index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass  # not a tensor: named by the check below
    return _opt(t, name, shape, dtype, device).data_ptr()


def _need(t, name, shape, dtype, device):
    """Address of a required tensor argument."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device.index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _req(t, name, shape, dtype, device).data_ptr()


class _Scratch(threading.local):
    """Cached workspaces of the calling thread.  Two threads may use the same stream at once, and
    the launches of their calls then alternate on it: a workspace they shared would be emptied by
    one call between the other's launches."""

    def __init__(self):
        self.of = {}


_scratch = _Scratch()


def _run(name: str, args, dev: torch.device, size_fn=None, workspace: Optional[torch.Tensor] = None):
    """ssm_<name>(args) on torch's current stream of `dev`, with that device current and with a
    workspace where size_fn(args) asks for one: a cached one of this thread and stream, or in a
    graph capture one of the graph's own.  Invalid sizes are reported by the call itself, which
    checks its arguments before anything is launched."""
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _run(name, args, dev, size_fn, workspace)
    L = lib()
    ref = ctypes.byref(args)
    stream = _raw_stream(dev.index)
    if size_fn is not None:
        need = getattr(L, size_fn)(ref)
        if need != _NO_SIZE and need > 0:
            if workspace is None:
                key = (dev.index, stream)
                workspace = _scratch.of.get(key)
                if torch.cuda.is_current_stream_capturing():
                    workspace = torch.empty(need, dtype=torch.uint8, device=dev)
                elif workspace is None or workspace.numel() < need:
                    workspace = _scratch.of[key] = torch.empty(max(need, 1 << 20), dtype=torch.uint8, device=dev)
            have = workspace.numel() * workspace.element_size()
            if workspace.device != dev or not workspace.is_contiguous() or have < need:
                raise ValueError("workspace must be a contiguous tensor on %s of >= %d bytes" % (dev, need))
            args.workspace = workspace.data_ptr()
            args.workspace_bytes = have
    status = getattr(L, name)(ref, stream)
    if status != SSM_OK:
        _check(status, name)


def _gpu(t, name: str, dims: int, shape: str) -> torch.device:
    if not isinstance(t, torch.Tensor) or t.dim() != dims or t.device.type != "cuda":
        raise ValueError("%s must be a %s GPU tensor" % (name, shape))
    return t.device


def _gates(a, x, gate, mode, A, in_gate, gate_bias, in_bias, dev):
    """Check the gate inputs against x's shape and put them into `a`."""
    code = GATE_MODES.get(mode)
    if code is None:
        raise ValueError("mode must be one of %s, got %r" % (", ".join(GATE_MODES), mode))
    shape, io = x.shape, x.dtype
    a.io_dtype, a.mode = _io_code(io), code
    a.x = _need(x, "x", shape, io, dev)
    a.gate = _need(gate, "gate", shape, io, dev)
    if in_gate is not None:
        a.in_gate = _arg(in_gate, "in_gate", shape, io, dev)
    per_channel, f32 = (shape[-1],), torch.float32
    if A is not None:
        a.A = _arg(A, "A", per_channel, f32, dev)
    if gate_bias is not None:
        a.gate_bias = _arg(gate_bias, "gate_bias", per_channel, f32, dev)
    if in_bias is not None:
        a.in_bias = _arg(in_bias, "in_bias", per_channel, f32, dev)


def _resets(reset, shape, dev):
    """A reset mask as the library's bytes: uint8, or bool (the same bytes, 0 or 1)."""
    if reset is None:
        return None
    if isinstance(reset, torch.Tensor) and reset.dtype == torch.bool:
        reset = reset.view(torch.uint8)
    return _arg(reset, "reset", shape, torch.uint8, dev)


def gated_scan_fwd(x: torch.Tensor, gate: torch.Tensor, mode: str = "rate",
                   A: Optional[torch.Tensor] = None, in_gate: Optional[torch.Tensor] = None,
                   gate_bias: Optional[torch.Tensor] = None, in_bias: Optional[torch.Tensor] = None,
                   reset: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                   return_final_state: bool = False, y: Optional[torch.Tensor] = None,
                   h_final: Optional[torch.Tensor] = None, checkpoints: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """ssm_gated_scan_fwd: h_t = a_t h_{t-1} + b_t per channel.  x, gate, in_gate: (B, L, D) bf16
    or fp32; A, gate_bias, in_bias: (D,) fp32; reset: (B, L) uint8 or bool; h0: (B, D) fp32.

    mode "decay": a = gate, b = x.  "sigmoid": s = sigmoid(gate + gate_bias), a = 1 - s, b = s x.
    "rate": a = exp(A sigmoid(gate + gate_bias)), b = sqrt(1 - a^2) sigmoid(in_gate + in_bias) x.
    Decays outside [-1, 1] (A > 0) are computed as long as products of up to 256 of them stay below
    2^127; where A > 0 the input's weight is 0.

    Returns (y, h_final or None).  A float32 tensor `checkpoints` of gated_checkpoint_shape(B, L, D)
    also receives the state entering every GATED_BLOCK-step block, for gated_scan_bwd."""
    dev = _gpu(x, "x", 3, "(B, L, D)")
    B, L, D = x.shape
    f32 = torch.float32
    given = (y, h_final, checkpoints)
    a = GatedScanArgs(batch=B, seqlen=L, dim=D)
    _gates(a, x, gate, mode, A, in_gate, gate_bias, in_bias, dev)
    if reset is not None:
        a.reset = _resets(reset, (B, L), dev)
    if h0 is not None:
        a.h0 = _arg(h0, "h0", (B, D), f32, dev)
    if y is None:
        y = torch.empty_like(x)
        a.y = y.data_ptr()
    else:
        a.y = _need(y, "y", (B, L, D), x.dtype, dev)
    if h_final is not None:
        a.h_final = _arg(h_final, "h_final", (B, D), f32, dev)
    elif return_final_state:
        h_final = torch.empty((B, D), device=dev, dtype=f32)
        a.h_final = h_final.data_ptr()
    if checkpoints is not None:
        a.checkpoints = _arg(checkpoints, "checkpoints", gated_checkpoint_shape(B, L, D), f32, dev)
    _run("ssm_gated_scan_fwd", a, dev, "ssm_gated_scan_workspace_size", workspace)
    _changed(*given)
    return y, h_final


def gated_scan_bwd(x: torch.Tensor, gate: torch.Tensor, dy: torch.Tensor, mode: str = "rate",
                   A: Optional[torch.Tensor] = None, in_gate: Optional[torch.Tensor] = None,
                   gate_bias: Optional[torch.Tensor] = None, in_bias: Optional[torch.Tensor] = None,
                   reset: Optional[torch.Tensor] = None, h0: Optional[torch.Tensor] = None,
                   dh_final: Optional[torch.Tensor] = None, checkpoints: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> dict:
    """ssm_gated_scan_bwd: the gradients of gated_scan_fwd for dL/dy = dy, dL/dh_final = dh_final.
    `checkpoints` are the ones a gated_scan_fwd call with the same inputs wrote (else the backward
    recomputes them).

    Returns a dict with dx, dgate (x's dtype) and, for the inputs given, din_gate (x's dtype), dA,
    dgate_bias, din_bias, dh0 (float32)."""
    dev = _gpu(x, "x", 3, "(B, L, D)")
    B, L, D = x.shape
    f32 = torch.float32
    a = GatedScanBwdArgs(batch=B, seqlen=L, dim=D)
    _gates(a, x, gate, mode, A, in_gate, gate_bias, in_bias, dev)
    a.dy = _need(dy, "dy", (B, L, D), x.dtype, dev)
    out = dict(dx=torch.empty_like(x), dgate=torch.empty_like(x))
    if in_gate is not None:
        out["din_gate"] = torch.empty_like(x)
    if mode == "rate":
        out["dA"] = torch.empty(D, device=dev, dtype=f32) if A is None else torch.empty_like(A)
    if gate_bias is not None:
        out["dgate_bias"] = torch.empty_like(gate_bias)
    if in_bias is not None:
        out["din_bias"] = torch.empty_like(in_bias)
    if reset is not None:
        a.reset = _resets(reset, (B, L), dev)
    if h0 is not None:
        a.h0 = _arg(h0, "h0", (B, D), f32, dev)
        out["dh0"] = torch.empty_like(h0)
    if dh_final is not None:
        a.dh_final = _arg(dh_final, "dh_final", (B, D), f32, dev)
    if checkpoints is not None:
        a.checkpoints = _arg(checkpoints, "checkpoints", gated_checkpoint_shape(B, L, D), f32, dev)
    for name, t in out.items():
        setattr(a, name, t.data_ptr())
    _run("ssm_gated_scan_bwd", a, dev, "ssm_gated_scan_bwd_workspace_size", workspace)
    return out


def gated_scan_step(state: torch.Tensor, x: torch.Tensor, gate: torch.Tensor, mode: str = "rate",
                    A: Optional[torch.Tensor] = None, in_gate: Optional[torch.Tensor] = None,
                    gate_bias: Optional[torch.Tensor] = None, in_bias: Optional[torch.Tensor] = None,
                    reset: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ssm_gated_scan_step: one decode token; advances `state` (B, D) fp32 in place and returns
    y (B, D).  x, gate, in_gate: (B, D) bf16 or fp32; reset: (B,) uint8 or bool, rows whose state
    is taken as 0 (a new sequence); the rest as in gated_scan_fwd."""
    a, out = gated_scan_step_args(state, x, gate, mode, A, in_gate, gate_bias, in_bias, reset, y)
    _run("ssm_gated_scan_step", a, state.device)
    _changed(state, y)
    return out


def gated_scan_step_args(state, x, gate, mode="rate", A=None, in_gate=None, gate_bias=None, in_bias=None,
                         reset=None, y=None):
    """The checked ssm_gated_step_args_t of a gated_scan_step call, and its y (allocated when not
    given), for callers that launch the same step repeatedly through lib().ssm_gated_scan_step.
    The tensors must outlive the struct; autograd does not see what such launches write."""
    dev = _gpu(state, "state", 2, "(B, D) float32")
    shape = state.shape
    if not isinstance(x, torch.Tensor) or x.shape != shape:
        raise ValueError("x must be a %s tensor like the state" % (tuple(shape),))
    a = GatedStepArgs()
    a.batch, a.dim = shape
    a.state = _need(state, "state", shape, torch.float32, dev)
    _gates(a, x, gate, mode, A, in_gate, gate_bias, in_bias, dev)
    if reset is not None:
        a.reset = _resets(reset, (shape[0],), dev)
    if y is None:
        y = torch.empty_like(x)
        a.y = y.data_ptr()
    else:
        a.y = _need(y, "y", shape, x.dtype, dev)
    return a, y


class _GatedScanFn(torch.autograd.Function):
    """gated_scan as a torch autograd function: the forward writes the checkpoints, the
    backward reads them (ssm_gated_scan_fwd / _bwd)."""

    @staticmethod
    def forward(ctx, x, gate, A, in_gate, gate_bias, in_bias, h0, mode, reset):
        _gpu(x, "x", 3, "(B, L, D)")
        ck = None
        if any(ctx.needs_input_grad):
            ck = torch.empty(gated_checkpoint_shape(*x.shape), device=x.device, dtype=torch.float32)
        y, hf = gated_scan_fwd(x, gate, mode, A=A, in_gate=in_gate, gate_bias=gate_bias, in_bias=in_bias,
                               reset=reset, h0=h0, return_final_state=True, checkpoints=ck)
        ctx.save_for_backward(x, gate, A, in_gate, gate_bias, in_bias, h0, reset, ck)
        ctx.mode = mode
        return y, hf

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh_final):
        x, gate, A, in_gate, gate_bias, in_bias, h0, reset, ck = ctx.saved_tensors
        g = gated_scan_bwd(x, gate, dy.contiguous(), ctx.mode, A=A, in_gate=in_gate, gate_bias=gate_bias,
                           in_bias=in_bias, reset=reset, h0=h0, dh_final=dh_final.contiguous(), checkpoints=ck)
        return (g["dx"], g["dgate"], g.get("dA"), g.get("din_gate"), g.get("dgate_bias"), g.get("din_bias"),
                g.get("dh0"), None, None)


def gated_scan(x: torch.Tensor, gate: torch.Tensor, mode: str = "rate", A: Optional[torch.Tensor] = None,
               in_gate: Optional[torch.Tensor] = None, gate_bias: Optional[torch.Tensor] = None,
               in_bias: Optional[torch.Tensor] = None, reset: Optional[torch.Tensor] = None,
               h0: Optional[torch.Tensor] = None):
    """The gated recurrence as a differentiable torch op (arguments as in gated_scan_fwd): returns
    (y, h_final), and backward() runs ssm_gated_scan_bwd from the checkpoints the forward kept.

    To capture a backward() into a graph, capture it on leaves that no earlier, still living
    autograd graph has used (torch's own rule for gradient accumulation under capture)."""
    return _GatedScanFn.apply(x, gate, A, in_gate, gate_bias, in_bias, h0, mode, reset)


# ----------------------------------------------------------------------------- fused norms
def _add_norm(a, x, w, residual, scale, post_w, eps, shape, dev):
    D, io, f32 = shape[-1], x.dtype, torch.float32
    a.rows, a.dim, a.eps = x.numel() // D, D, float(eps)
    a.io_dtype = a.res_dtype = _io_code(io)
    a.x = _need(x, "x", shape, io, dev)
    a.w = _need(w, "w", (D,), f32, dev)
    if residual is not None:
        if not isinstance(residual, torch.Tensor):
            raise TypeError("residual must be a torch.Tensor")
        if residual.dtype is not io:
            a.res_dtype = _io_code(residual.dtype)
        a.residual = _arg(residual, "residual", shape, residual.dtype, dev)
    if scale is not None:
        a.scale = _arg(scale, "scale", (D,), f32, dev)
    if post_w is not None:
        a.post_w = _arg(post_w, "post_w", (D,), f32, dev)


def _shape_of(x):
    if not isinstance(x, torch.Tensor) or x.dim() < 1 or x.device.type != "cuda" or x.shape[-1] < 1:
        raise ValueError("x must be a (..., D) GPU tensor")
    return x.shape


def add_rmsnorm_fwd(x: torch.Tensor, w: torch.Tensor, residual: Optional[torch.Tensor] = None,
                    scale: Optional[torch.Tensor] = None, post_w: Optional[torch.Tensor] = None,
                    eps: float = 1e-5, y: Optional[torch.Tensor] = None,
                    res_out: Optional[torch.Tensor] = None):
    """ssm_add_rmsnorm_fwd: u = x, or RMSNorm(x) * post_w; res_out = residual + scale * u;
    y = RMSNorm(res_out) * w.  x: (..., D) bf16 or fp32; residual: x's shape, bf16 or fp32 (the
    residual stream keeps its dtype; without one res_out has x's); w, scale, post_w: (D,) fp32.
    `res_out` may be `residual` (updated in place).  Returns (y, res_out)."""
    shape = _shape_of(x)
    dev = x.device
    a = AddNormArgs()
    _add_norm(a, x, w, residual, scale, post_w, eps, shape, dev)
    stream = x if residual is None else residual
    given = (y, res_out)
    if y is None:
        y = torch.empty_like(x)
        a.y = y.data_ptr()
    else:
        a.y = _need(y, "y", shape, x.dtype, dev)
    if res_out is None:
        res_out = torch.empty_like(stream)
        a.res_out = res_out.data_ptr()
    else:
        a.res_out = _need(res_out, "res_out", shape, stream.dtype, dev)
    _run("ssm_add_rmsnorm_fwd", a, dev)
    _changed(*given)
    return y, res_out


def add_rmsnorm_bwd(x: torch.Tensor, w: torch.Tensor, residual: Optional[torch.Tensor], dy: torch.Tensor,
                    dres_out: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                    post_w: Optional[torch.Tensor] = None, eps: float = 1e-5,
                    workspace: Optional[torch.Tensor] = None) -> dict:
    """ssm_add_rmsnorm_bwd: the gradients of add_rmsnorm_fwd on the same x and residual (the
    residual before an in-place update) for dL/dy = dy and dL/dres_out = dres_out.

    Returns a dict with dx (x's dtype), dw and, for the inputs given, dresidual (residual's dtype),
    dscale, dpost_w (float32)."""
    shape = _shape_of(x)
    dev = x.device
    a = AddNormBwdArgs()
    _add_norm(a, x, w, residual, scale, post_w, eps, shape, dev)
    a.dy = _need(dy, "dy", shape, x.dtype, dev)
    if dres_out is not None:
        a.dres_out = _arg(dres_out, "dres_out", shape, x.dtype if residual is None else residual.dtype, dev)
    out = dict(dx=torch.empty_like(x), dw=torch.empty_like(w))
    if residual is not None:
        out["dresidual"] = torch.empty_like(residual)
    if scale is not None:
        out["dscale"] = torch.empty_like(w)
    if post_w is not None:
        out["dpost_w"] = torch.empty_like(w)
    for name, t in out.items():
        setattr(a, name, t.data_ptr())
    _run("ssm_add_rmsnorm_bwd", a, dev, "ssm_add_rmsnorm_bwd_workspace_size", workspace)
    return out


class _AddNormFn(torch.autograd.Function):
    """add_rmsnorm as a torch autograd function (ssm_add_rmsnorm_fwd / _bwd)."""

    @staticmethod
    def forward(ctx, x, w, residual, scale, post_w, eps):
        y, r = add_rmsnorm_fwd(x, w, residual, scale=scale, post_w=post_w, eps=eps)
        ctx.save_for_backward(x, w, residual, scale, post_w)
        ctx.eps = eps
        return y, r

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dres_out):
        x, w, residual, scale, post_w = ctx.saved_tensors
        g = add_rmsnorm_bwd(x, w, residual, dy.contiguous(), dres_out.contiguous(), scale=scale, post_w=post_w,
                            eps=ctx.eps)
        return g["dx"], g["dw"], g.get("dresidual"), g.get("dscale"), g.get("dpost_w"), None


def add_rmsnorm(x: torch.Tensor, w: torch.Tensor, residual: Optional[torch.Tensor] = None,
                scale: Optional[torch.Tensor] = None, post_w: Optional[torch.Tensor] = None,
                eps: float = 1e-5):
    """The fused residual sum and norm as a differentiable torch op (arguments as in
    add_rmsnorm_fwd): returns (y, res_out).  A captured backward(): as with gated_scan."""
    return _AddNormFn.apply(x, w, residual, scale, post_w, eps)


def _gated_norm(a, x, z, w, groups, gate_first, eps, shape, dev):
    D = shape[-1]
    if int(groups) != groups:
        raise ValueError("groups must be a whole number, got %r" % (groups,))
    a.rows, a.dim, a.groups, a.eps = x.numel() // D, D, int(groups), float(eps)
    a.io_dtype, a.gate_first = _io_code(x.dtype), int(bool(gate_first))
    a.x = _need(x, "x", shape, x.dtype, dev)
    a.z = _need(z, "z", shape, x.dtype, dev)
    a.w = _need(w, "w", (D,), torch.float32, dev)


def gated_rmsnorm_fwd(x: torch.Tensor, z: torch.Tensor, w: torch.Tensor, groups: int = 1,
                      gate_first: bool = True, eps: float = 1e-5,
                      y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """ssm_gated_rmsnorm_fwd: with gate_first RMSNorm(x * silu(z)) * w, else RMSNorm(x) * w * silu(z),
    the mean square over each of `groups` groups of D / groups consecutive channels.  x, z: (..., D)
    bf16 or fp32; w: (D,) fp32.  `y` may be x or z."""
    shape = _shape_of(x)
    dev = x.device
    a = GatedNormArgs()
    _gated_norm(a, x, z, w, groups, gate_first, eps, shape, dev)
    out = torch.empty_like(x) if y is None else y
    a.y = out.data_ptr() if y is None else _need(y, "y", shape, x.dtype, dev)
    _run("ssm_gated_rmsnorm_fwd", a, dev)
    _changed(y)
    return out


def gated_rmsnorm_bwd(x: torch.Tensor, z: torch.Tensor, w: torch.Tensor, dy: torch.Tensor, groups: int = 1,
                      gate_first: bool = True, eps: float = 1e-5,
                      workspace: Optional[torch.Tensor] = None) -> dict:
    """ssm_gated_rmsnorm_bwd: the gradients of gated_rmsnorm_fwd for dL/dy = dy.  Returns a dict
    with dx, dz (x's dtype) and dw (float32)."""
    shape = _shape_of(x)
    dev = x.device
    a = GatedNormBwdArgs()
    _gated_norm(a, x, z, w, groups, gate_first, eps, shape, dev)
    a.dy = _need(dy, "dy", shape, x.dtype, dev)
    out = dict(dx=torch.empty_like(x), dz=torch.empty_like(z), dw=torch.empty_like(w))
    for name, t in out.items():
        setattr(a, name, t.data_ptr())
    _run("ssm_gated_rmsnorm_bwd", a, dev, "ssm_gated_rmsnorm_bwd_workspace_size", workspace)
    return out


class _GatedNormFn(torch.autograd.Function):
    """gated_rmsnorm as a torch autograd function (ssm_gated_rmsnorm_fwd / _bwd)."""

    @staticmethod
    def forward(ctx, x, z, w, groups, gate_first, eps):
        ctx.save_for_backward(x, z, w)
        ctx.opts = dict(groups=groups, gate_first=gate_first, eps=eps)
        return gated_rmsnorm_fwd(x, z, w, **ctx.opts)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, z, w = ctx.saved_tensors
        g = gated_rmsnorm_bwd(x, z, w, dy.contiguous(), **ctx.opts)
        return g["dx"], g["dz"], g["dw"], None, None, None


def gated_rmsnorm(x: torch.Tensor, z: torch.Tensor, w: torch.Tensor, groups: int = 1, gate_first: bool = True,
                  eps: float = 1e-5) -> torch.Tensor:
    """The gated norm as a differentiable torch op (arguments as in gated_rmsnorm_fwd).  A captured
    backward(): as with gated_scan."""
    return _GatedNormFn.apply(x, z, w, groups, gate_first, eps)
