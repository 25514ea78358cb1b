// ssm_internal.h -- host-side interface between the argument-checking C ABI
// (ssm_api.cpp) and the kernel launchers (*.hip).  Launchers assume their
// arguments were validated: sizes in range, required pointers non-NULL,
// outputs not aliasing inputs, workspace large enough.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ssm.h"

namespace ssm {

// Scan: bytes of workspace the chosen launch plan needs (0 if none).
size_t scan_workspace_bytes(const ssm_scan_args_t &a);
// Scan: enqueue the kernels.  a.batch, a.seqlen > 0.
hipError_t launch_scan_fwd(const ssm_scan_args_t &a, hipStream_t stream);
// Scan checkpoints for the backward: the state entering every 16-step block,
// [ceil(L / 16)][B][D][16] fp32 at `ckpt` (a.dstate == 16), from a.x, a.delta,
// a.A, a.Bm, a.h0, the delta bias/softplus and the conv prologue; no outputs
// (a.y, a.z, a.Dskip, a.h_final and a.workspace are not used).  a.batch, a.seqlen > 0.
hipError_t launch_scan_ckpt(const ssm_scan_args_t &a, float *ckpt, hipStream_t stream);

// Device address of the no-allocation scan's scratch array
// (SSM_NOALLOC_SCRATCH_BYTES, 256-aligned) on the device of `stream`.
hipError_t noalloc_scratch(hipStream_t stream, void **out);

// Standalone conv1d + SiLU.  B, L > 0.
hipError_t launch_conv1d_silu(int64_t B, int64_t L, int64_t D, int K, int io_dtype,
                              const void *x, const float *w, const float *bias, void *u,
                              hipStream_t stream);

// Decode step.  a.batch > 0.
hipError_t launch_state_update(const ssm_state_update_args_t &a, hipStream_t stream);

// Scan backward: workspace bytes and launch (a.batch > 0; a.seqlen may be 0).
size_t scan_bwd_workspace_bytes(const ssm_scan_bwd_args_t &a);
hipError_t launch_scan_bwd(const ssm_scan_bwd_args_t &a, hipStream_t stream);

// Mamba block (block.hip).
ssm_status_t block_plan_create(const ssm_block_dims_t &d, ssm_block_plan **out);
void block_plan_destroy(ssm_block_plan *p);
size_t block_workspace_bytes(const ssm_block_plan &p);
const ssm_block_dims_t &block_dims(const ssm_block_plan &p);
hipError_t launch_block_fwd(const ssm_block_plan &p, const ssm_block_weights_t &w, const void *h_in, void *h_out,
                            void *workspace, hipStream_t stream);

// SSD (Mamba-2) layer (ssd.hip).  a.batch > 0; sizes checked by ssd_supported.
bool ssd_supported(int64_t headdim, int64_t dstate);
size_t ssd_workspace_bytes(const ssm_ssd_args_t &a);
bool ssd_step_supported(int64_t dstate);
hipError_t launch_ssd_step(const ssm_ssd_step_args_t &a, hipStream_t stream);
hipError_t launch_ssd_fwd(const ssm_ssd_args_t &a, hipStream_t stream);

// Gated recurrence (gated_scan.hip, gated_scan_bwd.hip).  Forward and backward take
// batch, seqlen > 0; the step batch > 0.
size_t gated_scan_workspace_bytes(const ssm_gated_scan_args_t &a);
hipError_t launch_gated_scan_fwd(const ssm_gated_scan_args_t &a, hipStream_t stream);
hipError_t launch_gated_step(const ssm_gated_step_args_t &a, hipStream_t stream);
size_t gated_scan_bwd_workspace_bytes(const ssm_gated_scan_bwd_args_t &a);
hipError_t launch_gated_scan_bwd(const ssm_gated_scan_bwd_args_t &a, hipStream_t stream);
// out[i] = in ? in[i] : 0 for i < n (the state of an empty recurrence, the gradients of none).
hipError_t launch_copy_or_zero(float *out, const float *in, int64_t n, hipStream_t stream);

// out[k][d] = sum over i < n of part[k][i][d] for k < K <= 3 (out[k] may be NULL: not formed), added in a
// fixed order; scratch of column_sums_scratch_bytes (colsum.hip).  n >= 1.
size_t column_sums_scratch_bytes(int64_t n, int64_t D, int K);
hipError_t launch_column_sums(const float *part, int64_t n, int64_t D, int K, float *const out[], float *scratch,
                              hipStream_t stream);

// Fused norms (add_norm.hip, gated_norm.hip), rows > 0.
hipError_t launch_add_norm_fwd(const ssm_add_norm_args_t &a, hipStream_t stream);
size_t add_norm_bwd_workspace_bytes(const ssm_add_norm_bwd_args_t &a);
hipError_t launch_add_norm_bwd(const ssm_add_norm_bwd_args_t &a, hipStream_t stream);
hipError_t launch_gated_norm_fwd(const ssm_gated_norm_args_t &a, hipStream_t stream);
size_t gated_norm_bwd_workspace_bytes(const ssm_gated_norm_bwd_args_t &a);
hipError_t launch_gated_norm_bwd(const ssm_gated_norm_bwd_args_t &a, hipStream_t stream);

// Gated delta rule (gated_delta.hip, gated_delta_bwd.hip): batch, seqlen > 0; the step batch > 0.
size_t gated_delta_workspace_bytes(const ssm_gated_delta_args_t &a);
hipError_t launch_gated_delta_fwd(const ssm_gated_delta_args_t &a, hipStream_t stream);
size_t gated_delta_bwd_workspace_bytes(const ssm_gated_delta_bwd_args_t &a);
hipError_t launch_gated_delta_bwd(const ssm_gated_delta_bwd_args_t &a, hipStream_t stream);
hipError_t launch_gated_delta_step(const ssm_gated_delta_step_args_t &a, hipStream_t stream);

// e4m3 with block scales (quant_fp8.hip, matmul_fp8.hip): rows, m > 0.
hipError_t launch_quantize_fp8(const ssm_quantize_fp8_args_t &a, hipStream_t stream);
hipError_t launch_add_norm_fp8(const ssm_add_norm_fp8_args_t &a, hipStream_t stream);
hipError_t launch_matmul_fp8(const ssm_matmul_fp8_args_t &a, hipStream_t stream);

// Copy or zero-fill the final state for an empty (L == 0) scan.
hipError_t launch_empty_scan_state(const ssm_scan_args_t &a, hipStream_t stream);

}  // namespace ssm
