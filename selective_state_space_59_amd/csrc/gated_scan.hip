// gated_scan.hip -- the gated linear recurrence h_t = a_t h_{t-1} + b_t, forward and
// decode step, on gfx950 (gated_device.h has the gates).
//
// One thread per (batch row, channel), sequential in time: the plain form.
#include "gated_device.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

template <typename IO, int MODE, bool IG>
__global__ __launch_bounds__(64) void gated_scan_kernel(ssm_gated_scan_args_t a) {
    const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
    if (d >= a.dim) return;
    GateChannel c = {a.A ? a.A[d] : 0.0f, a.gate_bias ? a.gate_bias[d] : 0.0f, a.in_bias ? a.in_bias[d] : 0.0f};
    float h = a.h0 ? a.h0[b * a.dim + d] : 0.0f;
    for (int64_t t = 0; t < a.seqlen; ++t) {
        const int64_t i = (b * a.seqlen + t) * a.dim + d;
        if (a.checkpoints && t % SSM_GATED_BLOCK == 0)
            a.checkpoints[((t / SSM_GATED_BLOCK) * a.batch + b) * a.dim + d] = h;
        float at, bt;
        gate_step<MODE, IG>(load_io<IO>(a.x, i), load_io<IO>(a.gate, i), IG ? load_io<IO>(a.in_gate, i) : 0.0f, c, at,
                            bt);
        const bool cut = a.reset && a.reset[b * a.seqlen + t];
        h = cut ? bt : __builtin_fmaf(at, h, bt);
        store_io<IO>(a.y, i, h);
    }
    if (a.h_final) a.h_final[b * a.dim + d] = h;
}

template <typename IO, int MODE, bool IG>
__global__ __launch_bounds__(64) void gated_step_kernel(ssm_gated_step_args_t a) {
    const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
    if (d >= a.dim) return;
    GateChannel c = {a.A ? a.A[d] : 0.0f, a.gate_bias ? a.gate_bias[d] : 0.0f, a.in_bias ? a.in_bias[d] : 0.0f};
    const int64_t i = b * a.dim + d;
    float at, bt;
    gate_step<MODE, IG>(load_io<IO>(a.x, i), load_io<IO>(a.gate, i), IG ? load_io<IO>(a.in_gate, i) : 0.0f, c, at, bt);
    const float h = a.reset && a.reset[b] ? bt : __builtin_fmaf(at, a.state[i], bt);
    a.state[i] = h;
    store_io<IO>(a.y, i, h);
}

__global__ __launch_bounds__(256) void copy_or_zero_kernel(float *out, const float *in, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) out[i] = in ? in[i] : 0.0f;
}

}  // namespace

size_t gated_scan_workspace_bytes(const ssm_gated_scan_args_t &) { return 0; }

hipError_t launch_gated_scan_fwd(const ssm_gated_scan_args_t &a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.dim + 63) / 64), (unsigned)a.batch);
    gate_dispatch(a.io_dtype, a.mode, a.in_gate != nullptr, [&](auto io, auto mode, auto ig) {
        gated_scan_kernel<decltype(io), decltype(mode)::value, decltype(ig)::value><<<grid, 64, 0, stream>>>(a);
    });
    return hipGetLastError();
}

hipError_t launch_gated_step(const ssm_gated_step_args_t &a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.dim + 63) / 64), (unsigned)a.batch);
    gate_dispatch(a.io_dtype, a.mode, a.in_gate != nullptr, [&](auto io, auto mode, auto ig) {
        gated_step_kernel<decltype(io), decltype(mode)::value, decltype(ig)::value><<<grid, 64, 0, stream>>>(a);
    });
    return hipGetLastError();
}

hipError_t launch_copy_or_zero(float *out, const float *in, int64_t n, hipStream_t stream) {
    copy_or_zero_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(out, in, n);
    return hipGetLastError();
}

}  // namespace ssm
