// gated_scan_bwd.hip -- gradients of the gated linear recurrence on gfx950.
//
//   lambda_t = dy_t + mu_{t+1},  mu_t = a_t lambda_t (0 at a reset),  mu_L = dh_final
//   da_t = lambda_t h_{t-1},  db_t = lambda_t,  dh0 = mu_0
//
// One thread per (batch row, channel): the plain form.  Block by block from the last to the
// first it recomputes the block's states from its checkpoint and walks back over them.
#include "gated_device.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

template <typename IO, int MODE, bool IG>
__global__ __launch_bounds__(64) void gated_bwd_kernel(ssm_gated_scan_bwd_args_t a, const float *ck, float *part) {
    __shared__ float before[SSM_GATED_BLOCK][64];
    const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
    if (d >= a.dim) return;
    GateChannel c = {a.A ? a.A[d] : 0.0f, a.gate_bias ? a.gate_bias[d] : 0.0f, a.in_bias ? a.in_bias[d] : 0.0f};
    float mu = a.dh_final ? a.dh_final[b * a.dim + d] : 0.0f;
    float sA = 0.0f, sg = 0.0f, si = 0.0f;
    for (int64_t blk = (a.seqlen - 1) / SSM_GATED_BLOCK; blk >= 0; --blk) {
        const int64_t t0 = blk * SSM_GATED_BLOCK;
        const int n = (int)(a.seqlen - t0 < SSM_GATED_BLOCK ? a.seqlen - t0 : SSM_GATED_BLOCK);
        float h = ck[(blk * a.batch + b) * a.dim + d];
        for (int k = 0; k < n; ++k) {
            const int64_t i = (b * a.seqlen + t0 + k) * a.dim + d;
            before[k][threadIdx.x] = h;
            float at, bt;
            gate_step<MODE, IG>(load_io<IO>(a.x, i), load_io<IO>(a.gate, i), IG ? load_io<IO>(a.in_gate, i) : 0.0f, c,
                                at, bt);
            h = a.reset && a.reset[b * a.seqlen + t0 + k] ? bt : __builtin_fmaf(at, h, bt);
        }
        for (int k = n - 1; k >= 0; --k) {
            const int64_t i = (b * a.seqlen + t0 + k) * a.dim + d;
            const float x = load_io<IO>(a.x, i), g = load_io<IO>(a.gate, i), ig = IG ? load_io<IO>(a.in_gate, i) : 0.0f;
            const bool cut = a.reset && a.reset[b * a.seqlen + t0 + k];
            const float lam = load_io<IO>(a.dy, i) + mu;
            const GateGrad o = gate_grad<MODE, IG>(x, g, ig, c, cut ? 0.0f : lam * before[k][threadIdx.x], lam);
            float at, bt;
            gate_step<MODE, IG>(x, g, ig, c, at, bt);
            mu = cut ? 0.0f : at * lam;
            store_io<IO>(a.dx, i, o.dx);
            store_io<IO>(a.dgate, i, o.dg);
            if (IG) store_io<IO>(a.din_gate, i, o.di);
            sA += o.dA;
            sg += o.dg;
            si += o.di;
        }
    }
    if (a.dh0) a.dh0[b * a.dim + d] = mu;
    const int64_t n = a.batch * a.dim, i = b * a.dim + d;
    part[i] = sA;
    part[n + i] = sg;
    part[2 * n + i] = si;
}

__global__ __launch_bounds__(256) void gated_sum_kernel(const float *part, int64_t B, int64_t D, float *dA, float *dg,
                                                        float *di) {
    const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (d >= D) return;
    float s[3] = {};
    for (int k = 0; k < 3; ++k)
        for (int64_t b = 0; b < B; ++b) s[k] += part[(k * B + b) * D + d];
    if (dA) dA[d] = s[0];
    if (dg) dg[d] = s[1];
    if (di) di[d] = s[2];
}

size_t r256(size_t v) { return (v + 255) & ~(size_t)255; }
size_t ckpt_bytes(const ssm_gated_scan_bwd_args_t &a) {
    return r256((size_t)((a.seqlen + SSM_GATED_BLOCK - 1) / SSM_GATED_BLOCK * a.batch * a.dim) * 4);
}

// The forward call that writes the checkpoints alone (y and h_final NULL).
ssm_gated_scan_args_t forward_of(const ssm_gated_scan_bwd_args_t &a) {
    ssm_gated_scan_args_t f = {};
    f.batch = a.batch;
    f.seqlen = a.seqlen;
    f.dim = a.dim;
    f.io_dtype = a.io_dtype;
    f.mode = a.mode;
    f.x = a.x;
    f.gate = a.gate;
    f.in_gate = a.in_gate;
    f.A = a.A;
    f.gate_bias = a.gate_bias;
    f.in_bias = a.in_bias;
    f.reset = a.reset;
    f.h0 = a.h0;
    return f;
}

}  // namespace

size_t gated_scan_bwd_workspace_bytes(const ssm_gated_scan_bwd_args_t &a) {
    const size_t sums = r256((size_t)(3 * a.batch * a.dim) * 4);
    return sums + (a.checkpoints ? 0 : ckpt_bytes(a) + gated_scan_workspace_bytes(forward_of(a)));
}

hipError_t launch_gated_scan_bwd(const ssm_gated_scan_bwd_args_t &a, hipStream_t stream) {
    float *part = static_cast<float *>(a.workspace);
    const float *ck = a.checkpoints;
    hipError_t e = hipSuccess;
    if (!ck) {
        char *at = static_cast<char *>(a.workspace) + r256((size_t)(3 * a.batch * a.dim) * 4);
        ssm_gated_scan_args_t f = forward_of(a);
        f.checkpoints = reinterpret_cast<float *>(at);
        f.workspace = at + ckpt_bytes(a);
        ck = f.checkpoints;
        e = launch_gated_scan_fwd(f, stream);
    }
    const dim3 grid((unsigned)((a.dim + 63) / 64), (unsigned)a.batch);
    if (e == hipSuccess) {
        gate_dispatch(a.io_dtype, a.mode, a.in_gate != nullptr, [&](auto io, auto mode, auto ig) {
            gated_bwd_kernel<decltype(io), decltype(mode)::value, decltype(ig)::value>
                <<<grid, 64, 0, stream>>>(a, ck, part);
        });
        e = hipGetLastError();
    }
    if (e == hipSuccess) {
        gated_sum_kernel<<<(unsigned)((a.dim + 255) / 256), 256, 0, stream>>>(part, a.batch, a.dim, a.dA, a.dgate_bias,
                                                                              a.din_bias);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace ssm
