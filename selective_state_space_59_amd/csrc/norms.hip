// norms.hip -- the fused norms around a block on gfx950: residual sum + RMSNorm
// (ssm_add_rmsnorm_*) and the RMSNorm of a gated layer output (ssm_gated_rmsnorm_*),
// forward and backward.
//
// One wave per row (or per group of a row), element by element: the plain form.
#include "ssm_device.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int s = 32; s >= 1; s /= 2) v += __shfl_xor(v, s, 64);
    return v;
}

__device__ __forceinline__ float load_any(const void *p, int64_t i, int32_t dt) {
    return dt == SSM_BF16 ? load_io<io_bf16>(p, i) : load_io<io_f32>(p, i);
}
__device__ __forceinline__ void store_any(void *p, int64_t i, float v, int32_t dt) {
    if (dt == SSM_BF16)
        store_io<io_bf16>(p, i, v);
    else
        store_io<io_f32>(p, i, v);
}

__device__ __forceinline__ float inv_rms(float sum, int64_t n, float eps) { return 1.0f / sqrtf(sum / (float)n + eps); }

struct Boundary {
    const ssm_add_norm_bwd_args_t &a;
    int64_t base;
    float k;  // 1 / rms(x), with a post norm
    __device__ float x(int64_t i) const { return load_any(a.x, base + i, a.io_dtype); }
    __device__ float u(int64_t i) const { return a.post_w ? x(i) * k * a.post_w[i] : x(i); }
    __device__ float r(int64_t i) const {
        const float v = u(i), s = a.scale ? v * a.scale[i] : v;
        return a.residual ? load_any(a.residual, base + i, a.res_dtype) + s : s;
    }
};

__device__ __forceinline__ Boundary boundary(const ssm_add_norm_bwd_args_t &a, int64_t row, int lane, float *q) {
    Boundary m = {a, row * a.dim, 1.0f};
    float acc = 0.0f;
    if (a.post_w) {
        for (int64_t i = lane; i < a.dim; i += 64) acc += m.x(i) * m.x(i);
        m.k = inv_rms(wave_sum(acc), a.dim, a.eps);
        acc = 0.0f;
    }
    for (int64_t i = lane; i < a.dim; i += 64) {
        const float r = m.r(i);
        acc += r * r;
    }
    *q = inv_rms(wave_sum(acc), a.dim, a.eps);
    return m;
}

__global__ __launch_bounds__(64) void add_norm_kernel(ssm_add_norm_bwd_args_t a, void *res_out, void *y) {
    float q;
    const Boundary m = boundary(a, blockIdx.x, threadIdx.x, &q);
    for (int64_t i = threadIdx.x; i < a.dim; i += 64) {
        const float r = m.r(i);
        store_any(y, m.base + i, r * q * a.w[i], a.io_dtype);
        if (res_out) store_any(res_out, m.base + i, r, a.res_dtype);
    }
}

__global__ __launch_bounds__(64) void add_norm_bwd_kernel(ssm_add_norm_bwd_args_t a, float *stat) {
    float q;
    const Boundary m = boundary(a, blockIdx.x, threadIdx.x, &q);
    const int64_t D = a.dim;
    float acc = 0.0f;
    for (int64_t i = threadIdx.x; i < D; i += 64) acc += load_any(a.dy, m.base + i, a.io_dtype) * a.w[i] * m.r(i);
    const float p = wave_sum(acc) / (float)D * q * q * q;
    auto dr = [&](int64_t i) {
        const float up = a.dres_out ? load_any(a.dres_out, m.base + i, a.res_dtype) : 0.0f;
        return up + q * a.w[i] * load_any(a.dy, m.base + i, a.io_dtype) - m.r(i) * p;
    };
    float p2 = 0.0f;
    if (a.post_w) {
        acc = 0.0f;
        for (int64_t i = threadIdx.x; i < D; i += 64)
            acc += dr(i) * (a.scale ? a.scale[i] : 1.0f) * a.post_w[i] * m.x(i);
        p2 = wave_sum(acc) / (float)D * m.k * m.k * m.k;
    }
    for (int64_t i = threadIdx.x; i < D; i += 64) {
        const float d = dr(i);
        float du = a.scale ? d * a.scale[i] : d;
        if (a.post_w) du = m.k * a.post_w[i] * du - m.x(i) * p2;
        store_any(a.dx, m.base + i, du, a.io_dtype);
        if (a.dresidual && a.dresidual != a.dres_out) store_any(a.dresidual, m.base + i, d, a.res_dtype);
    }
    if (threadIdx.x == 0) {
        float *s = stat + 4 * (int64_t)blockIdx.x;
        s[0] = q;
        s[1] = p;
        s[2] = m.k;
    }
}

__global__ __launch_bounds__(64) void add_norm_sums_kernel(ssm_add_norm_bwd_args_t a, const float *stat) {
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (i >= a.dim) return;
    float dw = 0.0f, ds = 0.0f, dp = 0.0f;
    for (int64_t row = 0; row < a.rows; ++row) {
        const float q = stat[4 * row], p = stat[4 * row + 1];
        const Boundary m = {a, row * a.dim, stat[4 * row + 2]};
        const float dy = load_any(a.dy, m.base + i, a.io_dtype), r = m.r(i);
        const float up = a.dres_out ? load_any(a.dres_out, m.base + i, a.res_dtype) : 0.0f;
        const float d = up + q * a.w[i] * dy - r * p;
        dw += dy * r * q;
        ds += d * m.u(i);
        dp += d * (a.scale ? a.scale[i] : 1.0f) * m.x(i) * m.k;
    }
    a.dw[i] = dw;
    if (a.dscale) a.dscale[i] = ds;
    if (a.dpost_w) a.dpost_w[i] = dp;
}

__global__ __launch_bounds__(64) void copy_rows_kernel(ssm_add_norm_bwd_args_t a, const float *stat) {
    // dresidual in place of dres_out, after the sums have read it
    const int64_t base = (int64_t)blockIdx.x * a.dim;
    const float q = stat[4 * (int64_t)blockIdx.x], p = stat[4 * (int64_t)blockIdx.x + 1];
    const Boundary m = {a, base, stat[4 * (int64_t)blockIdx.x + 2]};
    for (int64_t i = threadIdx.x; i < a.dim; i += 64) {
        const float d = load_any(a.dres_out, base + i, a.res_dtype) +
                        q * a.w[i] * load_any(a.dy, base + i, a.io_dtype) - m.r(i) * p;
        store_any(a.dresidual, base + i, d, a.res_dtype);
    }
}

__global__ __launch_bounds__(64) void gated_norm_kernel(ssm_gated_norm_bwd_args_t a, void *y) {
    const int64_t S = a.dim / a.groups, base = (int64_t)blockIdx.x * S, wo = (blockIdx.x % a.groups) * S;
    float acc = 0.0f;
    auto val = [&](int64_t i, float *g) {
        const float x = load_any(a.x, base + i, a.io_dtype), z = load_any(a.z, base + i, a.io_dtype);
        *g = silu(z);
        return a.gate_first ? x * *g : x;
    };
    float g;
    for (int64_t i = threadIdx.x; i < S; i += 64) {
        const float v = val(i, &g);
        acc += v * v;
    }
    const float q = inv_rms(wave_sum(acc), S, a.eps);
    for (int64_t i = threadIdx.x; i < S; i += 64) {
        const float v = val(i, &g);
        store_any(y, base + i, a.gate_first ? v * q * a.w[wo + i] : v * q * a.w[wo + i] * g, a.io_dtype);
    }
}

__global__ __launch_bounds__(64) void gated_norm_bwd_kernel(ssm_gated_norm_bwd_args_t a, float *stat) {
    const int64_t S = a.dim / a.groups, base = (int64_t)blockIdx.x * S, wo = (blockIdx.x % a.groups) * S;
    auto ld = [&](const void *p, int64_t i) { return load_any(p, base + i, a.io_dtype); };
    float acc = 0.0f, dot = 0.0f;
    for (int64_t i = threadIdx.x; i < S; i += 64) {
        const float g = silu(ld(a.z, i)), x = ld(a.x, i), v = a.gate_first ? x * g : x;
        acc += v * v;
        dot += v * a.w[wo + i] * (a.gate_first ? ld(a.dy, i) : ld(a.dy, i) * g);
    }
    const float q = inv_rms(wave_sum(acc), S, a.eps), p = wave_sum(dot) / (float)S * q * q * q;
    for (int64_t i = threadIdx.x; i < S; i += 64) {
        const float z = ld(a.z, i), x = ld(a.x, i), dy = ld(a.dy, i), w = a.w[wo + i];
        const float sg = hw_rcp(1.0f + hw_exp2(-z * kLog2e)), g = z * sg, slope = sg * (1.0f + z * (1.0f - sg));
        float dx, dz;
        if (a.gate_first) {
            const float dv = q * w * dy - x * g * p;
            dx = dv * g;
            dz = dv * x * slope;
        } else {
            dx = q * w * dy * g - x * p;
            dz = dy * x * q * w * slope;
        }
        store_any(a.dx, base + i, dx, a.io_dtype);
        store_any(a.dz, base + i, dz, a.io_dtype);
    }
    if (threadIdx.x == 0) stat[blockIdx.x] = q;
}

__global__ __launch_bounds__(64) void gated_norm_sums_kernel(ssm_gated_norm_bwd_args_t a, const float *stat) {
    const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (i >= a.dim) return;
    const int64_t g = i / (a.dim / a.groups);
    float dw = 0.0f;
    for (int64_t row = 0; row < a.rows; ++row) {
        const int64_t k = row * a.dim + i;
        dw += load_any(a.dy, k, a.io_dtype) * load_any(a.x, k, a.io_dtype) * silu(load_any(a.z, k, a.io_dtype)) *
              stat[row * a.groups + g];
    }
    a.dw[i] = dw;
}

}  // namespace

hipError_t launch_add_norm_fwd(const ssm_add_norm_args_t &a, hipStream_t stream) {
    ssm_add_norm_bwd_args_t b = {};
    b.rows = a.rows;
    b.dim = a.dim;
    b.io_dtype = a.io_dtype;
    b.res_dtype = a.res_dtype;
    b.x = a.x;
    b.residual = a.residual;
    b.scale = a.scale;
    b.post_w = a.post_w;
    b.w = a.w;
    b.eps = a.eps;
    add_norm_kernel<<<(unsigned)a.rows, 64, 0, stream>>>(b, a.res_out, a.y);
    return hipGetLastError();
}

size_t add_norm_bwd_workspace_bytes(const ssm_add_norm_bwd_args_t &a) { return (size_t)a.rows * 16; }

hipError_t launch_add_norm_bwd(const ssm_add_norm_bwd_args_t &a, hipStream_t stream) {
    float *stat = static_cast<float *>(a.workspace);
    add_norm_bwd_kernel<<<(unsigned)a.rows, 64, 0, stream>>>(a, stat);
    add_norm_sums_kernel<<<(unsigned)((a.dim + 63) / 64), 64, 0, stream>>>(a, stat);
    if (a.dresidual && a.dresidual == a.dres_out) copy_rows_kernel<<<(unsigned)a.rows, 64, 0, stream>>>(a, stat);
    return hipGetLastError();
}

hipError_t launch_gated_norm_fwd(const ssm_gated_norm_args_t &a, hipStream_t stream) {
    ssm_gated_norm_bwd_args_t b = {};
    b.rows = a.rows;
    b.dim = a.dim;
    b.groups = a.groups;
    b.io_dtype = a.io_dtype;
    b.gate_first = a.gate_first;
    b.x = a.x;
    b.z = a.z;
    b.w = a.w;
    b.eps = a.eps;
    gated_norm_kernel<<<(unsigned)(a.rows * a.groups), 64, 0, stream>>>(b, a.y);
    return hipGetLastError();
}

size_t gated_norm_bwd_workspace_bytes(const ssm_gated_norm_bwd_args_t &a) { return (size_t)(a.rows * a.groups) * 4; }

hipError_t launch_gated_norm_bwd(const ssm_gated_norm_bwd_args_t &a, hipStream_t stream) {
    float *stat = static_cast<float *>(a.workspace);
    gated_norm_bwd_kernel<<<(unsigned)(a.rows * a.groups), 64, 0, stream>>>(a, stat);
    gated_norm_sums_kernel<<<(unsigned)((a.dim + 63) / 64), 64, 0, stream>>>(a, stat);
    return hipGetLastError();
}

}  // namespace ssm
