// quant_fp8.hip -- e4m3 with block scales (ssm_quantize_fp8, ssm_add_rmsnorm_fp8) on gfx950.  Per block of
// 128 columns (and 1 or 128 rows) with largest magnitude m:
//   scale = max(m, 2^-100) / 448,   q = e4m3(x / scale)
// 16 lanes of 8 elements each hold a row of a block, so m is four steps between lanes and a lane stores
// 8 bytes.  The magnitude is compared as an integer, which lets a NaN through.  Bound by HBM:
// the norm of 16384 x 2560 with an fp32 stream, post norm and scale 90 us, 5.1 TB/s, as fast as a plain copy; 16384 x
// 10240 quantised by rows and by 128 rows 107 and 94 us in bf16 (4.7 and 5.4 TB/s), 142 and 148 in fp32.
#include "norm_rows.h"

namespace ssm {
namespace {

constexpr int kQuantLanes = SSM_FP8_BLOCK / 8;
constexpr uint32_t kLeastBits = 27u << 23;  // 2^-100

__device__ __forceinline__ uint32_t magnitude8(const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
    return m;
}

// Largest magnitude over 16 lanes.
__device__ __forceinline__ uint32_t magnitude16(uint32_t m) {
#pragma unroll
    for (int s = 1; s < kQuantLanes; s *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, s, 64));
    return m;
}

__device__ __forceinline__ float scale_of(uint32_t m) { return __uint_as_float(max(m, kLeastBits)) / 448.0f; }

// x / scale as a product with the reciprocal and one correction: the rounded quotient, which bf16 values
// often put on a border between two e4m3 ones.  (The correction is formed from t scale - x, whose zero has the
// sign that leaves a t of -0 as it is.)
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float scale) {
    const float inv = 1.0f / scale;
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = x[e] * inv;
        q[e] = __builtin_fmaf(-__builtin_fmaf(t, scale, -x[e]), inv, t);
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false), hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Blocks of one row: 16 a workgroup, counted along the rows.
template <typename IO>
__global__ __launch_bounds__(256) void quant_rows_kernel(ssm_quantize_fp8_args_t a, int per_row) {
    const int64_t base = (int64_t)blockIdx.x * 16;
    const int64_t row0 = base / per_row;
    const unsigned at = (unsigned)(base - row0 * per_row) + threadIdx.x / kQuantLanes;
    const int64_t row = row0 + at / (unsigned)per_row;
    const int block = at % (unsigned)per_row;
    const int64_t i = 128 * block + 8 * (int)(threadIdx.x % kQuantLanes);
    const bool in = row < a.rows && i < a.dim;
    float x[8] = {};
    if (in) {
        const Raw<IO, 8> r = load_raw<IO, 8>(a.x, row * a.dim + i, 8);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = r[e];
    }
    const float scale = scale_of(magnitude16(magnitude8(x)));
    if (!in) return;
    *reinterpret_cast<uint2 *>(static_cast<char *>(a.q) + row * a.dim + i) = quantise8(x, scale);
    if (threadIdx.x % kQuantLanes == 0) a.scales[row * per_row + block] = scale;
}

// Blocks of 128 rows: one a workgroup, 16 rows at a time, held in registers between the two passes.
template <typename IO>
__global__ __launch_bounds__(256) void quant_tiles_kernel(ssm_quantize_fp8_args_t a, int per_row) {
    __shared__ uint32_t most[4];
    const int64_t band = blockIdx.x / per_row;
    const int block = blockIdx.x % per_row;
    const int64_t i = 128 * block + 8 * (int)(threadIdx.x % kQuantLanes);
    const int64_t row0 = band * SSM_FP8_BLOCK + threadIdx.x / kQuantLanes;
    Raw<IO, 8> r[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t row = row0 + 16 * j;
        r[j] = row < a.rows && i < a.dim ? load_raw<IO, 8>(a.x, row * a.dim + i, 8) : Raw<IO, 8>{};
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = r[j][e];
        m = max(m, magnitude8(x));
    }
#pragma unroll
    for (int s = 1; s < 64; s *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, s, 64));
    if (threadIdx.x % 64 == 0) most[threadIdx.x / 64] = m;
    __syncthreads();
    const float scale = scale_of(max(max(most[0], most[1]), max(most[2], most[3])));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t row = row0 + 16 * j;
        if (row >= a.rows || i >= a.dim) continue;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = r[j][e];
        *reinterpret_cast<uint2 *>(static_cast<char *>(a.q) + row * a.dim + i) = quantise8(x, scale);
    }
    if (threadIdx.x == 0) a.scales[band * per_row + block] = scale;
}

// The norm as in add_norm.hip, each row's groups of 16 lanes quantising their block at the end.
template <typename IO, typename RES, bool EXTRA, typename SH>
__global__ __launch_bounds__(SH::THREADS) void add_norm_fp8_kernel(ssm_add_norm_fp8_args_t p, int64_t slots) {
    constexpr int TEAM = SH::TEAM, NR = SH::NR;
    const ssm_add_norm_args_t &a = p.norm;
    __shared__ SumSlots sums;
    int turn = 0;
    const int lane = TEAM == 0 ? threadIdx.x : threadIdx.x % (TEAM ? TEAM : 1), width = TEAM == 0 ? blockDim.x : TEAM;
    const TeamRows t = team_rows<TEAM>(1, slots);
    const int D = (int)a.dim, per_row = (D + 127) / 128;
    const float inv_n = 1.0f / (float)D;
    const bool post = EXTRA && a.post_w, scaled = EXTRA && a.scale;
    float w[NR][8], pw[NR][8] = {}, sc[NR][8] = {};
    int n[NR];
#pragma unroll
    for (int c = 0; c < NR; ++c) {
        const int i = 8 * (lane + c * width);
        n[c] = i < D ? 8 : 0;
        load_vec(a.w, i, n[c], w[c]);
        if (post) load_vec(a.post_w, i, n[c], pw[c]);
        if (scaled) load_vec(a.scale, i, n[c], sc[c]);
    }
    for (int64_t row = t.row; row < a.rows; row += t.step) {
        const int64_t base = row * D;
        Raw<IO, 8> x[NR];
        Raw<RES, 8> res[NR];
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            const int i = 8 * (lane + c * width);
            x[c] = load_raw<IO, 8>(a.x, base + i, n[c]);
            res[c] = a.residual ? load_raw<RES, 8>(a.residual, base + i, n[c]) : Raw<RES, 8>{};
        }
        float k = 1.0f;
        if (post) {
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < NR; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = __builtin_fmaf(x[c][e], x[c][e], s);
            k = inv_rms(team_sum<TEAM>(s, sums, turn), inv_n, a.eps);
        }
        float r[NR][8], s = 0.0f;
#pragma unroll
        for (int c = 0; c < NR; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float u = x[c][e];
                if constexpr (EXTRA) {
                    if (post) u = u * k * pw[c][e];
                    r[c][e] = scaled ? __builtin_fmaf(sc[c][e], u, res[c][e]) : res[c][e] + u;
                } else {
                    r[c][e] = res[c][e] + u;
                }
                s = __builtin_fmaf(r[c][e], r[c][e], s);
            }
        const float q = inv_rms(team_sum<TEAM>(s, sums, turn), inv_n, a.eps);
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            const int i = 8 * (lane + c * width);
            if (a.res_out) store_raw<RES>(a.res_out, base + i, n[c], r[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[c][e] = r[c][e] * q * w[c][e];
            const float scale = scale_of(magnitude16(magnitude8(r[c])));
            if (n[c] == 0) continue;
            *reinterpret_cast<uint2 *>(static_cast<char *>(p.q) + base + i) = quantise8(r[c], scale);
            if (lane % kQuantLanes == 0) p.scales[row * per_row + i / 128] = scale;
        }
    }
}

// Rows longer than kBlockRow: a workgroup of 1024 reads the row again for each pass.
template <typename IO, typename RES>
__global__ __launch_bounds__(1024) void add_norm_fp8_long_kernel(ssm_add_norm_fp8_args_t p) {
    const ssm_add_norm_args_t &a = p.norm;
    __shared__ SumSlots sums;
    int turn = 0;
    const int D = (int)a.dim, per_row = (D + 127) / 128;
    const float inv_n = 1.0f / (float)D;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t base = row * D;
        float k = 1.0f;
        const auto stream8 = [&](int i, float (&r)[8]) {
            const Raw<IO, 8> x = load_raw<IO, 8>(a.x, base + i, 8);
            const Raw<RES, 8> res = a.residual ? load_raw<RES, 8>(a.residual, base + i, 8) : Raw<RES, 8>{};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float u = a.post_w ? x[e] * k * a.post_w[i + e] : x[e];
                r[e] = a.scale ? __builtin_fmaf(a.scale[i + e], u, res[e]) : res[e] + u;
            }
        };
        if (a.post_w) {
            float s = 0.0f;
            for (int i = 8 * threadIdx.x; i < D; i += 8192) {
                const Raw<IO, 8> x = load_raw<IO, 8>(a.x, base + i, 8);
#pragma unroll
                for (int e = 0; e < 8; ++e) s = __builtin_fmaf(x[e], x[e], s);
            }
            k = inv_rms(team_sum<0>(s, sums, turn), inv_n, a.eps);
        }
        float s = 0.0f, r[8];
        for (int i = 8 * threadIdx.x; i < D; i += 8192) {
            stream8(i, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = __builtin_fmaf(r[e], r[e], s);
        }
        const float q = inv_rms(team_sum<0>(s, sums, turn), inv_n, a.eps);
        for (int i0 = 0; i0 < D; i0 += 8192) {
            const int i = i0 + 8 * (int)threadIdx.x;
            const bool in = i < D;
            float y[8] = {};
            if (in) {
                stream8(i, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = r[e] * q * a.w[i + e];
            }
            const float scale = scale_of(magnitude16(magnitude8(y)));
            if (!in) continue;
            if (a.res_out) store_raw<RES>(a.res_out, base + i, 8, r);
            *reinterpret_cast<uint2 *>(static_cast<char *>(p.q) + base + i) = quantise8(y, scale);
            if (threadIdx.x % kQuantLanes == 0) p.scales[row * per_row + i / 128] = scale;
        }
    }
}

template <typename IO, typename RES>
void launch_norm(const ssm_add_norm_fp8_args_t &p, hipStream_t stream) {
    const int64_t D = p.norm.dim, rows = p.norm.rows;
    const auto go = [&](auto sh) {
        using SH = decltype(sh);
        const RowGrid g = row_grid(SH::TEAM, D, rows, 1, 1024);
        if (p.norm.post_w || p.norm.scale)
            add_norm_fp8_kernel<IO, RES, true, SH><<<g.blocks, g.threads, 0, stream>>>(p, g.slots);
        else
            add_norm_fp8_kernel<IO, RES, false, SH><<<g.blocks, g.threads, 0, stream>>>(p, g.slots);
    };
    // (teams of 16 lanes at least: a block of 128)
    if (D <= 128) go(Shape<16, 1>{});
    else if (D <= 256) go(Shape<32, 1>{});
    else if (D <= 512) go(Shape<64, 1>{});
    else if (D <= 768) go(Shape<32, 3>{});
    else if (D <= 1024) go(Shape<64, 2>{});
    else if (D <= 2048) go(Shape<64, 4>{});
    else if (D <= 4096) go(Shape<0, 1, 512>{});
    else if (D <= kBlockRow) go(Shape<0, 1, 1024>{});
    else
        add_norm_fp8_long_kernel<IO, RES><<<(unsigned)std::min<int64_t>(rows, 2048), 1024, 0, stream>>>(p);
}

}  // namespace

hipError_t launch_quantize_fp8(const ssm_quantize_fp8_args_t &a, hipStream_t stream) {
    const int per_row = (int)((a.dim + 127) / 128);
    if (a.block_rows == 1) {
        const unsigned blocks = (unsigned)((a.rows * per_row + 15) / 16);
        if (a.io_dtype == SSM_BF16)
            quant_rows_kernel<io_bf16><<<blocks, 256, 0, stream>>>(a, per_row);
        else
            quant_rows_kernel<io_f32><<<blocks, 256, 0, stream>>>(a, per_row);
    } else {
        const unsigned blocks = (unsigned)((a.rows + SSM_FP8_BLOCK - 1) / SSM_FP8_BLOCK * per_row);
        if (a.io_dtype == SSM_BF16)
            quant_tiles_kernel<io_bf16><<<blocks, 256, 0, stream>>>(a, per_row);
        else
            quant_tiles_kernel<io_f32><<<blocks, 256, 0, stream>>>(a, per_row);
    }
    return hipGetLastError();
}

hipError_t launch_add_norm_fp8(const ssm_add_norm_fp8_args_t &a, hipStream_t stream) {
    const bool bf = a.norm.io_dtype == SSM_BF16, rbf = a.norm.res_dtype == SSM_BF16;
    if (bf && rbf) launch_norm<io_bf16, io_bf16>(a, stream);
    else if (bf) launch_norm<io_bf16, io_f32>(a, stream);
    else if (rbf) launch_norm<io_f32, io_bf16>(a, stream);
    else launch_norm<io_f32, io_f32>(a, stream);
    return hipGetLastError();
}

}  // namespace ssm
