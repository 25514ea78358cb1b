// add_norm.hip -- residual sum + RMSNorm between two blocks (ssm_add_rmsnorm_fwd / _bwd) on
// gfx950.  Per row, with u = x or RMS(x) post_w:
//   r = residual + scale u,   q = 1 / sqrt(mean(r^2) + eps),   y = r q w
// and back, for dy and the stream's own gradient dres:
//   dr = dres + q w dy - r q^3 mean(w dy r)                      (dresidual)
//   du = scale dr;   dx = du, or k post_w du - x k^3 mean(post_w du x) with k = 1 / rms(x)
//   dw = sum dy r q,  dscale = sum dr u,  dpost_w = sum du x k   over the rows
//
// Bound by HBM: each row is read once into registers and its results are written from there.
// Measured: 16384 x 768 bf16 with an fp32 stream, forward 31 us (4.8 TB/s), backward 40 us (5.6);
// 16384 x 2560 bf16 with post norm and scale, forward 55 us (6.1 TB/s, caches included), backward
// 126 us (4.0 TB/s: five-wave workgroups of 124 registers a lane, two to a CU).  On fp32 rows over 4096
// with a post norm or scale the backward's 1024 threads have 128 registers each and keep 12 bytes
// (44 with a bf16 stream) in scratch.
//
// The norm takes r before its rounding to the stream's type, and the backward forms it again from
// x and residual: a stream rounded to bf16 would put its rounding (2^-9) into dw, which is summed
// in fp32.
#include "norm_rows.h"

namespace ssm {
namespace {

// r of one group; k: 1 / rms(x) with a post norm.  u is left in `u`.
template <typename IO, typename RES, bool EXTRA, int E>
__device__ __forceinline__ void stream_group(const Raw<IO, E> &x, const Raw<RES, E> &res, const float (&pw)[E],
                                        const float (&sc)[E], bool post, bool scale, float k, float (&u)[E],
                                        float (&r)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
        u[e] = x[e];
        if constexpr (EXTRA) {
            if (post) u[e] = u[e] * k * pw[e];
            r[e] = scale ? __builtin_fmaf(sc[e], u[e], res[e]) : res[e] + u[e];
        } else {
            r[e] = res[e] + u[e];
        }
    }
}

template <typename IO, typename RES, bool EXTRA, typename SH>
__global__ __launch_bounds__(SH::THREADS) void add_norm_kernel(ssm_add_norm_args_t a, int64_t slots) {
    constexpr int TEAM = SH::TEAM, NR = SH::NR, E = SH::E;
    __shared__ SumSlots sums;
    int turn = 0;
    const int lane = TEAM == 0 ? threadIdx.x : threadIdx.x % (TEAM ? TEAM : 1), width = TEAM == 0 ? blockDim.x : TEAM;
    const TeamRows t = team_rows<TEAM>(1, slots);
    const int D = (int)a.dim;
    const float inv_n = 1.0f / (float)D;
    const bool post = EXTRA && a.post_w, scale = EXTRA && a.scale;
    float w[NR][E], pw[NR][E] = {}, sc[NR][E] = {};
    int n[NR];
#pragma unroll
    for (int c = 0; c < NR; ++c) {
        const int i = E * (lane + c * width);
        n[c] = max(0, min(E, D - i));
        load_vec(a.w, i, n[c], w[c]);
        if (post) load_vec(a.post_w, i, n[c], pw[c]);
        if (scale) load_vec(a.scale, i, n[c], sc[c]);
    }
    for (int64_t row = t.row; row < a.rows; row += t.step) {
        const int64_t base = row * D;
        Raw<IO, E> x[NR];
        Raw<RES, E> res[NR];
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            const int i = E * (lane + c * width);
            x[c] = load_raw<IO, E>(a.x, base + i, n[c]);
            res[c] = a.residual ? load_raw<RES, E>(a.residual, base + i, n[c]) : Raw<RES, E>{};
        }
        float k = 1.0f;
        if (post) {
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < NR; ++c)
#pragma unroll
                for (int e = 0; e < E; ++e) s = __builtin_fmaf(x[c][e], x[c][e], s);
            k = inv_rms(team_sum<TEAM>(s, sums, turn), inv_n, a.eps);
        }
        float r[NR][E], u[E], s = 0.0f;
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            stream_group<IO, RES, EXTRA>(x[c], res[c], pw[c], sc[c], post, scale, k, u, r[c]);
#pragma unroll
            for (int e = 0; e < E; ++e) s = __builtin_fmaf(r[c][e], r[c][e], s);
        }
        const float q = inv_rms(team_sum<TEAM>(s, sums, turn), inv_n, a.eps);
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            const int i = E * (lane + c * width);
            if (a.res_out) store_raw<RES>(a.res_out, base + i, n[c], r[c]);
#pragma unroll
            for (int e = 0; e < E; ++e) u[e] = r[c][e] * q * w[c][e];
            store_raw<IO>(a.y, base + i, n[c], u);
        }
    }
}

template <typename IO, typename RES, bool EXTRA, typename SH>
__global__ __launch_bounds__(SH::THREADS) void add_norm_bwd_kernel(ssm_add_norm_bwd_args_t a, int64_t slots, float *part, int64_t prows) {
    constexpr int TEAM = SH::TEAM, NR = SH::NR, E = SH::E;
    __shared__ SumSlots sums;
    int turn = 0;
    const int lane = TEAM == 0 ? threadIdx.x : threadIdx.x % (TEAM ? TEAM : 1), width = TEAM == 0 ? blockDim.x : TEAM;
    const TeamRows t = team_rows<TEAM>(1, slots);
    const int D = (int)a.dim;
    const float inv_n = 1.0f / (float)D;
    const bool post = EXTRA && a.post_w, scale = EXTRA && a.scale;
    float w[NR][E], pw[NR][E] = {}, sc[NR][E] = {};
    float aw[NR][E] = {}, as[NR][E] = {}, ap[NR][E] = {};
    int n[NR];
#pragma unroll
    for (int c = 0; c < NR; ++c) {
        const int i = E * (lane + c * width);
        n[c] = max(0, min(E, D - i));
        load_vec(a.w, i, n[c], w[c]);
        if (post) load_vec(a.post_w, i, n[c], pw[c]);
        if (scale) load_vec(a.scale, i, n[c], sc[c]);
    }
    for (int64_t row = t.row; row < a.rows; row += t.step) {
        const int64_t base = row * D;
        Raw<IO, E> x[NR], dy[NR];
        Raw<RES, E> res[NR], up[NR];
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            const int i = E * (lane + c * width);
            x[c] = load_raw<IO, E>(a.x, base + i, n[c]);
            res[c] = a.residual ? load_raw<RES, E>(a.residual, base + i, n[c]) : Raw<RES, E>{};
            dy[c] = load_raw<IO, E>(a.dy, base + i, n[c]);
            up[c] = a.dres_out ? load_raw<RES, E>(a.dres_out, base + i, n[c]) : Raw<RES, E>{};
        }
        float k = 1.0f;
        if (post) {
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < NR; ++c)
#pragma unroll
                for (int e = 0; e < E; ++e) s = __builtin_fmaf(x[c][e], x[c][e], s);
            k = inv_rms(team_sum<TEAM>(s, sums, turn), inv_n, a.eps);
        }
        float u[NR][E], r[NR][E], s = 0.0f, dot = 0.0f;
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            stream_group<IO, RES, EXTRA>(x[c], res[c], pw[c], sc[c], post, scale, k, u[c], r[c]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s = __builtin_fmaf(r[c][e], r[c][e], s);
                dot = __builtin_fmaf(dy[c][e] * w[c][e], r[c][e], dot);
            }
        }
        team_sum<TEAM>(s, dot, sums, turn);
        const float q = inv_rms(s, inv_n, a.eps), m = dot * inv_n * q * q * q;
        float d2 = 0.0f;
#pragma unroll
        for (int c = 0; c < NR; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                aw[c][e] = __builtin_fmaf(dy[c][e] * q, r[c][e], aw[c][e]);
                // dr in r's place
                r[c][e] = __builtin_fmaf(q * w[c][e], dy[c][e], __builtin_fmaf(-m, r[c][e], up[c][e]));
                if constexpr (EXTRA) {
                    if (scale) as[c][e] = __builtin_fmaf(r[c][e], u[c][e], as[c][e]);
                    u[c][e] = scale ? r[c][e] * sc[c][e] : r[c][e];  // du
                    if (post) {
                        ap[c][e] = __builtin_fmaf(u[c][e] * k, x[c][e], ap[c][e]);
                        d2 = __builtin_fmaf(u[c][e] * pw[c][e], x[c][e], d2);
                    }
                }
            }
        if (post) {
            const float m2 = team_sum<TEAM>(d2, sums, turn) * inv_n * k * k * k;
#pragma unroll
            for (int c = 0; c < NR; ++c)
#pragma unroll
                for (int e = 0; e < E; ++e) u[c][e] = __builtin_fmaf(k * pw[c][e], u[c][e], -m2 * x[c][e]);
        }
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            const int i = E * (lane + c * width);
            if (a.dresidual) store_raw<RES>(a.dresidual, base + i, n[c], r[c]);
            if constexpr (EXTRA)
                store_raw<IO>(a.dx, base + i, n[c], u[c]);
            else
                store_raw<IO>(a.dx, base + i, n[c], r[c]);
        }
    }
    int64_t slot = t.row;
    bool writes = t.row < slots;
    if constexpr (TEAM == 64) {
        // the four waves hold the same columns
        __shared__ float lds[kTeamThreads * 8];
        waves_sum(aw, lds, lane);
        if (scale) waves_sum(as, lds, lane);
        if (post) waves_sum(ap, lds, lane);
        slot = blockIdx.x;
        writes = threadIdx.x < 64;
    }
    if (!writes) return;
#pragma unroll
    for (int c = 0; c < NR; ++c) {
        const int i = E * (lane + c * width);
        store_raw<io_f32>(part, slot * D + i, n[c], aw[c]);
        if (scale) store_raw<io_f32>(part, (prows + slot) * D + i, n[c], as[c]);
        if (post) store_raw<io_f32>(part, (2 * prows + slot) * D + i, n[c], ap[c]);
    }
}

// Rows longer than kBlockRow: a workgroup of 1024 reads the row again for each pass; its sums
// over rows stand in its row of the partial sums, where each element belongs to one thread.
template <typename IO, typename RES>
struct LongRow {
    const void *x, *residual;
    const float *post_w, *scale;
    int64_t base;
    float k;
    __device__ __forceinline__ float xv(int i) const { return load_io<IO>(x, base + i); }
    __device__ __forceinline__ float u(int i) const { return post_w ? xv(i) * k * post_w[i] : xv(i); }
    __device__ __forceinline__ float r(int i) const {
        const float res = residual ? load_io<RES>(residual, base + i) : 0.0f;
        return scale ? __builtin_fmaf(scale[i], u(i), res) : res + u(i);
    }
    // 1 / rms of x into k (with a post norm)
    __device__ __forceinline__ void post_rms(int D, float eps, SumSlots &sums, int &turn) {
        k = 1.0f;
        if (!post_w) return;
        float s = 0.0f;
        for (int i = threadIdx.x; i < D; i += 1024) s = __builtin_fmaf(xv(i), xv(i), s);
        k = inv_rms(team_sum<0>(s, sums, turn), 1.0f / (float)D, eps);
    }
};

template <typename IO, typename RES>
__global__ __launch_bounds__(1024) void add_norm_long_kernel(ssm_add_norm_args_t a) {
    __shared__ SumSlots sums;
    int turn = 0;
    const int D = (int)a.dim;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        LongRow<IO, RES> l = {a.x, a.residual, a.post_w, a.scale, row * D, 1.0f};
        l.post_rms(D, a.eps, sums, turn);
        float s = 0.0f;
        for (int i = threadIdx.x; i < D; i += 1024) {
            const float r = l.r(i);
            s = __builtin_fmaf(r, r, s);
        }
        const float q = inv_rms(team_sum<0>(s, sums, turn), 1.0f / (float)D, a.eps);
        for (int i = threadIdx.x; i < D; i += 1024) {
            const float r = l.r(i);
            store_io<IO>(a.y, l.base + i, r * q * a.w[i]);
            if (a.res_out) store_io<RES>(a.res_out, l.base + i, r);
        }
    }
}

template <typename IO, typename RES>
__global__ __launch_bounds__(1024) void add_norm_bwd_long_kernel(ssm_add_norm_bwd_args_t a, float *part, int64_t prows) {
    __shared__ SumSlots sums;
    int turn = 0;
    const int D = (int)a.dim;
    const float inv_n = 1.0f / (float)D;
    float *pw = part + blockIdx.x * (int64_t)D, *ps = pw + prows * D, *pp = ps + prows * D;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const bool first = row == blockIdx.x;
        LongRow<IO, RES> l = {a.x, a.residual, a.post_w, a.scale, row * D, 1.0f};
        l.post_rms(D, a.eps, sums, turn);
        float s = 0.0f, dot = 0.0f;
        for (int i = threadIdx.x; i < D; i += 1024) {
            const float r = l.r(i);
            s = __builtin_fmaf(r, r, s);
            dot = __builtin_fmaf(load_io<IO>(a.dy, l.base + i) * a.w[i], r, dot);
        }
        team_sum<0>(s, dot, sums, turn);
        const float q = inv_rms(s, inv_n, a.eps), m = dot * inv_n * q * q * q;
        auto dr = [&](int i, float r) {
            const float up = a.dres_out ? load_io<RES>(a.dres_out, l.base + i) : 0.0f;
            return __builtin_fmaf(q * a.w[i], load_io<IO>(a.dy, l.base + i), __builtin_fmaf(-m, r, up));
        };
        float m2 = 0.0f;
        if (a.post_w) {
            float d2 = 0.0f;
            for (int i = threadIdx.x; i < D; i += 1024) {
                const float d = dr(i, l.r(i)), du = a.scale ? d * a.scale[i] : d;
                d2 = __builtin_fmaf(du * a.post_w[i], l.xv(i), d2);
            }
            m2 = team_sum<0>(d2, sums, turn) * inv_n * l.k * l.k * l.k;
        }
        for (int i = threadIdx.x; i < D; i += 1024) {
            const float r = l.r(i), u = l.u(i), d = dr(i, r), du = a.scale ? d * a.scale[i] : d, x = l.xv(i);
            pw[i] = (first ? 0.0f : pw[i]) + load_io<IO>(a.dy, l.base + i) * q * r;
            if (a.scale) ps[i] = (first ? 0.0f : ps[i]) + d * u;
            if (a.post_w) pp[i] = (first ? 0.0f : pp[i]) + du * l.k * x;
            if (a.dresidual) store_io<RES>(a.dresidual, l.base + i, d);
            store_io<IO>(a.dx, l.base + i, a.post_w ? __builtin_fmaf(l.k * a.post_w[i], du, -m2 * x) : du);
        }
    }
}

template <typename F>
void with_types(int32_t io, int32_t res, F &&f) {
    if (io == SSM_BF16) {
        if (res == SSM_BF16)
            f(io_bf16{}, io_bf16{});
        else
            f(io_bf16{}, io_f32{});
    } else {
        if (res == SSM_BF16)
            f(io_f32{}, io_bf16{});
        else
            f(io_f32{}, io_f32{});
    }
}

// The forward's half waves of 513 to 768 channels against waves of two groups, 16384 rows of bf16: 640
// 14.1 and 14.9 us, 768 15.9 and 16.6; with post norm and scale, where they hold more registers, 640 17.0
// and 16.8, 768 17.0 and 18.3 (fp32 21.3 and 21.8, 29.0 and 27.7).
constexpr int64_t kFwdBlocks = 1024, kLongBlocks = 256;

// In the backward a lane of a workgroup takes 16 bytes a group from bf16 rows, and also from fp32
// rows as long as two workgroups of half as many elements a lane, 12 waves at most, fit a CU
// (8192 x 2560 fp32 with post norm and scale: 134 us, against 176 with 8 elements and 130 registers
// a lane; of 4096, where one fits either way, 239 against 219).
bool half_groups(int32_t io, int64_t D) { return io == SSM_F32 && D > 1024 && (D + 255) / 256 <= 12; }

// The launch shape of the backward for rows of D (the forward adds half a wave with NR = 3 and a
// wave with NR = 4: it holds less per row, and leaves no partial sums).
RowGrid bwd_grid(int64_t rows, int64_t D, int32_t io) {
    if (D > kBlockRow) return RowGrid{(unsigned)std::min(rows, kLongBlocks), 1024, std::min(rows, kLongBlocks)};
    return row_grid(D <= 64 ? 8 : D <= 256 ? 32 : D <= 1024 ? 64 : 0, D, rows, 1, bwd_blocks(D),
                    half_groups(io, D) ? 4 : 8);
}

// Rows of partial sums: one per workgroup where its waves add theirs up, else one per team.
int64_t partial_rows(int64_t rows, int64_t D, int32_t io) {
    const RowGrid g = bwd_grid(rows, D, io);
    return D > 256 ? g.blocks : g.slots;
}

// Column sums of a call: dw; dscale behind it; dpost_w in the third place.
int column_sums_of(const ssm_add_norm_bwd_args_t &a) { return a.post_w ? 3 : a.scale ? 2 : 1; }

size_t partial_bytes(int K, int64_t n, int64_t D) { return ((size_t)(K * n * D) * 4 + 255) & ~(size_t)255; }

}  // namespace

hipError_t launch_add_norm_fwd(const ssm_add_norm_args_t &a, hipStream_t stream) {
    const int64_t D = a.dim;
    with_types(a.io_dtype, a.res_dtype, [&](auto io, auto res) {
        using IO = decltype(io);
        using RES = decltype(res);
        auto go = [&](auto sh) {
            using SH = decltype(sh);
            const RowGrid g = row_grid(SH::TEAM, D, a.rows, 1, kFwdBlocks);
            if (a.post_w || a.scale)
                add_norm_kernel<IO, RES, true, SH><<<g.blocks, g.threads, 0, stream>>>(a, g.slots);
            else
                add_norm_kernel<IO, RES, false, SH><<<g.blocks, g.threads, 0, stream>>>(a, g.slots);
        };
        if (D <= 64) go(Shape<8, 1>{});
        else if (D <= 256) go(Shape<32, 1>{});
        else if (D <= 512) go(Shape<64, 1>{});
        else if (D <= 768) go(Shape<32, 3>{});
        else if (D <= 1024) go(Shape<64, 2>{});
        else if (D <= 2048) go(Shape<64, 4>{});
        else if (D <= 4096) go(Shape<0, 1, 512>{});
        else if (D <= kBlockRow) go(Shape<0, 1, 1024>{});
        else
            add_norm_long_kernel<IO, RES><<<(unsigned)std::min<int64_t>(a.rows, 2048), 1024, 0, stream>>>(a);
    });
    return hipGetLastError();
}

size_t add_norm_bwd_workspace_bytes(const ssm_add_norm_bwd_args_t &a) {
    const int64_t n = partial_rows(a.rows, a.dim, a.io_dtype);
    const int K = column_sums_of(a);
    return partial_bytes(K, n, a.dim) + column_sums_scratch_bytes(n, a.dim, K);
}

hipError_t launch_add_norm_bwd(const ssm_add_norm_bwd_args_t &a, hipStream_t stream) {
    const int64_t D = a.dim, n = partial_rows(a.rows, D, a.io_dtype);
    const RowGrid g = bwd_grid(a.rows, D, a.io_dtype);
    float *part = static_cast<float *>(a.workspace);
    with_types(a.io_dtype, a.res_dtype, [&](auto io, auto res) {
        using IO = decltype(io);
        using RES = decltype(res);
        auto go = [&](auto sh) {
            using SH = decltype(sh);
            if (a.post_w || a.scale)
                add_norm_bwd_kernel<IO, RES, true, SH><<<g.blocks, g.threads, 0, stream>>>(a, g.slots, part, n);
            else
                add_norm_bwd_kernel<IO, RES, false, SH><<<g.blocks, g.threads, 0, stream>>>(a, g.slots, part, n);
        };
        if (D <= 64) go(Shape<8, 1>{});
        else if (D <= 256) go(Shape<32, 1>{});
        else if (D <= 512) go(Shape<64, 1>{});
        else if (D <= 1024) go(Shape<64, 2>{});
        else if (half_groups(a.io_dtype, D)) {
            if constexpr (IO::bytes == 4) go(Shape<0, 1, 768, 4>{});
        } else if (D <= 4096) go(Shape<0, 1, 512>{});
        else if (D <= kBlockRow) go(Shape<0, 1, 1024>{});
        else
            add_norm_bwd_long_kernel<IO, RES><<<g.blocks, 1024, 0, stream>>>(a, part, n);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    float *out[3] = {a.dw, a.scale ? a.dscale : nullptr, a.post_w ? a.dpost_w : nullptr};
    const int K = column_sums_of(a);
    char *scratch = static_cast<char *>(a.workspace) + partial_bytes(K, n, D);
    return launch_column_sums(part, n, D, K, out, reinterpret_cast<float *>(scratch), stream);
}

}  // namespace ssm
