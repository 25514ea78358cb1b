// gated_norm.hip -- RMSNorm of a gated layer output over groups of channels
// (ssm_gated_rmsnorm_fwd / _bwd) on gfx950.  With g = SiLU(z), over a group:
//   gate first:  v = x g,  q = 1 / sqrt(mean(v^2) + eps),  y = v q w
//     dv = q w dy - v q^3 mean(w dy v);   dx = dv g;   dz = dv x g';   dw = sum dy v q
//   norm first:  y = x q w g, q of x
//     dx = q w g dy - x q^3 mean(w g dy x);   dz = dy x q w g';   dw = sum dy g x q
// with g' = s (1 + z (1 - s)), s the logistic of z.
//
// Bound by HBM: a group is read once into registers and its results are written from there
// (norm_rows.h has the launch shapes).  Measured in bf16: 16384 x 1536 forward 26.9 us (5.6 TB/s);
// 16384 x 5120 in 8 groups, forward 101 us (5.0 TB/s), backward 161 us (5.2 TB/s).
#include "norm_rows.h"

namespace ssm {
namespace {

__device__ __forceinline__ float logistic(float z) { return hw_rcp(1.0f + hw_exp2(-z * kLog2e)); }

template <typename IO, bool FIRST, typename SH>
__global__ __launch_bounds__(SH::THREADS) void gated_norm_kernel(ssm_gated_norm_args_t a, int64_t slots) {
    constexpr int TEAM = SH::TEAM, NR = SH::NR, E = SH::E;
    __shared__ SumSlots sums;
    int turn = 0;
    const int lane = TEAM == 0 ? threadIdx.x : threadIdx.x % (TEAM ? TEAM : 1), width = TEAM == 0 ? blockDim.x : TEAM;
    const TeamRows t = team_rows<TEAM>(a.groups, slots);
    const int S = (int)(a.dim / a.groups);
    const float inv_n = 1.0f / (float)S;
    const int64_t col = t.g * S;
    float w[NR][E];
    int n[NR];
#pragma unroll
    for (int c = 0; c < NR; ++c) {
        const int i = E * (lane + c * width);
        n[c] = max(0, min(E, S - i));
        load_vec(a.w, col + i, n[c], w[c]);
    }
    for (int64_t row = t.row; row < a.rows; row += t.step) {
        const int64_t base = row * a.dim + col;
        Raw<IO, E> x[NR], z[NR];
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            const int i = E * (lane + c * width);
            x[c] = load_raw<IO, E>(a.x, base + i, n[c]);
            z[c] = load_raw<IO, E>(a.z, base + i, n[c]);
        }
        float v[NR][E], s = 0.0f;
#pragma unroll
        for (int c = 0; c < NR; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[c][e] = FIRST ? x[c][e] * silu(z[c][e]) : x[c][e];
                s = __builtin_fmaf(v[c][e], v[c][e], s);
            }
        const float q = inv_rms(team_sum<TEAM>(s, sums, turn), inv_n, a.eps);
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            const int i = E * (lane + c * width);
#pragma unroll
            for (int e = 0; e < E; ++e) v[c][e] *= FIRST ? q * w[c][e] : q * w[c][e] * silu(z[c][e]);
            store_raw<IO>(a.y, base + i, n[c], v[c]);
        }
    }
}

template <typename IO, bool FIRST, typename SH>
__global__ __launch_bounds__(SH::THREADS) void gated_norm_bwd_kernel(
    ssm_gated_norm_bwd_args_t a, int64_t slots, float *part) {
    constexpr int TEAM = SH::TEAM, NR = SH::NR, E = SH::E;
    __shared__ SumSlots sums;
    int turn = 0;
    const int lane = TEAM == 0 ? threadIdx.x : threadIdx.x % (TEAM ? TEAM : 1), width = TEAM == 0 ? blockDim.x : TEAM;
    const TeamRows t = team_rows<TEAM>(a.groups, slots);
    const int S = (int)(a.dim / a.groups);
    const float inv_n = 1.0f / (float)S;
    const int64_t col = t.g * S;
    float w[NR][E], aw[NR][E] = {};
    int n[NR];
#pragma unroll
    for (int c = 0; c < NR; ++c) {
        const int i = E * (lane + c * width);
        n[c] = max(0, min(E, S - i));
        load_vec(a.w, col + i, n[c], w[c]);
    }
    Raw<IO, E> x[NR], z[NR], dy[NR], x1[NR], z1[NR], dy1[NR];
    auto load_row = [&](int64_t row, Raw<IO, E>(&x)[NR], Raw<IO, E>(&z)[NR], Raw<IO, E>(&dy)[NR]) {
        const int64_t base = row * a.dim + col;
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            const int i = E * (lane + c * width);
            x[c] = load_raw<IO, E>(a.x, base + i, n[c]);
            z[c] = load_raw<IO, E>(a.z, base + i, n[c]);
            dy[c] = load_raw<IO, E>(a.dy, base + i, n[c]);
        }
    };
    constexpr bool AHEAD = NR <= 2;  // the next row is on its way while this one's sums are formed
    if (AHEAD && t.row < a.rows) load_row(t.row, x1, z1, dy1);
    for (int64_t row = t.row; row < a.rows; row += t.step) {
        const int64_t base = row * a.dim + col;
        if constexpr (AHEAD) {
#pragma unroll
            for (int c = 0; c < NR; ++c) {
                x[c] = x1[c];
                z[c] = z1[c];
                dy[c] = dy1[c];
            }
            if (row + t.step < a.rows) load_row(row + t.step, x1, z1, dy1);
        } else {
            load_row(row, x, z, dy);
        }
        float sg[NR][E], s = 0.0f, dot = 0.0f;
#pragma unroll
        for (int c = 0; c < NR; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                sg[c][e] = logistic(z[c][e]);
                const float g = z[c][e] * sg[c][e], v = FIRST ? x[c][e] * g : x[c][e];
                const float up = FIRST ? dy[c][e] : dy[c][e] * g;
                s = __builtin_fmaf(v, v, s);
                dot = __builtin_fmaf(up * w[c][e], v, dot);
            }
        team_sum<TEAM>(s, dot, sums, turn);
        const float q = inv_rms(s, inv_n, a.eps), m = dot * inv_n * q * q * q;
#pragma unroll
        for (int c = 0; c < NR; ++c) {
            const int i = E * (lane + c * width);
            float dx[E], dz[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float g = z[c][e] * sg[c][e], slope = sg[c][e] * __builtin_fmaf(z[c][e], 1.0f - sg[c][e], 1.0f);
                const float qw = q * w[c][e];
                if constexpr (FIRST) {
                    const float v = x[c][e] * g, dv = __builtin_fmaf(qw, dy[c][e], -m * v);
                    dx[e] = dv * g;
                    dz[e] = dv * x[c][e] * slope;
                    aw[c][e] = __builtin_fmaf(dy[c][e] * q, v, aw[c][e]);
                } else {
                    const float up = dy[c][e] * g;
                    dx[e] = __builtin_fmaf(qw, up, -m * x[c][e]);
                    dz[e] = dy[c][e] * x[c][e] * qw * slope;
                    aw[c][e] = __builtin_fmaf(up * q, x[c][e], aw[c][e]);
                }
            }
            store_raw<IO>(a.dx, base + i, n[c], dx);
            store_raw<IO>(a.dz, base + i, n[c], dz);
        }
    }
    int64_t slot = t.row;
    bool writes = t.row < slots;
    if constexpr (TEAM == 64) {
        // the four waves hold the same columns
        __shared__ float lds[kTeamThreads * 8];
        waves_sum(aw, lds, lane);
        slot = blockIdx.x / a.groups;
        writes = threadIdx.x < 64;
    }
    if (!writes) return;
#pragma unroll
    for (int c = 0; c < NR; ++c) store_raw<io_f32>(part, slot * a.dim + col + E * (lane + c * width), n[c], aw[c]);
}

// Groups longer than kBlockRow: a workgroup of 1024 reads the group again for each pass.
template <typename IO, bool FIRST>
__global__ __launch_bounds__(1024) void gated_norm_long_kernel(ssm_gated_norm_args_t a, int64_t slots) {
    __shared__ SumSlots sums;
    int turn = 0;
    const TeamRows t = team_rows<0>(a.groups, slots);
    const int S = (int)(a.dim / a.groups);
    const int64_t col = t.g * S;
    for (int64_t row = t.row; row < a.rows; row += t.step) {
        const int64_t base = row * a.dim + col;
        float s = 0.0f;
        for (int i = threadIdx.x; i < S; i += 1024) {
            const float x = load_io<IO>(a.x, base + i), v = FIRST ? x * silu(load_io<IO>(a.z, base + i)) : x;
            s = __builtin_fmaf(v, v, s);
        }
        const float q = inv_rms(team_sum<0>(s, sums, turn), 1.0f / (float)S, a.eps);
        for (int i = threadIdx.x; i < S; i += 1024)
            store_io<IO>(a.y, base + i,
                         load_io<IO>(a.x, base + i) * silu(load_io<IO>(a.z, base + i)) * (q * a.w[col + i]));
    }
}

template <typename IO, bool FIRST>
__global__ __launch_bounds__(1024) void gated_norm_bwd_long_kernel(ssm_gated_norm_bwd_args_t a, int64_t slots,
                                                                   float *part) {
    __shared__ SumSlots sums;
    int turn = 0;
    const TeamRows t = team_rows<0>(a.groups, slots);
    const int S = (int)(a.dim / a.groups);
    const float inv_n = 1.0f / (float)S;
    const int64_t col = t.g * S;
    float *pw = part + t.row * a.dim + col;
    for (int64_t row = t.row; row < a.rows; row += t.step) {
        const int64_t base = row * a.dim + col;
        float s = 0.0f, dot = 0.0f;
        for (int i = threadIdx.x; i < S; i += 1024) {
            const float x = load_io<IO>(a.x, base + i), g = silu(load_io<IO>(a.z, base + i)), v = FIRST ? x * g : x;
            const float dy = load_io<IO>(a.dy, base + i);
            s = __builtin_fmaf(v, v, s);
            dot = __builtin_fmaf((FIRST ? dy : dy * g) * a.w[col + i], v, dot);
        }
        team_sum<0>(s, dot, sums, turn);
        const float q = inv_rms(s, inv_n, a.eps), m = dot * inv_n * q * q * q;
        for (int i = threadIdx.x; i < S; i += 1024) {
            const float x = load_io<IO>(a.x, base + i), z = load_io<IO>(a.z, base + i), dy = load_io<IO>(a.dy, base + i);
            const float sg = logistic(z), g = z * sg, slope = sg * __builtin_fmaf(z, 1.0f - sg, 1.0f);
            const float qw = q * a.w[col + i], dv = __builtin_fmaf(qw, FIRST ? dy : dy * g, -m * (FIRST ? x * g : x));
            store_io<IO>(a.dx, base + i, FIRST ? dv * g : dv);
            store_io<IO>(a.dz, base + i, FIRST ? dv * x * slope : dy * x * qw * slope);
            pw[i] = (row == t.row ? 0.0f : pw[i]) + dy * q * x * g;
        }
    }
}

constexpr int64_t kFwdBlocks = 2048, kLongBlocks = 256;

// Groups of 513 to 768 channels: half a wave with three groups of 8 a lane leaves fewer lanes idle
// than a wave with two, but each of its teams leaves a row of partial sums, which fall with the
// number of groups of a row.  Forward and backward in bf16, half waves against waves, in us: 16384 rows
// of 8 groups of 520 230 and 262, of 640 263 and 276, of 768 310 and 313; 32768 rows of 4 groups 231 and
// 261, 263 and 275, 311 and 314; of 1, 2 and 3 groups of 520 67, 123, 179 and 72, 137, 199, of 640 79, 141,
// 204 and 82, 145, 210, of 768 86, 160, 235 and 87, 159, 235.  (The backward's bound of 4 groups gives that
// much away below 4.)  Forward alone, 16384 rows: one group of 520 13.1 and 13.5, of 768 13.8 and 14.8;
// 8 groups 85 and 90, 114 and 118.
bool half_wave(int64_t S) { return S > 512 && S <= 768; }

int bwd_team(int64_t S, int64_t groups) {
    if (half_wave(S) && groups >= 4) return 32;
    return S <= 64 ? 8 : S <= 256 ? 32 : S <= 1024 ? 64 : 0;
}

RowGrid bwd_grid(int64_t rows, int64_t S, int64_t groups) {
    return row_grid(bwd_team(S, groups), std::min<int64_t>(S, kBlockRow), rows, groups,
                    S > kBlockRow ? kLongBlocks : bwd_blocks(S));
}

int64_t partial_rows(int64_t rows, int64_t S, int64_t groups) {
    const RowGrid g = bwd_grid(rows, S, groups);
    return bwd_team(S, groups) == 64 ? g.blocks / groups : g.slots;
}

}  // namespace

hipError_t launch_gated_norm_fwd(const ssm_gated_norm_args_t &a, hipStream_t stream) {
    const int64_t S = a.dim / a.groups;
    auto with = [&](auto io, auto first) {
        using IO = decltype(io);
        constexpr bool FIRST = decltype(first)::value;
        auto go = [&](auto sh) {
            using SH = decltype(sh);
            const RowGrid g = row_grid(SH::TEAM, S, a.rows, a.groups, kFwdBlocks);
            gated_norm_kernel<IO, FIRST, SH><<<g.blocks, g.threads, 0, stream>>>(a, g.slots);
        };
        if (S <= 64) go(Shape<8, 1>{});
        else if (S <= 256) go(Shape<32, 1>{});
        else if (S <= 512) go(Shape<64, 1>{});
        else if (half_wave(S)) go(Shape<32, 3>{});
        else if (S <= 1024) go(Shape<64, 2>{});
        else if (S <= 2048) go(Shape<64, 4>{});
        else if (S <= 4096) go(Shape<0, 1, 512>{});
        else if (S <= kBlockRow) go(Shape<0, 1, 1024>{});
        else {
            const RowGrid g = row_grid(0, kBlockRow, a.rows, a.groups, kFwdBlocks);
            gated_norm_long_kernel<IO, FIRST><<<g.blocks, 1024, 0, stream>>>(a, g.slots);
        }
    };
    auto with_io = [&](auto io) {
        if (a.gate_first)
            with(io, std::true_type{});
        else
            with(io, std::false_type{});
    };
    if (a.io_dtype == SSM_BF16)
        with_io(io_bf16{});
    else
        with_io(io_f32{});
    return hipGetLastError();
}

size_t gated_norm_bwd_workspace_bytes(const ssm_gated_norm_bwd_args_t &a) {
    const int64_t n = partial_rows(a.rows, a.dim / a.groups, a.groups);
    return (((size_t)(n * a.dim) * 4 + 255) & ~(size_t)255) + column_sums_scratch_bytes(n, a.dim, 1);
}

hipError_t launch_gated_norm_bwd(const ssm_gated_norm_bwd_args_t &a, hipStream_t stream) {
    const int64_t S = a.dim / a.groups, n = partial_rows(a.rows, S, a.groups);
    const RowGrid g = bwd_grid(a.rows, S, a.groups);
    float *part = static_cast<float *>(a.workspace);
    auto with = [&](auto io, auto first) {
        using IO = decltype(io);
        constexpr bool FIRST = decltype(first)::value;
        auto go = [&](auto sh) {
            gated_norm_bwd_kernel<IO, FIRST, decltype(sh)><<<g.blocks, g.threads, 0, stream>>>(a, g.slots, part);
        };
        if (S <= 64) go(Shape<8, 1>{});
        else if (S <= 256) go(Shape<32, 1>{});
        else if (S <= 512) go(Shape<64, 1>{});
        else if (bwd_team(S, a.groups) == 32) go(Shape<32, 3>{});
        else if (S <= 1024) go(Shape<64, 2>{});
        else if (S <= 4096) go(Shape<0, 1, 512>{});
        else if (S <= kBlockRow) go(Shape<0, 1, 1024>{});
        else gated_norm_bwd_long_kernel<IO, FIRST><<<g.blocks, 1024, 0, stream>>>(a, g.slots, part);
    };
    auto with_io = [&](auto io) {
        if (a.gate_first)
            with(io, std::true_type{});
        else
            with(io, std::false_type{});
    };
    if (a.io_dtype == SSM_BF16)
        with_io(io_bf16{});
    else
        with_io(io_f32{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    float *out[1] = {a.dw};
    char *scratch = static_cast<char *>(a.workspace) + (((size_t)(n * a.dim) * 4 + 255) & ~(size_t)255);
    return launch_column_sums(part, n, a.dim, 1, out, reinterpret_cast<float *>(scratch), stream);
}

}  // namespace ssm
