// norm_rows.h -- how the fused norms walk over rows (gfx950): teams, sums over a team, launch
// shapes.  A "row" here is what one mean square is taken over: a row of the tensor, or a group
// of its channels.
//
// A team of lanes owns a row, groups of 8 elements (or 4) a lane, read once into registers:
//   rows of up to 256      8 or 32 lanes, several rows a wave (adjacent groups side by side)
//   513 to 768             32 lanes of 3 groups (forwards; the gated backward over four groups or more)
//   up to 2048             one wave of up to 4 groups a lane: sums without a barrier (backwards up
//                          to 1024, whose column sums take registers too)
//   up to kBlockRow        one workgroup of as many waves as the row needs, one group a lane
//   longer                 one workgroup of 1024, reading the row again for each of its passes
// A team keeps its columns over all its rows, so the weights stay in registers and the
// gradients of the weights add up there.
#pragma once

#include <algorithm>

#include "ssm_internal.h"
#include "wide_io.h"

namespace ssm {

constexpr int kBlockRow = 8192;   // longest row held in a workgroup's registers
constexpr int kTeamThreads = 256; // workgroup of the teams of up to a wave

// TEAM lanes (1 << n up to 64, or 0: the workgroup, of at most THREADS) with NR groups of E each.
template <int TEAM_, int NR_, int THREADS_ = kTeamThreads, int E_ = 8>
struct Shape {
    static constexpr int TEAM = TEAM_, NR = NR_, THREADS = THREADS_, E = E_;
};

template <int TEAM>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int s = TEAM / 2; s >= 1; s /= 2) v += __shfl_xor(v, s, 64);
    return v;
}

// Sums over the team, of one or two values.  For a workgroup: through LDS with one barrier; the
// slots alternate, so that a wave still reading one sum meets no write of the next.
struct SumSlots {
    float v[2][2][16];
};

template <int TEAM>
__device__ __forceinline__ void team_sum(float &a, float &b, SumSlots &s, int &turn) {
    a = lanes_sum<TEAM == 0 ? 64 : TEAM>(a);
    b = lanes_sum<TEAM == 0 ? 64 : TEAM>(b);
    if constexpr (TEAM == 0) {
        const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            s.v[turn][0][wave] = a;
            s.v[turn][1][wave] = b;
        }
        __syncthreads();
        a = b = 0.0f;
        for (int i = 0; i < waves; ++i) {
            a += s.v[turn][0][i];
            b += s.v[turn][1][i];
        }
        turn ^= 1;
    }
}

template <int TEAM>
__device__ __forceinline__ float team_sum(float a, SumSlots &s, int &turn) {
    float b = 0.0f;
    team_sum<TEAM>(a, b, s, turn);
    return a;
}

__device__ __forceinline__ float inv_rms(float sum, float inv_n, float eps) {
    return 1.0f / sqrtf(__builtin_fmaf(sum, inv_n, eps));
}

// E weights (the first n of them) as floats.
template <int E>
__device__ __forceinline__ void load_vec(const float *p, int64_t i, int n, float (&w)[E]) {
    const Raw<io_f32, E> r = load_raw<io_f32, E>(p, i, n);
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = r[e];
}

// Column sums of the waves of a workgroup that hold the same columns: into wave 0's registers.
template <int NR>
__device__ __forceinline__ void waves_sum(float (&v)[NR][8], float *lds, int lane) {
    constexpr int W = kTeamThreads / 64;
    const int wave = threadIdx.x / 64;
#pragma unroll
    for (int c = 0; c < NR; ++c) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) lds[(wave * 8 + e) * 64 + lane] = v[c][e];
        __syncthreads();
        if (wave == 0)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                for (int i = 1; i < W; ++i) v[c][e] += lds[(i * 8 + e) * 64 + lane];
    }
}

// The rows of a team: group `g` of every row from `row` on, `step` apart.
struct TeamRows {
    int64_t g, row, step;
};

// How many workgroups, and over how many rows of the tensor they run at once (`slots`, the rows
// of partial sums too).
struct RowGrid {
    unsigned blocks, threads;
    int64_t slots;
};

// Team sizes of up to half a wave put the groups of a tensor row side by side; a wave or a
// workgroup takes one group (blockIdx % groups).
template <int TEAM>
__device__ __forceinline__ TeamRows team_rows(int64_t groups, int64_t slots) {
    if constexpr (TEAM == 0) return {blockIdx.x % groups, blockIdx.x / groups, slots};
    if constexpr (TEAM == 64) {
        const int64_t slot = blockIdx.x / groups * (kTeamThreads / 64) + threadIdx.x / 64;
        return {blockIdx.x % groups, slot, slots};
    }
    const int64_t t = (int64_t)blockIdx.x * (kTeamThreads / TEAM) + threadIdx.x / TEAM;
    const int64_t slot = t / groups;
    return {t % groups, slot < slots ? slot : (int64_t)1 << 62, slots};  // spare teams: no rows
}

// Workgroups of a backward: as many as run at once, since each walks over rows to its end.  With 8
// elements a lane a row of up to 2048 takes at most one wave of a SIMD, one of up to 4096 two, and the
// kernels' registers leave room for four.  Training steps of 16384 rows in bf16 with 512, 768, 1024 and
// 2048 workgroups: 1280 with a post norm and scale 153, 127, 112, 117 us, 2048 156, 138, 138, 149; plain
// 1280 107, 94, 86, 82, 2048 127, 127, 133, 141; of 2560 184 with 512, 220 with 768; 8192 rows of 5120 231
// with 512, 226 with 256.  fp32 rows of 1025 to 2048 of the add + norm hold 4 elements a lane, five to
// eight waves a row, and would be served as well or better by 512: 1280 168 against 173 us with 1024 (with
// post norm and scale 179, 187), 2048 259 against 272 (260, 282).
inline int64_t bwd_blocks(int64_t len) { return len <= 1024 ? 512 : len <= 2048 ? 1024 : len <= 4096 ? 512 : 256; }

// `blocks_wanted`: workgroups that keep the chip busy; E: elements of a lane's group.
inline RowGrid row_grid(int team, int64_t len, int64_t rows, int64_t groups, int64_t blocks_wanted, int E = 8) {
    RowGrid g;
    if (team == 0 || team == 64) {
        const int64_t per = team == 0 ? 1 : kTeamThreads / 64;
        const int64_t most = (rows + per - 1) / per, want = std::max<int64_t>(1, blocks_wanted / groups);
        const int64_t n = std::min(most, want);
        g.blocks = (unsigned)(n * groups);
        g.slots = n * per;
        g.threads = team == 0 ? (unsigned)std::min<int64_t>(1024, (len + 64 * E - 1) / (64 * E) * 64) : kTeamThreads;
    } else {
        const int64_t per = kTeamThreads / team;  // teams of a workgroup
        const int64_t most = (rows * groups + per - 1) / per, least = (groups + per - 1) / per;
        const int64_t n = std::max(least, std::min(most, blocks_wanted));
        g.blocks = (unsigned)n;
        g.slots = n * per / groups;
        g.threads = kTeamThreads;
    }
    return g;
}

}  // namespace ssm
