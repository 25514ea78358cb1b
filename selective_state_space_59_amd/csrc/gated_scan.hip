// gated_scan.hip -- the gated linear recurrence h_t = a_t h_{t-1} + b_t, forward and
// decode step, on gfx950 (gated_device.h has the gates, gated_tile.h the hand-over of states).
//
// Bound by HBM: x, gate and in_gate are read once, y is written once.  The sequence is cut into
// tiles of kRowGroups * R steps by 128 bytes of channels, one workgroup each, so that a layer
// with few channels still fills the chip.  In a tile a lane owns R consecutive steps of 16 bytes
// of channels: all its loads are issued at once, whole 128-byte lines per 8 lanes, and its steps
// run in registers from a zero state, keeping per step the state l and the product p of the
// decays.  The lane groups' (p, l) meet in LDS, where one wave, a lane per channel, runs over
// them, fetches the state that enters the tile (chain_enter) and leaves each group's entering
// state; y = p h + l then costs one fma per element and no second read.
#include <algorithm>

#include "gated_tile.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr int kFwdRows = 4;  // R

template <typename IO, int MODE, bool IG, int R>
__global__ __launch_bounds__(kGatedThreads) void gated_scan_kernel(ssm_gated_scan_args_t a, int chains, int tiles,
                                                                   u64_t *rec, unsigned *tickets) {
    constexpr int V = TileShape<IO>::V, CB = TileShape<IO>::CB, G = kRowGroups, T = G * R;
    __shared__ __attribute__((aligned(16))) float sp[G][CB], sl[G][CB];
    __shared__ int s_tile;
    const int tid = threadIdx.x;
    // consecutive workgroups take different chains, so that a chain stays on one XCD where the
    // number of chains is a multiple of 8
    const int chain = blockIdx.x % chains;
    int tile = 0;
    if (tiles > 1) {
        if (tid == 0) s_tile = (int)atomicAdd(&tickets[chain], 1u);
        __syncthreads();
        tile = s_tile;
    }
    const int nblk = (int)((a.dim + CB - 1) / CB);
    const int cblk = chain % nblk;
    const int64_t b = chain / nblk, L = a.seqlen, t0 = (int64_t)tile * T;
    const int D = (int)a.dim, d0 = cblk * CB + (tid % kLanesPerRow) * V, nv = min(V, D - d0), g = tid / kLanesPerRow;
    const int left = (int)min(L - t0, (int64_t)T);  // valid steps of this tile

    GateChannel c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int d = min(d0 + v, D - 1);
        c[v].A = MODE == SSM_GATE_RATE ? a.A[d] : 0.0f;
        c[v].gb = MODE != SSM_GATE_DECAY && a.gate_bias ? a.gate_bias[d] : 0.0f;
        c[v].ib = IG && a.in_bias ? a.in_bias[d] : 0.0f;
    }
    const int64_t row0 = (b * L + t0) * D * IO::bytes;
    uint32_t off[R];
#pragma unroll
    for (int j = 0; j < R; ++j)  // steps past the end read the last one and are made the identity below
        off[j] = ((uint32_t)min(g * R + j, left - 1) * (uint32_t)D + (uint32_t)d0) * IO::bytes;
    u32x4_t qx[R], qg[R], qi[R];
    load_rows<IO, R>(static_cast<const char *>(a.x) + row0, off, nv, qx);
    load_rows<IO, R>(static_cast<const char *>(a.gate) + row0, off, nv, qg);
    if constexpr (IG) load_rows<IO, R>(static_cast<const char *>(a.in_gate) + row0, off, nv, qi);
    bool cut[R];
#pragma unroll
    for (int j = 0; j < R; ++j) cut[j] = a.reset && a.reset[b * L + t0 + min(g * R + j, left - 1)] != 0;

    float p[R][V], l[R][V];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const bool in = g * R + j < left;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float at, bt;
            gate_step<MODE, IG>(lane_elem<IO>(qx[j], v), lane_elem<IO>(qg[j], v), IG ? lane_elem<IO>(qi[j], v) : 0.0f,
                                c[v], at, bt);
            const float pp = j ? p[j - 1][v] : 1.0f, pl = j ? l[j - 1][v] : 0.0f;
            p[j][v] = !in ? pp : cut[j] ? __builtin_nanf("") : at * pp;
            l[j][v] = !in ? pl : cut[j] ? bt : __builtin_fmaf(at, pl, bt);
        }
    }
#pragma unroll
    for (int v = 0; v < V; v += 4) {
        const int ch = (tid % kLanesPerRow) * V + v;
        *reinterpret_cast<float4 *>(&sp[g][ch]) = make_float4(p[R - 1][v], p[R - 1][v + 1], p[R - 1][v + 2], p[R - 1][v + 3]);
        *reinterpret_cast<float4 *>(&sl[g][ch]) = make_float4(l[R - 1][v], l[R - 1][v + 1], l[R - 1][v + 2], l[R - 1][v + 3]);
    }
    __syncthreads();
    if (tid < CB) {
        const int d = cblk * CB + tid;
        float tp = 1.0f, tl = 0.0f;
#pragma unroll 8
        for (int i = 0; i < G; ++i) {
            const float p = sp[i][tid];
            tl = run_apply(p, sl[i][tid], tl);
            tp *= p;
        }
        float h = tile == 0 && a.h0 && d < D ? a.h0[b * D + d] : 0.0f;
        u64_t *mine = rec + ((int64_t)chain * tiles + tile) * CB + tid;
        if (tile > 0) {
            if (tile + 1 < tiles) rec_put(mine, rec_hi(tp), tl);
            h = chain_enter(mine, CB, tile);
        }
        const float after = run_apply(tp, tl, h);
        if (tile + 1 < tiles)
            rec_put(mine, kRecState, after);
        else if (a.h_final && d < D)
            a.h_final[b * D + d] = after;
#pragma unroll 8
        for (int i = 0; i < G; ++i) {
            if (i * R % SSM_GATED_BLOCK == 0 && a.checkpoints && d < D && i * R < left)
                a.checkpoints[((t0 + i * R) / SSM_GATED_BLOCK * a.batch + b) * D + d] = h;
            const float p = sp[i][tid];
            sp[i][tid] = h;
            h = run_apply(p, sl[i][tid], h);
        }
    }
    __syncthreads();
    if (a.y) {
        float e[V];
#pragma unroll
        for (int v = 0; v < V; ++v) e[v] = sp[g][(tid % kLanesPerRow) * V + v];
        char *out = static_cast<char *>(a.y) + row0;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float f[V];
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = run_apply(p[j][v], l[j][v], e[v]);
            if (g * R + j < left) store_words<IO>(out + off[j], nv, lane_pack<IO>(f));
        }
    }
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

// Records to kRecEmpty, counters to 0.
__global__ __launch_bounds__(256) void chain_init_kernel(uint4 *rec, int64_t n16, unsigned *tickets, int chains) {
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n16; i += step)
        rec[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < chains; i += step) tickets[i] = 0;
}

ChainPlan fwd_plan(const ssm_gated_scan_args_t &a) {
    const int64_t cb = a.io_dtype == SSM_BF16 ? TileShape<io_bf16>::CB : TileShape<io_f32>::CB;
    const int64_t t = kRowGroups * kFwdRows;
    return ChainPlan{a.batch * ((a.dim + cb - 1) / cb), (a.seqlen + t - 1) / t, cb};
}

}  // namespace

static_assert(SSM_GATED_BLOCK % kFwdRows == 0 && kRowGroups * kFwdRows <= SSM_GATED_TILE, "tile and checkpoint sizes");
static_assert((kRowGroups * kFwdRows) % SSM_GATED_BLOCK == 0, "a tile begins at a checkpoint");

hipError_t launch_chain_init(const ChainPlan &p, void *workspace, hipStream_t stream) {
    const int64_t n16 = (int64_t)(p.rec_bytes() / 16);
    const unsigned blocks = (unsigned)std::min<int64_t>((std::max(n16, p.chains) + 255) / 256, 2048);
    chain_init_kernel<<<blocks, 256, 0, stream>>>(
        static_cast<uint4 *>(workspace), n16,
        reinterpret_cast<unsigned *>(static_cast<char *>(workspace) + p.rec_bytes()), (int)p.chains);
    return hipGetLastError();
}

size_t gated_scan_workspace_bytes(const ssm_gated_scan_args_t &a) { return fwd_plan(a).bytes(); }

hipError_t launch_gated_scan_fwd(const ssm_gated_scan_args_t &a, hipStream_t stream) {
    const ChainPlan p = fwd_plan(a);
    u64_t *rec = static_cast<u64_t *>(a.workspace);
    unsigned *tickets = reinterpret_cast<unsigned *>(static_cast<char *>(a.workspace) + p.rec_bytes());
    if (p.tiles > 1) {
        const hipError_t e = launch_chain_init(p, a.workspace, stream);
        if (e != hipSuccess) return e;
    }
    const unsigned grid = (unsigned)(p.chains * p.tiles);
    gate_dispatch(a.io_dtype, a.mode, a.in_gate != nullptr, [&](auto io, auto mode, auto ig) {
        gated_scan_kernel<decltype(io), decltype(mode)::value, decltype(ig)::value, kFwdRows>
            <<<grid, kGatedThreads, 0, stream>>>(a, (int)p.chains, (int)p.tiles, rec, tickets);
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
