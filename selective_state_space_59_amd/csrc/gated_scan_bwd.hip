// gated_scan_bwd.hip -- gradients of the gated linear recurrence on gfx950.
//
// With mu_t = a_t lambda_t (0 at a reset) the adjoint is a recurrence of the same decays, run
// backwards:
//   lambda_t = dy_t + mu_{t+1},  mu_t = a_t (dy_t + mu_{t+1}),  mu_L = dh_final,  dh0 = mu_0
//   da_t = lambda_t h_{t-1},  db_t = lambda_t,  and the chain rule of gated_device.h.
//
// One pass over HBM: x, gate, in_gate and dy are read once, dx, dgate and din_gate written once.  The
// tiles are the forward's (gated_tile.h), one checkpoint long or a whole shorter sequence, and chained
// from the last to the first.  A tile recomputes its states from its checkpoint in fp32, so neither y
// nor any state is read, and both directions share the product p of a lane's decays.  The rows stay in
// registers as they were read; a channel at a time is widened, its gates formed (once for the lane's
// run, once for its gradients: arithmetic is cheaper here than registers), and its gradients packed
// into the place of its inputs.
//
// Measured in bf16: 8 x 2048 x 1536 RATE with in_gate 91 us, 3.9 TB/s, bound by the issue of its 92
// vector instructions an element (13 of them exponentials, reciprocals and roots; 37% of the waves'
// cycles wait to issue, 33% otherwise); 4 x 4096 x 5120 SIGMOID with resets 180 us, 4.7 TB/s, 97
// registers, four waves a SIMD, where 52% of the cycles wait for the tile's phases.  Training steps in
// fp32, 8 x 2048 x 2560: SIGMOID 311 us, RATE with in_gate 431 us, four waves a SIMD.
//
// The launch bound holds bf16 RATE with in_gate at 128 registers, four waves a SIMD, and its lanes keep
// 24 bytes in scratch (32 at most, by width and length).  Without the bound or with three waves the
// layer's training step takes 158 us against 156; the other variants need at most 123 registers.
#include "gated_tile.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr int kBwdSteps = 128;
template <typename IO, int STEPS = kBwdSteps>
using BwdTile = Tile<IO, 4, 4, STEPS * 2>;
static_assert(BwdTile<io_bf16>::T == kBwdSteps && BwdTile<io_f32>::T == kBwdSteps, "tile sizes");
static_assert(kBwdSteps % SSM_GATED_BLOCK == 0, "a tile begins at a checkpoint");

template <bool IG>
__device__ __forceinline__ void pin_row(uint32_t &x, uint32_t &g, uint32_t &i, uint32_t &d) {
    asm volatile("" : "+v"(x), "+v"(g), "+v"(d));
    if constexpr (IG) asm volatile("" : "+v"(i));
}

template <typename IO, int MODE, bool IG, bool SPECIAL, int EDGE, int STEPS>
__global__ __launch_bounds__((BwdTile<IO, STEPS>::THREADS), 4) void gated_bwd_kernel(
    ssm_gated_scan_bwd_args_t a, const float *ck, float *part, int chains, int tiles, u64_t *rec, unsigned *tickets) {
    using TL = BwdTile<IO, STEPS>;
    constexpr int V = TL::V, CB = TL::CB, G = TL::G, R = TL::R, W = TL::W, T = TL::T;
    constexpr int PER = V / W;  // channels of a word
    // the groups' decay products, forward runs and backward runs; later their entering states
    // and the partial sums
    constexpr int NP = TL::THREADS / CB, GP = G / NP;  // runs of GP lane groups
    __shared__ __attribute__((aligned(16))) float sp[G][CB], sl[G][CB], sm[G][CB], pp[NP][CB], pl[NP][CB], pm[NP][CB],
        sc[3][CB];
    __shared__ int s_ticket;
    const int tid = threadIdx.x, chain = chain_of(blockIdx.x, chains, tiles);
    const int nblk = (int)((a.dim + CB - 1) / CB), cblk = chain % nblk;
    if (tid == 0) s_ticket = tiles > 1 ? (int)atomicAdd(&tickets[chain], 1u) : 0;
    if (tid < CB) {
        const int d = min(cblk * CB + tid, (int)a.dim - 1);
        sc[0][tid] = MODE == SSM_GATE_RATE ? a.A[d] * kLog2e : 0.0f;
        sc[1][tid] = MODE != SSM_GATE_DECAY && a.gate_bias ? a.gate_bias[d] * kLog2e : 0.0f;
        sc[2][tid] = IG && a.in_bias ? a.in_bias[d] * kLog2e : 0.0f;
    }
    __syncthreads();
    const int k = s_ticket;
    const int tile = tiles - 1 - k;
    const int64_t b = chain / nblk, L = a.seqlen, t0 = (int64_t)tile * T;
    const int D = (int)a.dim, lc = tid % TL::LANES * V, g = tid / TL::LANES;
    const Cols col = cols_of<EDGE>(cblk * CB + lc, D, V);
    const int left = (int)min(L - t0, (int64_t)T);
    const int64_t row0 = (b * L + t0) * D * IO::bytes;
    uint32_t off[R];
#pragma unroll
    for (int j = 0; j < R; ++j)
        off[j] = ((uint32_t)min(g * R + j, left - 1) * (uint32_t)D + (uint32_t)col.load) * IO::bytes;
    uint32_t mark[R] = {};  // ahead of the rows: loads come back in order
    if (SPECIAL && a.reset)
#pragma unroll
        for (int j = 0; j < R; ++j) mark[j] = a.reset[b * L + t0 + min(g * R + j, left - 1)];
    Words<W> qx[R], qg[R], qi[R], qd[R];
    load_rows<IO, EDGE>(static_cast<const char *>(a.x) + row0, off, col.nv, qx);
    load_rows<IO, EDGE>(static_cast<const char *>(a.gate) + row0, off, col.nv, qg);
    if constexpr (IG) load_rows<IO, EDGE>(static_cast<const char *>(a.in_gate) + row0, off, col.nv, qi);
    load_rows<IO, EDGE>(static_cast<const char *>(a.dy) + row0, off, col.nv, qd);
    if constexpr (EDGE == kRagged) {
        shift_rows<IO>(qx, col.shift);
        shift_rows<IO>(qg, col.shift);
        if constexpr (IG) shift_rows<IO>(qi, col.shift);
        shift_rows<IO>(qd, col.shift);
    }
    bool cut[R], in[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        cut[j] = mark[j] != 0;
        in[j] = g * R + j < left;
    }
    auto channel = [&](int v) { return GateChannel{sc[0][lc + v], sc[1][lc + v], sc[2][lc + v]}; };

    {
        float p[V], l[V], m[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const GateChannel c = channel(v);
            float at[R], bt[R];
#pragma unroll
            for (int j = 0; j < R; ++j)
                gate_step<MODE, IG>(lane_elem<IO>(qx[j], v), lane_elem<IO>(qg[j], v),
                                    IG ? lane_elem<IO>(qi[j], v) : 0.0f, c, at[j], bt[j]);
            p[v] = 1.0f;
            l[v] = m[v] = 0.0f;
            if constexpr (!SPECIAL) {
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    l[v] = __builtin_fmaf(at[j], l[v], bt[j]);
                    p[v] *= at[j];
                    m[v] = at[R - 1 - j] * (lane_elem<IO>(qd[R - 1 - j], v) + m[v]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    l[v] = !in[j] ? l[v] : cut[j] ? bt[j] : __builtin_fmaf(at[j], l[v], bt[j]);
                    p[v] = !in[j] ? p[v] : cut[j] ? __builtin_nanf("") : at[j] * p[v];
                }
#pragma unroll
                for (int j = R - 1; j >= 0; --j)
                    m[v] = !in[j] ? m[v] : cut[j] ? 0.0f : at[j] * (lane_elem<IO>(qd[j], v) + m[v]);
            }
            __builtin_amdgcn_sched_barrier(0);  // a channel at a time: fewer live registers
        }
        lds_put<V>(&sp[g][lc], p);
        lds_put<V>(&sl[g][lc], l);
        lds_put<V>(&sm[g][lc], m);
    }
    __syncthreads();
    // a thread per channel and run of GP groups: the runs first, then one thread per channel over
    // the runs, and out to the groups again
    {
        const int ch = tid % CB, pt = tid / CB, d = cblk * CB + ch;
        float tp = 1.0f, tl = 0.0f, tm = 0.0f;
#pragma unroll
        for (int i = 0; i < GP; ++i) {
            const int f = pt * GP + i, r = pt * GP + GP - 1 - i;
            tl = run_apply<MODE>(sp[f][ch], sl[f][ch], tl);
            tm = run_apply<MODE>(sp[r][ch], sm[r][ch], tm);
            tp *= sp[f][ch];
        }
        pp[pt][ch] = tp;
        pl[pt][ch] = tl;
        pm[pt][ch] = tm;
        __syncthreads();
        if (pt == 0) {
            tp = 1.0f;
            tm = 0.0f;
#pragma unroll
            for (int i = NP - 1; i >= 0; --i) {
                tm = run_apply<MODE>(pp[i][ch], pm[i][ch], tm);
                tp *= pp[i][ch];
            }
            u64_t *mine = rec + ((int64_t)chain * tiles + k) * CB + ch;
            if (k > 0 && k + 1 < tiles) rec_put(mine, rec_hi(tp), tm);
            float h = d < D ? ck[(t0 / SSM_GATED_BLOCK * a.batch + b) * D + d] : 0.0f;
            float mu = k == 0 && a.dh_final && d < D ? a.dh_final[b * D + d] : 0.0f;
            if (k > 0) mu = chain_enter<MODE>(mine, CB, k);
            const float after = run_apply<MODE>(tp, tm, mu);
            if (k + 1 < tiles)
                rec_put(mine, kRecState, after);
            else if (a.dh0 && d < D)
                a.dh0[b * D + d] = after;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float l = pl[i][ch];
                pl[i][ch] = h;
                h = run_apply<MODE>(pp[i][ch], l, h);
            }
#pragma unroll
            for (int i = NP - 1; i >= 0; --i) {
                const float m = pm[i][ch];
                pm[i][ch] = mu;
                mu = run_apply<MODE>(pp[i][ch], m, mu);
            }
        }
        __syncthreads();
        float h = pl[pt][ch], mu = pm[pt][ch];
#pragma unroll
        for (int i = 0; i < GP; ++i) {
            const float l = sl[pt * GP + i][ch];
            sl[pt * GP + i][ch] = h;
            h = run_apply<MODE>(sp[pt * GP + i][ch], l, h);
        }
#pragma unroll
        for (int i = GP - 1; i >= 0; --i) {
            const float m = sm[pt * GP + i][ch];
            sm[pt * GP + i][ch] = mu;
            mu = run_apply<MODE>(sp[pt * GP + i][ch], m, mu);
        }
    }
    __syncthreads();
    // What follows forms the gates again from the rows.  The empty asm statements keep the
    // compiler from carrying gates over from above, and from putting a word's gradients off until
    // the stores: either would double the registers.
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int w = 0; w < W; ++w) pin_row<IG>(qx[j].w[w], qg[j].w[w], qi[j].w[w], qd[j].w[w]);
#pragma unroll
    for (int w = 0; w < W; ++w) {
        float ox[R][PER], og[R][PER], oi[R][PER];
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int v = w * PER + u;
            const GateChannel c = channel(v);
            float h = sl[g][lc + v], mu = sm[g][lc + v], da[R], lam[R], sA = 0.0f, sg = 0.0f, si = 0.0f;
            const float A = c.A2 * 0.69314718055994531f;
            Gate<MODE, IG> t[R];
#pragma unroll
            for (int j = 0; j < R; ++j)
                t[j] = gate_of<MODE, IG>(lane_elem<IO>(qg[j], v), IG ? lane_elem<IO>(qi[j], v) : 0.0f, c);
            if constexpr (!SPECIAL) {
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    da[j] = h;
                    h = __builtin_fmaf(t[j].a, h, t[j].w * lane_elem<IO>(qx[j], v));
                }
#pragma unroll
                for (int j = R - 1; j >= 0; --j) {
                    lam[j] = lane_elem<IO>(qd[j], v) + mu;
                    da[j] *= lam[j];
                    mu = t[j].a * lam[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    da[j] = h;
                    const float b = t[j].w * lane_elem<IO>(qx[j], v);
                    h = cut[j] ? b : __builtin_fmaf(t[j].a, h, b);
                }
#pragma unroll
                for (int j = R - 1; j >= 0; --j) {  // steps past the end: no gradient
                    lam[j] = in[j] ? lane_elem<IO>(qd[j], v) + mu : 0.0f;
                    da[j] = cut[j] || !in[j] ? 0.0f : da[j] * lam[j];
                    mu = !in[j] ? mu : cut[j] ? 0.0f : t[j].a * lam[j];
                }
            }
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const GateGrad o = gate_grad<MODE, IG>(t[j], lane_elem<IO>(qx[j], v), A, da[j], lam[j]);
                ox[j][u] = o.dx;
                og[j][u] = o.dg;
                oi[j][u] = o.di;
                sA += o.dA;
                sg += o.dg;
                si += o.di;
            }
            if constexpr (MODE != SSM_GATE_DECAY) {
                // this lane's own words: read above, by no other lane
                sp[g][lc + v] = sg;
                if constexpr (MODE == SSM_GATE_RATE) sl[g][lc + v] = sA;
                if constexpr (IG) sm[g][lc + v] = si;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if constexpr (IO::bytes == 2) {
                qx[j].w[w] = pack_bf16x2(ox[j][0], ox[j][PER - 1]);
                qg[j].w[w] = pack_bf16x2(og[j][0], og[j][PER - 1]);
                if constexpr (IG) qi[j].w[w] = pack_bf16x2(oi[j][0], oi[j][PER - 1]);
            } else {
                qx[j].w[w] = __float_as_uint(ox[j][0]);
                qg[j].w[w] = __float_as_uint(og[j][0]);
                if constexpr (IG) qi[j].w[w] = __float_as_uint(oi[j][0]);
            }
            pin_row<IG>(qx[j].w[w], qg[j].w[w], qi[j].w[w], qd[j].w[w]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
        if (!SPECIAL || in[j]) {
            const uint32_t at = off[j] + col.shift * IO::bytes;
            store_row<IO>(static_cast<char *>(a.dx) + row0 + at, col.nv, qx[j]);
            store_row<IO>(static_cast<char *>(a.dgate) + row0 + at, col.nv, qg[j]);
            if constexpr (IG) store_row<IO>(static_cast<char *>(a.din_gate) + row0 + at, col.nv, qi[j]);
        }
    if constexpr (MODE != SSM_GATE_DECAY) {
        // this tile's row of the partial sums: gate_bias, then A, then in_bias
        __syncthreads();
        constexpr int K = MODE == SSM_GATE_SIGMOID ? 1 : IG ? 3 : 2;
        for (int i = tid; i < K * CB; i += TL::THREADS) {
            const int which = i / CB, ch = i % CB, d = cblk * CB + ch;
            if (d >= D) continue;
            const float(*s)[CB] = which == 0 ? sp : which == 1 ? sl : sm;
            float v = 0.0f;
#pragma unroll 8
            for (int j = 0; j < G; ++j) v += s[j][ch];
            part[((int64_t)which * a.batch * tiles + b * tiles + tile) * D + d] = v;
        }
    }
}

struct BwdPlan {
    ChainPlan chain;
    int64_t rows;  // partial rows of each sum
    int sums;
    size_t o_part, o_scratch, o_ck, o_fwd, total;
};

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

// The workspace is sized without looking at which gradients are asked for.
BwdPlan plan_of(const ssm_gated_scan_bwd_args_t &a) {
    const int64_t cb = a.io_dtype == SSM_BF16 ? BwdTile<io_bf16>::CB : BwdTile<io_f32>::CB;
    const int64_t tiles = (a.seqlen + kBwdSteps - 1) / kBwdSteps;
    BwdPlan p;
    p.chain = ChainPlan{a.batch * ((a.dim + cb - 1) / cb), tiles, cb};
    p.rows = a.batch * tiles;
    p.sums = a.mode == SSM_GATE_DECAY ? 0 : a.mode == SSM_GATE_SIGMOID ? 1 : 3;
    size_t o = p.chain.bytes();
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) & ~(size_t)255;
        return at;
    };
    p.o_part = take((size_t)(p.sums * p.rows * a.dim) * 4);
    p.o_scratch = take(column_sums_scratch_bytes(p.rows, a.dim, p.sums));
    p.o_ck = p.o_fwd = o;
    if (!a.checkpoints) {
        p.o_ck = take((size_t)((a.seqlen + SSM_GATED_BLOCK - 1) / SSM_GATED_BLOCK * a.batch * a.dim) * 4);
        p.o_fwd = take(gated_scan_workspace_bytes(forward_of(a)));
    }
    p.total = o;
    return p;
}

}  // namespace

size_t gated_scan_bwd_workspace_bytes(const ssm_gated_scan_bwd_args_t &a) { return plan_of(a).total; }

hipError_t launch_gated_scan_bwd(const ssm_gated_scan_bwd_args_t &a, hipStream_t stream) {
    const BwdPlan p = plan_of(a);
    char *ws = static_cast<char *>(a.workspace);
    const float *ck = a.checkpoints;
    hipError_t e = hipSuccess;
    if (!ck) {
        ssm_gated_scan_args_t f = forward_of(a);
        f.checkpoints = reinterpret_cast<float *>(ws + p.o_ck);
        f.workspace = ws + p.o_fwd;
        ck = f.checkpoints;
        e = launch_gated_scan_fwd(f, stream);
    }
    if (e == hipSuccess && p.chain.tiles > 1) e = launch_chain_init(p.chain, ws, stream);
    if (e != hipSuccess) return e;
    float *part = reinterpret_cast<float *>(ws + p.o_part);
    unsigned *tickets = reinterpret_cast<unsigned *>(ws + p.chain.rec_bytes());
    const unsigned grid = (unsigned)(p.chain.chains * p.chain.tiles);
    gate_dispatch(a.io_dtype, a.mode, a.in_gate != nullptr, [&](auto io, auto mode, auto ig) {
        auto go = [&](auto special, auto edge, auto steps) {
            using TL = BwdTile<decltype(io), decltype(steps)::value>;
            gated_bwd_kernel<decltype(io), decltype(mode)::value, decltype(ig)::value, decltype(special)::value,
                             decltype(edge)::value, TL::T>
                <<<grid, TL::THREADS, 0, stream>>>(a, ck, part, (int)p.chain.chains, (int)p.chain.tiles,
                                                   reinterpret_cast<u64_t *>(ws), tickets);
        };
        // the selects for resets and for a cut-off last tile: left out where neither is there and
        // the width is whole
        const Edge edge = edge_of(a.dim, BwdTile<decltype(io)>::V);
        if (edge == kWhole && !a.reset && a.seqlen % kBwdSteps == 0)
            go(std::false_type{}, std::integral_constant<int, kWhole>{}, std::integral_constant<int, kBwdSteps>{});
        else
            with_edge(edge, [&](auto e) {
                with_steps<kBwdSteps>(a.seqlen, [&](auto steps) { go(std::true_type{}, e, steps); });
            });
    });
    e = hipGetLastError();
    float *out[3] = {a.dgate_bias, a.dA, a.din_bias};
    if (e == hipSuccess && p.sums > 0 && (out[0] || out[1] || out[2]))
        e = launch_column_sums(part, p.rows, a.dim, p.sums, out, reinterpret_cast<float *>(ws + p.o_scratch), stream);
    return e;
}

}  // namespace ssm
