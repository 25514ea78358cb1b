// gated_scan_bwd.hip -- gradients of the gated linear recurrence on gfx950.
//
// With mu_t = a_t lambda_t (0 at a reset) the adjoint is a recurrence of the same decays, run
// backwards:
//   lambda_t = dy_t + mu_{t+1},  mu_t = a_t (dy_t + mu_{t+1}),  mu_L = dh_final,  dh0 = mu_0
//   da_t = lambda_t h_{t-1},  db_t = lambda_t,  and the chain rule of gated_device.h.
//
// Bound by HBM: x, gate, in_gate and dy are read once, dx, dgate and din_gate written once.  The
// tiles are the forward's (gated_tile.h), one checkpoint long, and chained from the last to the
// first.  A tile recomputes its states from its checkpoint in fp32, so neither y nor any state is
// read, and both directions share the product p of a lane's decays.  The rows stay in registers
// as they were read; a channel at a time is widened, its gates formed (once for the lane's run,
// once for its gradients: arithmetic is cheaper here than registers), and its gradients packed
// into the place of its inputs.
#include "gated_tile.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr int R = 4, G = kRowGroups, T = G * R;
static_assert(T == SSM_GATED_BLOCK, "a tile begins at its checkpoint");

template <typename IO, int MODE, bool IG>
__global__ __launch_bounds__(kGatedThreads) void gated_bwd_kernel(ssm_gated_scan_bwd_args_t a, const float *ck,
                                                                  float *part, int chains, int tiles, u64_t *rec,
                                                                  unsigned *tickets) {
    constexpr int V = TileShape<IO>::V, CB = TileShape<IO>::CB, PER = V / 4;  // channels of a register
    // the groups' decay products, forward runs and backward runs; later their entering states
    // and the partial sums
    __shared__ __attribute__((aligned(16))) float sp[G][CB], sl[G][CB], sm[G][CB];
    __shared__ int s_ticket;
    const int tid = threadIdx.x, chain = blockIdx.x % chains;
    int k = 0;
    if (tiles > 1) {
        if (tid == 0) s_ticket = (int)atomicAdd(&tickets[chain], 1u);
        __syncthreads();
        k = s_ticket;
    }
    const int tile = tiles - 1 - k;
    const int nblk = (int)((a.dim + CB - 1) / CB), cblk = chain % nblk;
    const int64_t b = chain / nblk, L = a.seqlen, t0 = (int64_t)tile * T;
    const int D = (int)a.dim, lc = (tid % kLanesPerRow) * V, d0 = cblk * CB + lc, nv = min(V, D - d0);
    const int g = tid / kLanesPerRow, left = (int)min(L - t0, (int64_t)T);
    const int64_t row0 = (b * L + t0) * D * IO::bytes;
    uint32_t off[R];
#pragma unroll
    for (int j = 0; j < R; ++j)
        off[j] = ((uint32_t)min(g * R + j, left - 1) * (uint32_t)D + (uint32_t)d0) * IO::bytes;
    u32x4_t qx[R], qg[R], qi[R], qd[R];
    load_rows<IO, R>(static_cast<const char *>(a.x) + row0, off, nv, qx);
    load_rows<IO, R>(static_cast<const char *>(a.gate) + row0, off, nv, qg);
    if constexpr (IG) load_rows<IO, R>(static_cast<const char *>(a.in_gate) + row0, off, nv, qi);
    load_rows<IO, R>(static_cast<const char *>(a.dy) + row0, off, nv, qd);
    bool cut[R], in[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        cut[j] = a.reset && a.reset[b * L + t0 + min(g * R + j, left - 1)] != 0;
        in[j] = g * R + j < left;
    }
    auto channel = [&](int v) {
        const int d = min(d0 + v, D - 1);
        GateChannel c;
        c.A = MODE == SSM_GATE_RATE ? a.A[d] : 0.0f;
        c.gb = MODE != SSM_GATE_DECAY && a.gate_bias ? a.gate_bias[d] : 0.0f;
        c.ib = IG && a.in_bias ? a.in_bias[d] : 0.0f;
        return c;
    };

#pragma unroll
    for (int v0 = 0; v0 < V; v0 += 4) {
        float p[4], l[4], m[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int v = v0 + u;
            const GateChannel c = channel(v);
            float at[R];
            p[u] = 1.0f;
            l[u] = m[u] = 0.0f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                float bt;
                gate_step<MODE, IG>(lane_elem<IO>(qx[j], v), lane_elem<IO>(qg[j], v),
                                    IG ? lane_elem<IO>(qi[j], v) : 0.0f, c, at[j], bt);
                l[u] = !in[j] ? l[u] : cut[j] ? bt : __builtin_fmaf(at[j], l[u], bt);
                p[u] = !in[j] ? p[u] : cut[j] ? __builtin_nanf("") : at[j] * p[u];
            }
#pragma unroll
            for (int j = R - 1; j >= 0; --j)
                m[u] = !in[j] ? m[u] : cut[j] ? 0.0f : at[j] * (lane_elem<IO>(qd[j], v) + m[u]);
        }
        *reinterpret_cast<float4 *>(&sp[g][lc + v0]) = make_float4(p[0], p[1], p[2], p[3]);
        *reinterpret_cast<float4 *>(&sl[g][lc + v0]) = make_float4(l[0], l[1], l[2], l[3]);
        *reinterpret_cast<float4 *>(&sm[g][lc + v0]) = make_float4(m[0], m[1], m[2], m[3]);
    }
    __syncthreads();
    if (tid < CB) {
        const int d = cblk * CB + tid;
        // the tile's own run, from its last group to its first
        float tp = 1.0f, tm = 0.0f;
#pragma unroll 8
        for (int i = G - 1; i >= 0; --i) {
            const float p = sp[i][tid];
            tm = run_apply(p, sm[i][tid], tm);
            tp *= p;
        }
        u64_t *mine = rec + ((int64_t)chain * tiles + k) * CB + tid;
        if (k > 0 && k + 1 < tiles) rec_put(mine, rec_hi(tp), tm);
        // the states entering the groups, while the records before this one appear
        float h = d < D ? ck[((int64_t)tile * a.batch + b) * D + d] : 0.0f;
#pragma unroll 8
        for (int i = 0; i < G; ++i) {
            const float l = sl[i][tid];
            sl[i][tid] = h;
            h = run_apply(sp[i][tid], l, h);
        }
        float mu = k == 0 && a.dh_final && d < D ? a.dh_final[b * D + d] : 0.0f;
        if (k > 0) mu = chain_enter(mine, CB, k);
        const float after = run_apply(tp, tm, mu);
        if (k + 1 < tiles)
            rec_put(mine, kRecState, after);
        else if (a.dh0 && d < D)
            a.dh0[b * D + d] = after;
#pragma unroll 8
        for (int i = G - 1; i >= 0; --i) {
            const float m = sm[i][tid];
            sm[i][tid] = mu;
            mu = run_apply(sp[i][tid], m, mu);
        }
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        float ox[R][PER], og[R][PER], oi[R][PER];
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int v = w * PER + u;
            const GateChannel c = channel(v);
            float h = sl[g][lc + v], mu = sm[g][lc + v], at[R], hp[R], sA = 0.0f, sg = 0.0f, si = 0.0f;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                float bt;
                gate_step<MODE, IG>(lane_elem<IO>(qx[j], v), lane_elem<IO>(qg[j], v),
                                    IG ? lane_elem<IO>(qi[j], v) : 0.0f, c, at[j], bt);
                hp[j] = h;
                h = cut[j] ? bt : __builtin_fmaf(at[j], h, bt);
            }
#pragma unroll
            for (int j = R - 1; j >= 0; --j) {
                const float lam = lane_elem<IO>(qd[j], v) + mu;
                const GateGrad o = gate_grad<MODE, IG>(lane_elem<IO>(qx[j], v), lane_elem<IO>(qg[j], v),
                                                       IG ? lane_elem<IO>(qi[j], v) : 0.0f, c,
                                                       cut[j] ? 0.0f : lam * hp[j], lam);
                mu = !in[j] ? mu : cut[j] ? 0.0f : at[j] * lam;
                ox[j][u] = o.dx;
                og[j][u] = o.dg;
                oi[j][u] = o.di;
                sA += in[j] ? o.dA : 0.0f;
                sg += in[j] ? o.dg : 0.0f;
                si += in[j] ? o.di : 0.0f;
            }
            if constexpr (MODE != SSM_GATE_DECAY) {
                // this lane's own words: read above, by no other lane
                sp[g][lc + v] = sg;
                if constexpr (MODE == SSM_GATE_RATE) sl[g][lc + v] = sA;
                if constexpr (IG) sm[g][lc + v] = si;
            }
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if constexpr (IO::bytes == 2) {
                qx[j][w] = pack_bf16x2(ox[j][0], ox[j][PER - 1]);
                qg[j][w] = pack_bf16x2(og[j][0], og[j][PER - 1]);
                if constexpr (IG) qi[j][w] = pack_bf16x2(oi[j][0], oi[j][PER - 1]);
            } else {
                qx[j][w] = __float_as_uint(ox[j][0]);
                qg[j][w] = __float_as_uint(og[j][0]);
                if constexpr (IG) qi[j][w] = __float_as_uint(oi[j][0]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
        if (in[j]) {
            store_words<IO>(static_cast<char *>(a.dx) + row0 + off[j], nv, qx[j]);
            store_words<IO>(static_cast<char *>(a.dgate) + row0 + off[j], nv, qg[j]);
            if constexpr (IG) store_words<IO>(static_cast<char *>(a.din_gate) + row0 + off[j], nv, qi[j]);
        }
    if constexpr (MODE != SSM_GATE_DECAY) {
        // this tile's row of the partial sums: gate_bias, then A, then in_bias
        __syncthreads();
        const int which = tid / CB, ch = tid % CB, d = cblk * CB + ch;
        constexpr int K = MODE == SSM_GATE_SIGMOID ? 1 : IG ? 3 : 2;
        if (which < K && d < D) {
            const float(*s)[CB] = which == 0 ? sp : which == 1 ? sl : sm;
            float v = 0.0f;
#pragma unroll 8
            for (int i = 0; i < G; ++i) v += s[i][ch];
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
    const int64_t cb = a.io_dtype == SSM_BF16 ? TileShape<io_bf16>::CB : TileShape<io_f32>::CB;
    const int64_t tiles = (a.seqlen + T - 1) / T;
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
        p.o_ck = take((size_t)(tiles * a.batch * a.dim) * 4);
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
        gated_bwd_kernel<decltype(io), decltype(mode)::value, decltype(ig)::value>
            <<<grid, kGatedThreads, 0, stream>>>(a, ck, part, (int)p.chain.chains, (int)p.chain.tiles,
                                                 reinterpret_cast<u64_t *>(ws), tickets);
    });
    e = hipGetLastError();
    float *out[3] = {a.dgate_bias, a.dA, a.din_bias};
    if (e == hipSuccess && p.sums > 0 && (out[0] || out[1] || out[2]))
        e = launch_column_sums(part, p.rows, a.dim, p.sums, out, reinterpret_cast<float *>(ws + p.o_scratch), stream);
    return e;
}

}  // namespace ssm
