// gated_delta_bwd.hip -- gradients of the gated delta rule (ssm_gated_delta_bwd) on gfx950.  With the
// forward's names (gated_delta.hip), N the inverse of I + B diag(beta), U = diag(beta) E, S the state
// entering a chunk, dS the gradient of the state leaving it:
//   dU = P^T dO + leave K dS,  dX = N^T diag(beta) dU = dV
//   gradient of S:  through dS + (scale enter Q)^T dO - (enter K)^T dX
// which back_chain_kernel carries from the last chunk to the first, a workgroup 16 or 32 value channels as in the
// forward.  Then, for all chunks at once (grads_kernel), with dP = dO U^T (s <= t), Y = dX E^T (s < t) and
// dB = -Y diag(beta):
//   dq = scale enter dO S^T + scale (dP D) K
//   dk = leave U dS^T - enter dX S^T + scale (dP D)^T Q + (dB D) K + (dB D)^T K
//   dbeta_s = E_s . dU_s - sum_t B_ts Y_ts
//   dG_t = sum_s Z_ts - sum_s Z_st + q.(scale enter dO S^T) - k.(enter dX S^T) - k.(leave U dS^T),
//   Z = dP P + dB B;   dG_end += sum_t k.(leave U dS^T) + through <dS, S>;   dg = suffix sums of dG within a document
// dbeta never divides by beta: E is kept in place of U.
#include "delta_tile.h"
#include "wide_io.h"

#include <algorithm>

namespace ssm {
namespace delta {
namespace {

struct BackArgs {
    Call a;
    const char *blocks;
    const float *ck, *dh_final;
    const void *dout;
    void *dv;
    float *dh0;
    float *after, *dx, *edu;  // workspace: (B,H,n,K,V), (B,H,n,64,V), (B,H,n,slices,64)
    int slices;
};

template <typename IO, int KP, int NC>
struct BackLds {
    static constexpr int PL = Op<IO>::kPlanes;
    Slab<IO, 16 * NC, KP, PL> ds;       // column by column, as right operands
    Slab<IO, 16 * NC, kC, PL> u, w, q;  // diag(beta) dU; -enter dX; scale enter dO
    Slab<IO, 16 * NC, kC, 1> dout;
};

// The forward's chain (chain_kernel) backwards: wave w has the steps 16 w .. + 15 and the rows KP/4 w .. of
// the state's gradient.  8 x 2048 steps of 12 heads of 128, bf16: 261 us, bound as the forward's by the chain of
// a chunk's products; it writes 302 MB.
template <typename IO, int KP, int NC>
__global__ __launch_bounds__(kThreads, 2) void back_chain_kernel(BackArgs p) {
    using O = Op<IO>;
    using E = typename O::elem;
    using Block = ChunkBlock<IO, KP, true>;
    using Lds = BackLds<IO, KP, NC>;
    constexpr int KX = KP / 32, ST = KP / 64, PL = Lds::PL;
    extern __shared__ __attribute__((aligned(16))) char raw[];
    Lds &s = *reinterpret_cast<Lds *>(raw);
    const Call &a = p.a;
    const ChainPlace place = chain_place(a.B * a.H, p.slices);
    if (!place.any) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane % 16, grp = lane / 16;
    const int64_t head = place.head, b = head / a.H;
    const int h = (int)(head % a.H), hk = h / (a.H / a.Hk);
    const int row = 16 * wave + r16, mine = 16 * wave + 4 * grp;
    const char *blocks = p.blocks + head * a.n * Block::kBytes;
    const char *k_base = bytes(static_cast<const char *>(a.k), b * a.k_batch + (int64_t)hk * a.K, IO::bytes);
    const int64_t o_first = (b * a.L * a.H + h) * a.V * IO::bytes;
    const char *do_base = static_cast<const char *>(p.dout) + o_first;
    char *dv_base = static_cast<char *>(p.dv) + o_first;
    const uint32_t k_step = (uint32_t)a.k_token * IO::bytes, o_step = (uint32_t)(a.H * a.V) * IO::bytes;
    const uint32_t v_row = (uint32_t)a.V * 4;  // a state's row in bytes
    // lanes past the last channels repeat them, store nothing and count for nothing
    const int vw = channel<NC>(place.slice, r16);
    const uint32_t v0 = min(vw, a.V - NC);
    const bool live = vw < a.V;

    f4 ds[ST][NC];
#pragma unroll
    for (int j = 0; j < ST; ++j)
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int k0 = 16 * (ST * wave + j) + 4 * grp;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ds[j][n][i] = p.dh_final && k0 + i < a.K ? p.dh_final[(head * a.K + k0 + i) * a.V + v0 + n] : 0.0f;
            s.ds.put4(16 * n + r16, k0, ds[j][n]);
        }

    typename O::Ex kf[KX], ktf[ST][2], qtf[ST][2];
    typename O::template Sum<PL> inv[2], att[2];
    f4 k_enter, k_leave, q_enter, beta;
    float through;
    Elements<IO, NC> rdo[4];
    Elements<io_f32, NC> rerr[4];
    // a step of the chunk that is there
    const auto step_of = [&](int64_t c, int t) { return (uint32_t)min((int64_t)t, a.L - 1 - c * kC); };
    const auto load_k = [&](int64_t c) {
        const char *kc = k_base + c * kC * (int64_t)k_step;
        const uint32_t t = step_of(c, row) * k_step;
#pragma unroll
        for (int x = 0; x < KX; ++x)
            kf[x] = O::load(&at<E>(kc, t + (32 * x + 8 * grp < a.K ? 32 * x + 8 * grp : 0) * IO::bytes));
    };
    const auto load_vec = [&](int64_t c) {
        const char *vec = blocks + c * Block::kBytes;
        k_enter = at<f4>(vec, (kVecKEnter * kC + mine) * 4);
        k_leave = at<f4>(vec, (kVecKLeave * kC + mine) * 4);
        q_enter = at<f4>(vec, (kVecQEnter * kC + mine) * 4);
        beta = at<f4>(vec, (kVecBeta * kC + mine) * 4);
        through = at<float>(vec, kVecThrough * kC * 4);
    };
    const auto load_dout = [&](int64_t c) {
        const char *dc = do_base + c * kC * (int64_t)o_step;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            rdo[i] = Elements<IO, NC>::load(dc, step_of(c, mine + i) * o_step + v0 * IO::bytes);
    };
    const auto load_err = [&](int64_t c) {
        const char *err = reinterpret_cast<const char *>(p.ck) + ((c * a.B * a.H + head) * (a.K + kC) + a.K) * (int64_t)v_row;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            rerr[i] = Elements<io_f32, NC>::load(err + i * (int64_t)v_row, mine * v_row + v0 * 4);
    };
    constexpr int TILE = 512 * IO::bytes;
    const uint32_t in_tile = lane * 8 * IO::bytes;
    // (the waves of the lower half have no first block of columns: they load the second twice)
    const int tile1 = (2 * wave + 1) * TILE, tile0 = tile1 - (1 - wave / 2) * TILE;
    const auto load_matrix = [&](typename O::template Sum<PL> (&m)[2], int64_t c, size_t off) {
        const char *from = blocks + c * Block::kBytes + off;
        m[0] = O::template planes<PL>(&at<E>(from + tile0, in_tile), Block::PLANE);
        m[1] = O::template planes<PL>(&at<E>(from + tile1, in_tile), Block::PLANE);
    };
    const auto load_rows = [&](typename O::Ex (&m)[ST][2], int64_t c, size_t off) {
        const char *from = blocks + c * Block::kBytes + off + 2 * ST * wave * TILE;
#pragma unroll
        for (int j = 0; j < ST; ++j)
#pragma unroll
            for (int y = 0; y < 2; ++y) m[j][y] = O::load(&at<E>(from + (2 * j + y) * TILE, in_tile));
    };
    // this chunk's dO, as an operand and against the state; steps past the end as 0
    f4 dout[NC];
    const auto put_dout = [&](int64_t c) {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dout[n][i] = (c + 1) * kC <= a.L || c * kC + mine + i < a.L ? rdo[i].get(n) : 0.0f;
            s.dout.put4(16 * n + r16, mine, dout[n]);
        }
    };
    const int64_t last = a.n - 1;
    load_dout(last);
    load_k(last);
    load_vec(last);
    load_matrix(att, last, Block::kAtt);
    load_err(last);
    load_matrix(inv, last, Block::kInv);
    load_rows(ktf, last, Block::kKt);
    load_rows(qtf, last, Block::kQt);
    put_dout(last);
    load_dout(last > 0 ? last - 1 : 0);
    __syncthreads();
    for (int64_t c = last; c >= 0; --c) {
        const int64_t next = c > 0 ? c - 1 : 0, chunk = head * a.n + c;
        const bool whole = (c + 1) * kC <= a.L;
        if (!whole || a.K != KP)
#pragma unroll
            for (int x = 0; x < KX; ++x)
                if (c * kC + row >= a.L || 32 * x + 8 * grp >= a.K) kf[x] = typename O::Ex{};
        // dU = leave K dS + P^T dO
        f4 du[NC] = {};
#pragma unroll
        for (int x = 0; x < KX; ++x)
#pragma unroll
            for (int n = 0; n < NC; ++n)
                du[n] = O::mul(du[n], kf[x], s.ds.get(16 * n + r16, 32 * x + 8 * grp));
        load_k(next);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) du[n][i] = k_leave[i] != 0.0f ? k_leave[i] * du[n][i] : 0.0f;
            if (wave < 2) du[n] = O::mul(du[n], att[0], s.dout.get_exact(16 * n + r16, 8 * grp));
            du[n] = O::mul(du[n], att[1], s.dout.get_exact(16 * n + r16, 32 + 8 * grp));
            s.u.put4(16 * n + r16, mine, beta * du[n]);
            s.q.put4(16 * n + r16, mine, q_enter * dout[n]);
        }
        load_matrix(att, next, Block::kAtt);
        // E . dU over the slice's channels
        f4 e;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float own = 0.0f;
#pragma unroll
            for (int n = 0; n < NC; ++n) own = __builtin_fmaf(rerr[i].get(n), du[n][i], own);
            e[i] = sum16(live ? own : 0.0f);
        }
        if (r16 == 0) *reinterpret_cast<f4 *>(p.edu + (chunk * p.slices + place.slice) * kC + mine) = e;
        load_err(next);
        store_rows<ST, NC>(reinterpret_cast<char *>(p.after) + chunk * a.K * (int64_t)v_row, v_row, a.K,
                           16 * ST * wave + 4 * grp, a.K == KP, v0, live, ds);
        __syncthreads();
        // dX = N^T diag(beta) dU
        char *dvc = dv_base + (c * kC + 16 * wave) * (int64_t)o_step;
        char *dxc = reinterpret_cast<char *>(p.dx) + chunk * kC * (int64_t)v_row;
        f4 dx[NC] = {};
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            if (wave < 2) dx[n] = O::mul(dx[n], inv[0], s.u.get(16 * n + r16, 8 * grp));
            dx[n] = O::mul(dx[n], inv[1], s.u.get(16 * n + r16, 32 + 8 * grp));
            s.w.put4(16 * n + r16, mine, -k_enter * dx[n]);
        }
        if (live)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[NC];
#pragma unroll
                for (int n = 0; n < NC; ++n) x[n] = dx[n][i];
                store_floats<NC>(dxc + i * (int64_t)v_row, mine * v_row + v0 * 4, x);
                if (whole || c * kC + mine + i < a.L)
                    store_elements<IO, NC>(dvc + i * (int64_t)o_step, 4 * grp * o_step + v0 * IO::bytes, x);
            }
        load_matrix(inv, next, Block::kInv);
        const float pass = through;
        load_vec(next);
        __syncthreads();
        // dS <- through dS + (scale enter Q)^T dO - (enter K)^T dX
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const auto w0 = s.w.get(16 * n + r16, 8 * grp), w1 = s.w.get(16 * n + r16, 32 + 8 * grp);
            const auto q0 = s.q.get(16 * n + r16, 8 * grp), q1 = s.q.get(16 * n + r16, 32 + 8 * grp);
#pragma unroll
            for (int j = 0; j < ST; ++j) {
                f4 &d = ds[j][n];
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = pass != 0.0f ? pass * d[i] : 0.0f;
                d = O::mul(O::mul(d, qtf[j][0], q0), qtf[j][1], q1);
                d = O::mul(O::mul(d, ktf[j][0], w0), ktf[j][1], w1);
                s.ds.put4(16 * n + r16, 16 * (ST * wave + j) + 4 * grp, d);
            }
        }
        load_rows(ktf, next, Block::kKt);
        load_rows(qtf, next, Block::kQt);
        put_dout(next);
        load_dout(next > 0 ? next - 1 : 0);
        __syncthreads();
    }
    if (p.dh0)
        store_rows<ST, NC>(reinterpret_cast<char *>(p.dh0) + head * a.K * (int64_t)v_row, v_row, a.K,
                           16 * ST * wave + 4 * grp, a.K == KP, v0, live, ds);
}

// --------------------------------------------------------------------------- all chunks at once
constexpr int kGradThreads = 512, kVB = 32;  // value channels of a pass

struct GradArgs {
    Call a;
    const char *blocks;
    const float *ck, *after, *dx, *edu;
    const void *dout;
    void *dq, *dk, *dbeta;
    float *dg;
    int slices;
};

template <typename IO, int KP>
struct GradLds {
    using Rows = HeadRows<IO, KP>;
    using E = typename Op<IO>::elem;
    static constexpr int TSTRIDE = kC + 16 / IO::bytes;
    static constexpr bool kTransposed = IO::bytes == 2;
    alignas(16) E q[kC * Rows::STRIDE], k[kC * Rows::STRIDE];
    Gates gates;
    float row_z[4][kC], col_z[4][kC], col_by[4][kC], edu[kC];
    alignas(16) float row_a[KP / 16][kC], row_b[KP / 16][kC];
    float dots[kGradThreads / 64];
    alignas(16) union {
        struct {
            Slab<IO, kC, kVB, 1> dout;
            Slab<IO, kC, kVB, 3> dx, err;
            Slab<IO, KP, kVB, 3> before, after;
        } in;
        struct {
            alignas(16) E kt[kTransposed ? KP * TSTRIDE : 8], qt[kTransposed ? KP * TSTRIDE : 8];
            Slab<IO, kC, kC, 2> m1, m2, m3;  // these feed outputs of the tensors' type alone
        } out;
    };
};

// The lower tiles of the 64 x 64 matrices, dealt to eight waves: tile `i` of ten.
__device__ __forceinline__ void lower_tile(int i, int &ti, int &tj) {
    ti = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3;
    tj = i - ti * (ti + 1) / 2;
}

// One chunk of one key head, over the value heads that share it.  Wave w has the result columns
// 16 (w % KT) .. + 15 of the products with K channels and, with KP = 64, half of their rows.  8 x 2048 steps of
// 12 heads of 128, bf16: 361 us for 0.7 GB, bound by latency: half of the waves' cycles wait, mostly for the
// value slices' way through LDS (27000 of a chunk's 75000 cycles), at one workgroup a CU (142 KB of LDS).
template <typename IO, int KP>
__global__ __launch_bounds__(kGradThreads) void grads_kernel(GradArgs p) {
    using O = Op<IO>;
    using E = typename O::elem;
    using Rows = HeadRows<IO, KP>;
    using Lds = GradLds<IO, KP>;
    constexpr int KT = KP / 16, NT = KT / 2, SR = KP / 64;  // SR: state rows' pieces a thread
    extern __shared__ __attribute__((aligned(16))) char raw[];
    Lds &s = *reinterpret_cast<Lds *>(raw);
    const Call &a = p.a;
    const int64_t c = blockIdx.x, b = blockIdx.z, t0 = c * kC;
    const int hk = blockIdx.y, share = a.H / a.Hk;
    {
        typename Rows::template Regs<8> rq, rk;
        Rows::template load<8>(rq, a.q, b * a.q_batch + (int64_t)hk * a.K, a.q_token, t0, a.L, a.K);
        Rows::template load<8>(rk, a.k, b * a.k_batch + (int64_t)hk * a.K, a.k_token, t0, a.L, a.K);
        Rows::template cut<8>(rq, t0, a.L, a.K);
        Rows::template cut<8>(rk, t0, a.L, a.K);
        Rows::template store<8>(rq, s.q);
        Rows::template store<8>(rk, s.k);
    }
    f4 dq[NT] = {}, dk[NT] = {};
    for (int h = hk * share; h < (hk + 1) * share; ++h) {
        // The thread's place, formed anew for each head: the compiler would else keep hundreds of addresses
        // that depend on nothing but it across the heads, in scratch memory.
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r16 = lane % 16, grp = lane / 16;
        const int kd = wave % KT, first = wave / KT * NT;
        const int64_t chunk = (b * a.H + h) * a.n + c;
        const float *before = p.ck + ((c * a.B + b) * a.H + h) * (a.K + kC) * a.V, *err = before + (int64_t)a.K * a.V;
        const float *after = p.after + chunk * a.K * a.V, *dx = p.dx + chunk * kC * a.V;
        const int row = tid / 8, col = tid % 8 * 4;
        Raw<IO, 4> rdo;
        f4 rdx, rerr, rs[SR], ra[SR];
        // (rows and channels past the ends come from elsewhere and are cleared when they are put down)
        const bool step_in = t0 + row < a.L;
        const int64_t o_row = ((b * a.L + (step_in ? t0 + row : a.L - 1)) * a.H + h) * a.V;
        const auto fetch = [&](int v0) {
            const int v = v0 + col < a.V ? v0 + col : 0;
            rdo = load_raw<IO, 4>(p.dout, o_row + v, 4);
            rdx = *reinterpret_cast<const f4 *>(dx + row * a.V + v);
            rerr = *reinterpret_cast<const f4 *>(err + row * a.V + v);
#pragma unroll
            for (int j = 0; j < SR; ++j) {
                const int k = row + 64 * j, at = (k < a.K ? k : 0) * a.V + v;
                rs[j] = *reinterpret_cast<const f4 *>(before + at);
                ra[j] = *reinterpret_cast<const f4 *>(after + at);
            }
        };
        fetch(0);
        {  // the chunk's gates, as prepare_kernel formed them
            using Block = ChunkBlock<IO, KP, true>;
            const uint32_t *from = reinterpret_cast<const uint32_t *>(p.blocks + chunk * Block::kBytes + Block::kGates);
            for (int i = tid; i < (int)sizeof(Gates) / 4; i += kGradThreads)
                reinterpret_cast<uint32_t *>(&s.gates)[i] = from[i];
        }
        f4 os[NT] = {}, xs[NT] = {}, es[NT] = {}, dp[2] = {}, yy[2] = {};
        float dot = 0.0f;
        for (int v0 = 0; v0 < a.V; v0 += kVB) {
            __syncthreads();
            const f4 zero = {0, 0, 0, 0};
            const bool in = v0 + col < a.V;
            s.in.dout.put4(row, col, in && step_in ? f4{rdo[0], rdo[1], rdo[2], rdo[3]} : zero);
            s.in.dx.put4(row, col, in ? rdx : zero);
            s.in.err.put4(row, col, in ? rerr : zero);
#pragma unroll
            for (int j = 0; j < SR; ++j) {
                if (!in || row + 64 * j >= a.K) rs[j] = ra[j] = zero;
                s.in.before.put4(row + 64 * j, col, rs[j]);
                s.in.after.put4(row + 64 * j, col, ra[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) dot = __builtin_fmaf(rs[j][i], ra[j][i], dot);
            }
            __syncthreads();
            if (v0 + kVB < a.V) fetch(v0 + kVB);
            const auto sb = s.in.before.get(16 * kd + r16, 8 * grp), sa = s.in.after.get(16 * kd + r16, 8 * grp);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int t = 16 * (first + j) + r16;
                os[j] = O::mul(os[j], s.in.dout.get_exact(t, 8 * grp), sb);
                xs[j] = O::mul(xs[j], s.in.dx.get(t, 8 * grp), sb);
                es[j] = O::mul(es[j], s.in.err.get(t, 8 * grp), sa);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (wave + 8 * j < 10) {
                    int ti, tj;
                    lower_tile(wave + 8 * j, ti, tj);
                    const auto e = s.in.err.get(16 * tj + r16, 8 * grp);
                    dp[j] = O::mul(dp[j], s.in.dout.get_exact(16 * ti + r16, 8 * grp), e);
                    yy[j] = O::mul(yy[j], s.in.dx.get(16 * ti + r16, 8 * grp), e);
                }
        }
        __syncthreads();  // the slabs make room for the matrices
#pragma unroll
        for (int d = 1; d < 64; d *= 2) dot += __shfl_xor(dot, d, 64);
        if (lane == 0) s.dots[wave] = dot;
        if constexpr (Lds::kTransposed)
            for (int i = tid; i < kC * KP / 8; i += kGradThreads) {
                const int t = i % kC, k = i / kC * 8;
                const auto kv = O::load(s.k + t * Rows::STRIDE + k), qv = O::load(s.q + t * Rows::STRIDE + k);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s.out.kt[(k + j) * Lds::TSTRIDE + t] = kv.v[j];
                    s.out.qt[(k + j) * Lds::TSTRIDE + t] = qv.v[j];
                }
            }
        // (the three matrices lie side by side; what the tiles below do not write is 0)
        for (int i = tid; i < (int)(3 * sizeof(s.out.m1) / 16); i += kGradThreads)
            reinterpret_cast<u4 *>(&s.out.m1)[i] = u4{0, 0, 0, 0};
        __syncthreads();
        if (wave == kGradThreads / 64 - 1) {  // (one of those with one tile)
            float e = 0.0f;
            for (int i = 0; i < p.slices; ++i) e += p.edu[(chunk * p.slices + i) * kC + lane];
            s.edu[lane] = e;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (wave + 8 * j < 10) {
                int ti, tj;
                lower_tile(wave + 8 * j, ti, tj);
                f4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
#pragma unroll
                for (int x = 0; x < KP / 32; ++x) {
                    const typename O::Ex kb = O::load(s.k + (16 * tj + r16) * Rows::STRIDE + 32 * x + 8 * grp);
                    kk = O::mul(kk, O::load(s.k + (16 * ti + r16) * Rows::STRIDE + 32 * x + 8 * grp), kb);
                    qk = O::mul(qk, O::load(s.q + (16 * ti + r16) * Rows::STRIDE + 32 * x + 8 * grp), kb);
                }
                const int u = 16 * tj + r16;
                const float rku = s.gates.rk[u], bu = s.gates.beta[u];
                float cz = 0.0f, cby = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 16 * ti + 4 * grp + i;
                    const float d = decay(s.gates, t, u), rqt = s.gates.rq[t], rkt = s.gates.rk[t];
                    const float below = u < t ? 1.0f : 0.0f;
                    const float dpv = u <= t ? bu * dp[j][i] : 0.0f, y = below * yy[j][i], db = -bu * y;
                    const float att = a.scale * d * rqt * rku * qk[i], bm = below * d * rkt * rku * kk[i];
                    const float z = dpv * att + db * bm, by = bm * y;
                    const float sq = a.scale * d * dpv, sb = d * db;
                    if (u <= t) {
                        s.out.m1.put(t, u, sq * rku);
                        s.out.m2.put(u, t, sq * rqt);
                    }
                    if (u < t) {
                        s.out.m3.put(t, u, sb * rku);
                        s.out.m3.put(u, t, sb * rkt);
                    }
                    cz += z;
                    cby += by;
                    const float rz = sum16(z);
                    if (r16 == 0) s.row_z[tj][t] = rz;
                }
#pragma unroll
                for (int d = 16; d < 64; d *= 2) {
                    cz += __shfl_xor(cz, d, 64);
                    cby += __shfl_xor(cby, d, 64);
                }
                if (grp == 0) {
                    s.col_z[ti][u] = cz;
                    s.col_by[ti][u] = cby;
                }
            }
        // the parts through the states
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * (first + j) + 4 * grp + i, k = 16 * kd + r16;
                const float en = s.gates.enter[t], lv = s.gates.leave[t] * s.gates.beta[t];
                const float tq = en != 0.0f ? a.scale * en * os[j][i] : 0.0f, tk = en != 0.0f ? en * xs[j][i] : 0.0f;
                const float lf = lv != 0.0f ? lv * es[j][i] : 0.0f;
                const float qv = s.gates.rq[t] * (float)s.q[t * Rows::STRIDE + k];
                const float kv = s.gates.rk[t] * (float)s.k[t * Rows::STRIDE + k];
                const float out = sum16(kv * lf), ra_ = sum16(qv * tq - kv * tk);
                if (r16 == 0) {
                    s.row_a[kd][t] = ra_ - out;
                    s.row_b[kd][t] = out;
                }
                dq[j][i] += tq;
                dk[j][i] += lf - tk;
            }
        __syncthreads();
        if (wave == 0) {
            const int t = lane;
            double dG = 0.0, leaves = 0.0;
            float dbeta = 0.0f;
            const int tile = t / 16;
            for (int i = 0; i < 4; ++i) {
                if (i <= tile) dG += s.row_z[i][t];
                if (i >= tile) {
                    dG -= s.col_z[i][t];
                    dbeta -= s.col_by[i][t];
                }
            }
            for (int i = 0; i < KT; ++i) {
                dG += s.row_a[i][t];
                leaves += s.row_b[i][t];
            }
            for (int d = 1; d < 64; d *= 2) leaves += __shfl_xor(leaves, d, 64);
            if (t == 63) {
                double through = 0.0;
                for (int i = 0; i < kGradThreads / 64; ++i) through += s.dots[i];
                dG += leaves + (s.gates.through != 0.0f ? s.gates.through * through : 0.0);
            }
            // (over a document's steps: those behind a reset add up to 0, but for their rounding)
            const int doc = s.gates.doc[t];
            for (int d = 1; d < 64; d *= 2) {
                const double down = __shfl_down(dG, d, 64);
                if (t + d < 64 && s.gates.doc[t + d] == doc) dG += down;
            }
            dbeta += s.edu[t];
            const bool cut = doc != (t ? s.gates.doc[t - 1] : 0);
            if (t0 + t < a.L) {
                const int64_t at = (b * a.L + t0 + t) * a.H + h;
                p.dg[at] = cut ? 0.0f : (float)dG;
                store_io<IO>(p.dbeta, at, dbeta);
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int ti = first + j;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                typename O::Ex kr, qr;
                if constexpr (Lds::kTransposed) {
                    kr = O::load(s.out.kt + (16 * kd + r16) * Lds::TSTRIDE + 32 * y + 8 * grp);
                    qr = O::load(s.out.qt + (16 * kd + r16) * Lds::TSTRIDE + 32 * y + 8 * grp);
                } else {
                    kr = Op<IO>::gather(s.k + (32 * y + 8 * grp) * Rows::STRIDE + 16 * kd + r16, Rows::STRIDE);
                    qr = Op<IO>::gather(s.q + (32 * y + 8 * grp) * Rows::STRIDE + 16 * kd + r16, Rows::STRIDE);
                }
                const int at = 32 * y + 8 * grp;
                if (y <= ti / 2) dq[j] = O::mul(dq[j], s.out.m1.get(16 * ti + r16, at), kr);
                if (y >= ti / 2) dk[j] = O::mul(dk[j], s.out.m2.get(16 * ti + r16, at), qr);
                dk[j] = O::mul(dk[j], s.out.m3.get(16 * ti + r16, at), kr);
            }
        }
        __syncthreads();
    }
    // through the norms: dx = r (dxhat - xhat (xhat . dxhat))
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane % 16, grp = lane / 16;
    const int kd = wave % KT, first = wave / KT * NT;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 16 * (first + j) + 4 * grp + i, k = 16 * kd + r16;
            const float qd = sum16(s.gates.rq[t] * (float)s.q[t * Rows::STRIDE + k] * dq[j][i]);
            const float kd_ = sum16(s.gates.rk[t] * (float)s.k[t * Rows::STRIDE + k] * dk[j][i]);
            if (r16 == 0) {
                s.row_a[kd][t] = qd;
                s.row_b[kd][t] = kd_;
            }
        }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int first_t = 16 * (first + j) + 4 * grp, k = 16 * kd + r16;
        f4 q_dot = {0, 0, 0, 0}, k_dot = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < KT; ++w) {
            q_dot += *reinterpret_cast<const f4 *>(&s.row_a[w][first_t]);
            k_dot += *reinterpret_cast<const f4 *>(&s.row_b[w][first_t]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = first_t + i;
            float oq = dq[j][i], ok = dk[j][i];
            E &qe = s.q[t * Rows::STRIDE + k], &ke = s.k[t * Rows::STRIDE + k];  // this lane's alone by now
            if (a.l2norm) {
                const float rq = s.gates.rq[t], rk = s.gates.rk[t];
                oq = rq * (oq - rq * (float)qe * q_dot[i]);
                ok = rk * (ok - rk * (float)ke * k_dot[i]);
            }
            qe = (E)oq;
            ke = (E)ok;
        }
    }
    __syncthreads();
    // out by rows, 16 bytes a lane
    for (int i = threadIdx.x; i < kC * KP / Rows::PER; i += kGradThreads) {
        const int t = i / (KP / Rows::PER), k = i % (KP / Rows::PER) * Rows::PER;
        if (t0 + t >= a.L || k >= a.K) continue;
        const int64_t at = ((b * a.L + t0 + t) * a.Hk + hk) * a.K + k;
        reinterpret_cast<u32x4_a2 *>(static_cast<E *>(p.dq) + at)[0] = *reinterpret_cast<const u4 *>(s.q + t * Rows::STRIDE + k);
        reinterpret_cast<u32x4_a2 *>(static_cast<E *>(p.dk) + at)[0] = *reinterpret_cast<const u4 *>(s.k + t * Rows::STRIDE + k);
    }
}

template <typename IO, int KP, int NC>
hipError_t back_chain(BackArgs p, GradArgs g, hipStream_t stream) {
    p.slices = g.slices = (p.a.V + 16 * NC - 1) / (16 * NC);
    back_chain_kernel<IO, KP, NC>
        <<<chain_grid(p.a.B * p.a.H, p.slices), kThreads, sizeof(BackLds<IO, KP, NC>), stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 chunks((unsigned)p.a.n, (unsigned)p.a.Hk, (unsigned)p.a.B);
    grads_kernel<IO, KP><<<chunks, kGradThreads, sizeof(GradLds<IO, KP>), stream>>>(g);
    return hipGetLastError();
}

template <typename IO, int KP>
hipError_t backward(const BackArgs &p, const GradArgs &g, hipStream_t stream) {
    // 32 value channels a workgroup where that leaves one for each CU, as forwards (8 x 2048 x 12 heads: 253 us, 320
    // with 16); floats keep to 16, as 32 would not fit the registers
    if constexpr (IO::bytes == 2)
        if (wide_slices(p.a)) return back_chain<IO, KP, 2>(p, g, stream);
    return back_chain<IO, KP, 1>(p, g, stream);
}

struct BackPlan {
    size_t blocks, after, dx, edu, ck, total;
};

BackPlan back_plan(const ssm_gated_delta_bwd_args_t &a) {
    const size_t n = (size_t)((a.seqlen + kC - 1) / kC), chunks = n * a.batch * a.heads;
    BackPlan p;
    p.blocks = marks_bytes((int64_t)chunks);
    p.after = p.blocks + up256(chunks * block_bytes(a.io_dtype, a.kdim, true));
    if (!a.checkpoints)
        p.after = std::max(p.after, chain_bytes(a.io_dtype, a.batch * a.heads, (int64_t)n, a.kdim, a.vdim));
    p.dx = p.after + up256(chunks * a.kdim * a.vdim * 4);
    p.edu = p.dx + up256(chunks * kC * a.vdim * 4);
    p.ck = p.edu + up256(chunks * ((a.vdim + 15) / 16) * kC * 4);
    p.total = p.ck + (a.checkpoints ? 0 : up256(chunks * (a.kdim + kC) * a.vdim * 4));
    return p;
}

}  // namespace

hipError_t launch_backward(const Call &c, const ssm_gated_delta_bwd_args_t &a, hipStream_t stream) {
    const BackPlan plan = back_plan(a);
    char *ws = static_cast<char *>(a.workspace);
    const float *ck = a.checkpoints;
    hipError_t e = hipSuccess;
    if (!ck) {
        float *own = reinterpret_cast<float *>(ws + plan.ck);
        e = launch_prepare(c, a.io_dtype, false, ws, stream);
        if (e == hipSuccess) e = launch_chain(c, a.io_dtype, ws, a.h0, nullptr, nullptr, own, stream);
        if (e != hipSuccess) return e;
        ck = own;
    }
    e = launch_prepare(c, a.io_dtype, true, ws, stream);
    if (e != hipSuccess) return e;
    float *after = reinterpret_cast<float *>(ws + plan.after), *dx = reinterpret_cast<float *>(ws + plan.dx);
    float *edu = reinterpret_cast<float *>(ws + plan.edu);
    char *blocks = ws + plan.blocks;
    const BackArgs p{c, blocks, ck, a.dh_final, a.dout, a.dv, a.dh0, after, dx, edu, 0};
    const GradArgs g{c, blocks, ck, after, dx, edu, a.dout, a.dq, a.dk, a.dbeta, a.dg, 0};
    if (a.io_dtype == SSM_BF16)
        e = a.kdim <= 64 ? backward<io_bf16, 64>(p, g, stream) : backward<io_bf16, 128>(p, g, stream);
    else
        e = a.kdim <= 64 ? backward<io_f32, 64>(p, g, stream) : backward<io_f32, 128>(p, g, stream);
    if (e != hipSuccess) return e;
    return launch_grow_back(c, a, reinterpret_cast<const uint32_t *>(ws), ck, blocks, edu, stream);
}

size_t backward_bytes(const ssm_gated_delta_bwd_args_t &a) { return back_plan(a).total; }

}  // namespace delta
}  // namespace ssm
