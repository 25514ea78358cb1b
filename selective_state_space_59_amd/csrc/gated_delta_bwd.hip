// gated_delta_bwd.hip -- gradients of the gated delta rule (ssm_gated_delta_bwd) on gfx950.  With the
// forward's names (gated_delta.hip), N the inverse of I + B diag(beta), U = diag(beta) E, S the state
// entering a chunk, dS the gradient of the state leaving it:
//   dU = P^T dO + leave K dS,  dX = N^T diag(beta) dU = dV
//   gradient of S:  through dS + (scale enter Q)^T dO - (enter K)^T dX
// which back_chain_kernel carries from the last chunk to the first, each wave 16 value channels as in the
// forward.  Then, for all chunks at once (grads_kernel), with dP = dO U^T (s <= t), Y = dX E^T (s < t) and
// dB = -Y diag(beta):
//   dq = scale enter dO S^T + scale (dP D) K
//   dk = leave U dS^T - enter dX S^T + scale (dP D)^T Q + (dB D) K + (dB D)^T K
//   dbeta_s = E_s . dU_s - sum_t B_ts Y_ts
//   dG_t = sum_s Z_ts - sum_s Z_st + q.(scale enter dO S^T) - k.(enter dX S^T) - k.(leave U dS^T),
//   Z = dP P + dB B;   dG_end += sum_t k.(leave U dS^T) + through <dS, S>;   dg = suffix sums of dG
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
    float *after, *dx, *edu;  // workspace: (B,H,n,K,V), (B,H,n,64,V), (B,H,n,ceil(V/16),64)
};

template <typename IO, int KP>
struct BackLds {
    using Rows = HeadRows<IO, KP>;
    using Block = ChunkBlock<IO>;
    using E = typename Op<IO>::elem;
    static constexpr bool kTransposed = IO::bytes == 2;
    alignas(16) E k[kC * Rows::STRIDE];
    alignas(16) E q[kTransposed ? 8 : kC * Rows::STRIDE];
    alignas(16) E kt[kTransposed ? KP * Rows::TSTRIDE : 8], qt[kTransposed ? KP * Rows::TSTRIDE : 8];
    alignas(16) E inv[Block::Inv::PLANES * Block::Inv::PLANE], att[Block::AttT::PLANES * Block::AttT::PLANE];
    alignas(16) float vec[kVecs * kC];
};

template <typename IO, int KP>
__global__ __launch_bounds__(kThreads) void back_chain_kernel(BackArgs p) {
    using O = Op<IO>;
    using E = typename O::elem;
    using Rows = HeadRows<IO, KP>;
    using Block = ChunkBlock<IO>;
    using Lds = BackLds<IO, KP>;
    constexpr int KT = KP / 16, PL = O::kPlanes;
    extern __shared__ __attribute__((aligned(16))) char raw[];
    Lds &s = *reinterpret_cast<Lds *>(raw);
    const Call &a = p.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane % 16, grp = lane / 16;
    const int64_t b = blockIdx.z;
    const int h = blockIdx.y, hk = h / (a.H / a.Hk);
    const int strip = blockIdx.x * (kThreads / 64) + wave, strips = (a.V + 15) / 16;
    // lanes past the last channel repeat it, store nothing and count for nothing
    const int vw = strip * 16 + r16, v = min(vw, a.V - 1);
    const bool live = vw < a.V;
    const int64_t head = b * a.H + h;
    const char *blocks = p.blocks + head * a.n * Block::kBytes;
    const int64_t q_off = b * a.q_batch + (int64_t)hk * a.K, k_off = b * a.k_batch + (int64_t)hk * a.K;

    f4 ds[KT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = pair_row(kt, grp, i);
            ds[kt][i] = p.dh_final && k < a.K ? p.dh_final[(head * a.K + k) * a.V + v] : 0.0f;
        }
    typename Rows::template Regs<4> rq, rk;
    typename Block::Inv::template Regs<kThreads> rinv;
    typename Block::AttT::template Regs<kThreads> ratt;
    float rvec[2];
    RawOne<IO> rdo[4][4];
    f4 rerr[4];
    const auto fetch = [&](int64_t c) {
        const char *block = blocks + c * Block::kBytes;
        Rows::template load<4>(rq, a.q, q_off, a.q_token, c * kC, a.L, a.K);
        Rows::template load<4>(rk, a.k, k_off, a.k_token, c * kC, a.L, a.K);
        Block::Inv::template load<kThreads>(rinv, reinterpret_cast<const E *>(block + Block::kVecBytes));
        Block::AttT::template load<kThreads>(
            ratt, reinterpret_cast<const E *>(block + Block::kVecBytes + Block::kInvBytes));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = min((int)threadIdx.x + kThreads * i, kVecs * kC - 1);
            rvec[i] = reinterpret_cast<const float *>(block)[at];
        }
        const float *err = p.ck + (((c * a.B + b) * a.H + h) * (a.K + kC) + a.K) * a.V + v;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = pair_row(tt, grp, i);
                const int64_t t = c * kC + r;
                rdo[tt][i] = load_one<IO>(p.dout, ((b * a.L + (t < a.L ? t : a.L - 1)) * a.H + h) * a.V + v);
                rerr[tt][i] = err[r * a.V];
            }
    };
    fetch(a.n - 1);
    for (int64_t c = a.n - 1; c >= 0; --c) {
        __syncthreads();
        const bool whole = (c + 1) * kC <= a.L;
        Rows::template cut<4>(rq, c * kC, a.L, a.K);
        Rows::template cut<4>(rk, c * kC, a.L, a.K);
        Rows::template store<4>(rk, s.k);
        if constexpr (Lds::kTransposed) {
            Rows::template store_transposed<4>(rk, s.kt);
            Rows::template store_transposed<4>(rq, s.qt);
        } else {
            Rows::template store<4>(rq, s.q);
        }
        Block::Inv::template store<kThreads>(rinv, s.inv);
        Block::AttT::template store<kThreads>(ratt, s.att);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = threadIdx.x + kThreads * i;
            if (at < kVecs * kC) s.vec[at] = rvec[i];
        }
        f4 dout[4], err[4];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dout[tt][i] = whole || c * kC + pair_row(tt, grp, i) < a.L ? rdo[tt][i].get() : 0.0f;
                err[tt][i] = live ? rerr[tt][i] : 0.0f;
            }
        }
        __syncthreads();
        if (c > 0) fetch(c - 1);

        const int64_t chunk = head * a.n + c;
        if (live) store_state<KT>(p.after + chunk * a.K * a.V + v, a.K, a.V, grp, ds);
        // dU = P^T dO + leave K dS
        f4 du[4] = {};
#pragma unroll
        for (int x = 0; x < KT / 2; ++x) {
            const auto st = O::template sum<PL>(ds[2 * x], ds[2 * x + 1]);
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
                du[tt] = O::mul(du[tt], O::load(s.k + pair_row16(tt, r16) * Rows::STRIDE + 32 * x + 8 * grp), st);
        }
        const typename O::Ex dx_in[2] = {O::exact(dout[0], dout[1]), O::exact(dout[2], dout[3])};
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
            const f4 lv = *reinterpret_cast<const f4 *>(s.vec + kVecKLeave * kC + pair_row(tt, grp, 0));
#pragma unroll
            for (int i = 0; i < 4; ++i) du[tt][i] = lv[i] != 0.0f ? lv[i] * du[tt][i] : 0.0f;
#pragma unroll
            for (int y = tt / 2; y < 2; ++y)
                du[tt] = O::mul(du[tt],
                                O::template planes<PL>(s.att + pair_row16(tt, r16) * Block::AttT::STRIDE + 32 * y + 8 * grp,
                                                       Block::AttT::PLANE),
                                dx_in[y]);
        }
        // E . dU over this wave's channels
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
            f4 e = err[tt] * du[tt];
#pragma unroll
            for (int d = 1; d < 16; d *= 2)
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] += __shfl_xor(e[i], d, 64);
            if (r16 == 0 && strip < strips)
                *reinterpret_cast<f4 *>(p.edu + (chunk * strips + strip) * kC + pair_row(tt, grp, 0)) = e;
        }
        // dX = N^T diag(beta) dU
        f4 dx[4] = {};
        {
            typename O::template Sum<PL> us[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const f4 b0 = *reinterpret_cast<const f4 *>(s.vec + kVecBeta * kC + pair_row(2 * y, grp, 0));
                const f4 b1 = *reinterpret_cast<const f4 *>(s.vec + kVecBeta * kC + pair_row(2 * y + 1, grp, 0));
                us[y] = O::template sum<PL>(du[2 * y] * b0, du[2 * y + 1] * b1);
            }
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int y = tt / 2; y < 2; ++y)
                    dx[tt] = O::mul(dx[tt],
                                    O::template planes<PL>(
                                        s.inv + pair_row16(tt, r16) * Block::Inv::STRIDE + 32 * y + 8 * grp,
                                        Block::Inv::PLANE),
                                    us[y]);
        }
        if (live) {
            float *to = p.dx + chunk * kC * a.V + v;
            const int64_t at = ((b * a.L + c * kC) * a.H + h) * a.V + v;
            const int step = a.H * a.V;
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = pair_row(tt, grp, i);
                    to[t * a.V] = dx[tt][i];
                    if (whole || c * kC + t < a.L) store_io<IO>(p.dv, at + (int64_t)t * step, dx[tt][i]);
                }
        }
        // dS <- through dS + (scale enter Q)^T dO - (enter K)^T dX
        typename O::template Sum<PL> qs[2], xs[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            f4 qo[2], kx[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                qo[j] = dout[2 * y + j] *
                        *reinterpret_cast<const f4 *>(s.vec + kVecQEnter * kC + pair_row(2 * y + j, grp, 0));
                kx[j] = -dx[2 * y + j] *
                        *reinterpret_cast<const f4 *>(s.vec + kVecKEnter * kC + pair_row(2 * y + j, grp, 0));
            }
            qs[y] = O::template sum<PL>(qo[0], qo[1]);
            xs[y] = O::template sum<PL>(kx[0], kx[1]);
        }
        const float through = s.vec[kVecThrough * kC];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ds[kt][i] = through != 0.0f ? through * ds[kt][i] : 0.0f;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                typename O::Ex lq, lk;
                if constexpr (Lds::kTransposed) {
                    lq = O::load(s.qt + pair_row16(kt, r16) * Rows::TSTRIDE + 32 * y + 8 * grp);
                    lk = O::load(s.kt + pair_row16(kt, r16) * Rows::TSTRIDE + 32 * y + 8 * grp);
                } else {
                    lq = Op<IO>::gather(s.q + (32 * y + 8 * grp) * Rows::STRIDE + pair_row16(kt, r16), Rows::STRIDE);
                    lk = Op<IO>::gather(s.k + (32 * y + 8 * grp) * Rows::STRIDE + pair_row16(kt, r16), Rows::STRIDE);
                }
                ds[kt] = O::mul(ds[kt], lq, qs[y]);
                ds[kt] = O::mul(ds[kt], lk, xs[y]);
            }
        }
    }
    if (p.dh0 && live) store_state<KT>(p.dh0 + head * a.K * a.V + v, a.K, a.V, grp, ds);
}

// --------------------------------------------------------------------------- all chunks at once
constexpr int kGradThreads = 512, kVB = 32;  // value channels of a pass

struct GradArgs {
    Call a;
    const float *ck, *after, *dx, *edu;
    const void *dout;
    void *dq, *dk, *dbeta;
    float *dg;
};

// `P` planes of ROWS x 32 numbers in LDS.
template <typename IO, int ROWS, int P>
struct Slab {
    using E = typename Op<IO>::elem;
    static constexpr int PLANES = IO::bytes == 2 ? P : 1;
    static constexpr int STRIDE = kVB + 16 / IO::bytes, PLANE = ROWS * STRIDE;
    alignas(16) E e[PLANES * PLANE];
    __device__ __forceinline__ void put4(int row, int col, f4 v) {
        if constexpr (IO::bytes == 4) {
            *reinterpret_cast<f4 *>(e + row * STRIDE + col) = v;
        } else {
#pragma unroll
            for (int p = 0; p < PLANES; ++p) {
                b4 q;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    q[i] = (__bf16)v[i];
                    v[i] -= (float)q[i];
                }
                *reinterpret_cast<b4 *>(e + p * PLANE + row * STRIDE + col) = q;
            }
        }
    }
    __device__ __forceinline__ auto get(int row, int col) const {
        return Op<IO>::template planes<PLANES>(e + row * STRIDE + col, PLANE);
    }
};

template <typename IO, int KP>
struct GradLds {
    using Rows = HeadRows<IO, KP>;
    using E = typename Op<IO>::elem;
    using Mat = ChunkMatrix<IO, 2>;  // these feed outputs of the tensors' type alone
    static constexpr bool kTransposed = IO::bytes == 2;
    alignas(16) E q[kC * Rows::STRIDE], k[kC * Rows::STRIDE];
    Gates gates;
    float row_z[4][kC], col_z[4][kC], col_by[4][kC];
    float row_a[KP / 16][kC], row_b[KP / 16][kC];
    float dots[kGradThreads / 64];
    alignas(16) union {
        struct {
            Slab<IO, kC, 1> dout;
            Slab<IO, kC, 3> dx, err;
            Slab<IO, KP, 3> before, after;
        } in;
        struct {
            alignas(16) E kt[kTransposed ? KP * Rows::TSTRIDE : 8], qt[kTransposed ? KP * Rows::TSTRIDE : 8];
            alignas(16) E m1[Mat::PLANES * Mat::PLANE], m2[Mat::PLANES * Mat::PLANE], m3[Mat::PLANES * Mat::PLANE];
        } out;
    };
};

// The lower tiles of the 64 x 64 matrices, dealt to eight waves: tile `i` of ten.
__device__ __forceinline__ void lower_tile(int i, int &ti, int &tj) {
    ti = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3;
    tj = i - ti * (ti + 1) / 2;
}

__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int d = 1; d < 16; d *= 2) x += __shfl_xor(x, d, 64);
    return x;
}

// One chunk of one key head, over the value heads that share it.  Wave w has the result columns
// 16 (w % KT) .. + 15 of the products with K channels and, with KP = 64, half of their rows.
template <typename IO, int KP>
__global__ __launch_bounds__(kGradThreads) void grads_kernel(GradArgs p) {
    using O = Op<IO>;
    using E = typename O::elem;
    using Rows = HeadRows<IO, KP>;
    using Lds = GradLds<IO, KP>;
    using Mat = typename Lds::Mat;
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
    __syncthreads();
    if (threadIdx.x < 256) {
        const int row = threadIdx.x / 4, part = threadIdx.x % 4;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const E *x = (which ? s.k : s.q) + row * Rows::STRIDE + part * (KP / 4);
            float t = 0.0f;
#pragma unroll
            for (int i = 0; i < KP / 4; ++i) t = __builtin_fmaf((float)x[i], (float)x[i], t);
            t += __shfl_xor(t, 1, 64);
            t += __shfl_xor(t, 2, 64);
            if (part == 0) (which ? s.gates.rk : s.gates.rq)[row] = a.l2norm ? 1.0f / sqrtf(t + kL2Eps) : 1.0f;
        }
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
        load_gates<IO>(a, b, h, t0, s.gates);
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
                os[j] = O::mul(os[j], O::load(s.in.dout.e + t * Slab<IO, kC, 1>::STRIDE + 8 * grp), sb);
                xs[j] = O::mul(xs[j], s.in.dx.get(t, 8 * grp), sb);
                es[j] = O::mul(es[j], s.in.err.get(t, 8 * grp), sa);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (wave + 8 * j < 10) {
                    int ti, tj;
                    lower_tile(wave + 8 * j, ti, tj);
                    const auto e = s.in.err.get(16 * tj + r16, 8 * grp);
                    dp[j] = O::mul(dp[j], O::load(s.in.dout.e + (16 * ti + r16) * Slab<IO, kC, 1>::STRIDE + 8 * grp), e);
                    yy[j] = O::mul(yy[j], s.in.dx.get(16 * ti + r16, 8 * grp), e);
                }
        }
        __syncthreads();  // the slabs make room for the matrices
#pragma unroll
        for (int d = 1; d < 64; d *= 2) dot += __shfl_xor(dot, d, 64);
        if (lane == 0) s.dots[wave] = dot;
        if constexpr (Lds::kTransposed)
            for (int i = tid; i < kC * KP; i += kGradThreads) {
                const int t = i % kC, k = i / kC;
                s.out.kt[k * Rows::TSTRIDE + t] = s.k[t * Rows::STRIDE + k];
                s.out.qt[k * Rows::TSTRIDE + t] = s.q[t * Rows::STRIDE + k];
            }
        for (int i = tid; i < Mat::PLANES * Mat::PLANE; i += kGradThreads) {
            s.out.m1[i] = (E)0.0f;
            s.out.m2[i] = (E)0.0f;
            s.out.m3[i] = (E)0.0f;
        }
        __syncthreads();
        const auto put = [](E *m, int r, int q, float v) {
#pragma unroll
            for (int i = 0; i < Mat::PLANES; ++i) {
                const E e = (E)v;
                m[i * Mat::PLANE + r * Mat::STRIDE + q] = e;
                v -= (float)e;
            }
        };
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
                        put(s.out.m1, t, u, sq * rku);
                        put(s.out.m2, u, t, sq * rqt);
                    }
                    if (u < t) {
                        put(s.out.m3, t, u, sb * rku);
                        put(s.out.m3, u, t, sb * rkt);
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
            for (int d = 1; d < 64; d *= 2) {
                const double down = __shfl_down(dG, d, 64);
                if (t + d < 64) dG += down;
            }
            const int strips = (a.V + 15) / 16;
            for (int i = 0; i < strips; ++i) dbeta += p.edu[(chunk * strips + i) * kC + t];
            const bool cut = s.gates.doc[t] != (t ? s.gates.doc[t - 1] : 0);
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
                    kr = O::load(s.out.kt + (16 * kd + r16) * Rows::TSTRIDE + 32 * y + 8 * grp);
                    qr = O::load(s.out.qt + (16 * kd + r16) * Rows::TSTRIDE + 32 * y + 8 * grp);
                } else {
                    kr = Op<IO>::gather(s.k + (32 * y + 8 * grp) * Rows::STRIDE + 16 * kd + r16, Rows::STRIDE);
                    qr = Op<IO>::gather(s.q + (32 * y + 8 * grp) * Rows::STRIDE + 16 * kd + r16, Rows::STRIDE);
                }
                const int at = (16 * ti + r16) * Mat::STRIDE + 32 * y + 8 * grp;
                if (y <= ti / 2) dq[j] = O::mul(dq[j], O::template planes<Mat::PLANES>(s.out.m1 + at, Mat::PLANE), kr);
                if (y >= ti / 2) dk[j] = O::mul(dk[j], O::template planes<Mat::PLANES>(s.out.m2 + at, Mat::PLANE), qr);
                dk[j] = O::mul(dk[j], O::template planes<Mat::PLANES>(s.out.m3 + at, Mat::PLANE), kr);
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
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 16 * (first + j) + 4 * grp + i, k = 16 * kd + r16;
            if (t0 + t >= a.L || k >= a.K) continue;
            float oq = dq[j][i], ok = dk[j][i];
            if (a.l2norm) {
                float qd = 0.0f, kdot = 0.0f;
#pragma unroll
                for (int w = 0; w < KT; ++w) {
                    qd += s.row_a[w][t];
                    kdot += s.row_b[w][t];
                }
                const float rq = s.gates.rq[t], rk = s.gates.rk[t];
                oq = rq * (oq - rq * (float)s.q[t * Rows::STRIDE + k] * qd);
                ok = rk * (ok - rk * (float)s.k[t * Rows::STRIDE + k] * kdot);
            }
            const int64_t at = ((b * a.L + t0 + t) * a.Hk + hk) * a.K + k;
            store_io<IO>(p.dq, at, oq);
            store_io<IO>(p.dk, at, ok);
        }
}

template <typename IO, int KP>
hipError_t backward(const BackArgs &p, const GradArgs &g, hipStream_t stream) {
    const unsigned per = 16 * (kThreads / 64);
    const dim3 grid(((unsigned)p.a.V + per - 1) / per, (unsigned)p.a.H, (unsigned)p.a.B);
    back_chain_kernel<IO, KP><<<grid, kThreads, sizeof(BackLds<IO, KP>), stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 chunks((unsigned)p.a.n, (unsigned)p.a.Hk, (unsigned)p.a.B);
    grads_kernel<IO, KP><<<chunks, kGradThreads, sizeof(GradLds<IO, KP>), stream>>>(g);
    return hipGetLastError();
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct BackPlan {
    size_t blocks, after, dx, edu, ck, total;
};

BackPlan back_plan(const ssm_gated_delta_bwd_args_t &a) {
    const size_t n = (size_t)((a.seqlen + kC - 1) / kC), chunks = n * a.batch * a.heads;
    BackPlan p;
    p.blocks = 0;
    p.after = up256(chunks * block_bytes(a.io_dtype));
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
    const BackArgs p{c, ws, ck, a.dh_final, a.dout, a.dv, a.dh0, after, dx, edu};
    const GradArgs g{c, ck, after, dx, edu, a.dout, a.dq, a.dk, a.dbeta, a.dg};
    if (a.io_dtype == SSM_BF16)
        return a.kdim <= 64 ? backward<io_bf16, 64>(p, g, stream) : backward<io_bf16, 128>(p, g, stream);
    return a.kdim <= 64 ? backward<io_f32, 64>(p, g, stream) : backward<io_f32, 128>(p, g, stream);
}

size_t backward_bytes(const ssm_gated_delta_bwd_args_t &a) { return back_plan(a).total; }

}  // namespace delta
}  // namespace ssm
