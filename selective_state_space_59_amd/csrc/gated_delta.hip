// gated_delta.hip -- the gated delta rule (ssm_gated_delta_fwd, _step) on gfx950.  Per head, with a
// state S of K x V:
//   S' = e^{g_t} S_{t-1},  e_t = v_t - S'^T k_t,  S_t = S' + beta_t k_t e_t^T,  o_t = scale S_t^T q_t
// In chunks of 64 steps, with G the running sum of g in the chunk, D_ts = e^{G_t - G_s} (0 across a
// reset), enter_t = e^{G_t}, leave_t = e^{G_end - G_t}, through = e^{G_end} and S the state entering:
//   B_ts = D_ts k_t.k_s (s < t),  P_ts = scale D_ts q_t.k_s (s <= t)
//   (I + B diag(beta)) E = V - enter K S                 the steps' errors, triangular
//   O  = scale enter Q S + P diag(beta) E
//   S <- through S + (leave K)^T diag(beta) E
// prepare_kernel forms the inverse of I + B diag(beta) and P for every chunk at once; chain_kernel
// then carries the states from chunk to chunk, each wave the 16 value channels whose states it holds in
// registers, apart from the others.
#include "delta_tile.h"

#include <algorithm>

namespace ssm {
namespace delta {
namespace {

// ---------------------------------------------------------------------------------- chunks
template <typename IO, int KP>
struct PrepareLds {
    using Rows = HeadRows<IO, KP>;
    alignas(16) typename Op<IO>::elem q[kC * Rows::STRIDE], k[kC * Rows::STRIDE];
    alignas(16) float a[kC][kC + 4];    // B diag(beta)
    alignas(16) float inv[kC][20];      // the inverses of its diagonal blocks, side by side: row, column within the block
    Gates gates;
};

// Reciprocal norms of the 64 rows (1 without l2norm), four lanes a row of the first 256 threads.
template <typename IO, int KP>
__device__ __forceinline__ void row_norms(const typename Op<IO>::elem *rows, bool l2norm, float *out) {
    if (threadIdx.x >= 256) return;
    const int row = threadIdx.x / 4, part = threadIdx.x % 4;
    float s = 0.0f;
    if (l2norm) {
        const auto *p = rows + row * HeadRows<IO, KP>::STRIDE + part * (KP / 4);
#pragma unroll
        for (int i = 0; i < KP / 4; ++i) s = __builtin_fmaf((float)p[i], (float)p[i], s);
        s += __shfl_xor(s, 1, 64);
        s += __shfl_xor(s, 2, 64);
    }
    if (part == 0) out[row] = l2norm ? 1.0f / sqrtf(s + kL2Eps) : 1.0f;
}

// One chunk of one head: wave w owns the rows 16 w .. + 15 of the two products K K^T and Q K^T, inverts
// its diagonal block of I + B diag(beta) by substitution (a column a lane), and then solves block column
// w of the inverse downwards.  Entries of the inverse stay of the size of the states' own factors, where
// powers of B would not, so equal keys in a row cost no digits.
template <typename IO, int KP, bool BWD>
__global__ __launch_bounds__(kThreads) void prepare_kernel(Call a, char *blocks) {
    using O = Op<IO>;
    using E = typename O::elem;
    using Rows = HeadRows<IO, KP>;
    using Block = ChunkBlock<IO>;
    __shared__ __attribute__((aligned(16))) PrepareLds<IO, KP> s;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane % 16, grp = lane / 16;
    const int64_t c = blockIdx.x, b = blockIdx.z;
    const int h = blockIdx.y, hk = h / (a.H / a.Hk);
    const int64_t t0 = c * kC;
    {
        typename Rows::template Regs<4> rq, rk;
        Rows::template load<4>(rq, a.q, b * a.q_batch + (int64_t)hk * a.K, a.q_token, t0, a.L, a.K);
        Rows::template load<4>(rk, a.k, b * a.k_batch + (int64_t)hk * a.K, a.k_token, t0, a.L, a.K);
        load_gates<IO>(a, b, h, t0, s.gates);
        Rows::template cut<4>(rq, t0, a.L, a.K);
        Rows::template cut<4>(rk, t0, a.L, a.K);
        Rows::template store<4>(rq, s.q);
        Rows::template store<4>(rk, s.k);
    }
    __syncthreads();
    row_norms<IO, KP>(s.q, a.l2norm, s.gates.rq);
    row_norms<IO, KP>(s.k, a.l2norm, s.gates.rk);
    __syncthreads();

    char *block = blocks + ((b * a.H + h) * a.n + c) * Block::kBytes;
    float *vec = reinterpret_cast<float *>(block);
    E *inv = reinterpret_cast<E *>(block + Block::kVecBytes);
    E *att = reinterpret_cast<E *>(block + Block::kVecBytes + Block::kInvBytes);
    if (threadIdx.x < kC) {
        const int t = threadIdx.x;
        vec[kVecKEnter * kC + t] = s.gates.enter[t] * s.gates.rk[t];
        vec[kVecKLeave * kC + t] = s.gates.leave[t] * s.gates.rk[t];
        vec[kVecQEnter * kC + t] = a.scale * s.gates.enter[t] * s.gates.rq[t];
        vec[kVecBeta * kC + t] = s.gates.beta[t];
        vec[kVecThrough * kC + t] = s.gates.through;
    }

    typename O::Ex qa[KP / 32], ka[KP / 32];
#pragma unroll
    for (int x = 0; x < KP / 32; ++x) {
        qa[x] = O::load(s.q + (16 * wave + r16) * Rows::STRIDE + 32 * x + 8 * grp);
        ka[x] = O::load(s.k + (16 * wave + r16) * Rows::STRIDE + 32 * x + 8 * grp);
    }
    for (int j = 0; j < 4; ++j) {
        f4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
        const int u = 16 * j + r16;
        if (j <= wave) {
#pragma unroll
            for (int x = 0; x < KP / 32; ++x) {
                const typename O::Ex kb = O::load(s.k + u * Rows::STRIDE + 32 * x + 8 * grp);
                kk = O::mul(kk, ka[x], kb);
                qk = O::mul(qk, qa[x], kb);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * wave + 4 * grp + i;
                const float d = decay(s.gates, t, u) * s.gates.rk[u];
                qk[i] *= a.scale * d * s.gates.rq[t];
                s.a[t][u] = u < t ? kk[i] * d * s.gates.rk[t] * s.gates.beta[u] : 0.0f;
            }
        } else if (j != (wave ^ 1)) {
            continue;  // above the pairs of tiles that are read
        }
        if constexpr (BWD) {
            Block::AttT::put4(att, u, 16 * wave + 4 * grp, qk);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) Block::Att::put(att, 16 * wave + 4 * grp + i, u, qk[i]);
        }
    }
    __syncthreads();
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float v = i == r16 ? 1.0f : 0.0f;
#pragma unroll
        for (int k = 0; k < i; ++k) v = __builtin_fmaf(-s.a[16 * wave + i][16 * wave + k], x[k], v);
        x[i] = v;
    }
    if (grp == 0)
#pragma unroll
        for (int i = 0; i < 16; ++i) s.inv[16 * wave + i][r16] = x[i];
    __syncthreads();

    // block column `wave`: N_jj, then N_ij = -N_ii sum_{k < i} A_ik N_kj
    f4 col[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f4 v = {0, 0, 0, 0};
        if (i == wave) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = s.inv[16 * i + 4 * grp + e][r16];
        } else if (i > wave) {
            f4 acc = {0, 0, 0, 0};
            for (int k = 0; k < i; ++k)
                if (k >= wave) {
                    const f4 left = *reinterpret_cast<const f4 *>(&s.a[16 * i + r16][16 * k + 4 * grp]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // (col is indexed by a loop variable: picked without an address)
                        const float right = k == 0 ? col[0][e] : k == 1 ? col[1][e] : col[2][e];
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(left[e], right, acc, 0, 0, 0);
                    }
                }
            const f4 left = *reinterpret_cast<const f4 *>(&s.inv[16 * i + r16][4 * grp]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v = __builtin_amdgcn_mfma_f32_16x16x4f32(left[e], -acc[e], v, 0, 0, 0);
        }
        col[i] = v;
        if (i >= wave || i == (wave ^ 1)) {
            if constexpr (BWD) {
                Block::Inv::put4(inv, 16 * wave + r16, 16 * i + 4 * grp, v);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) Block::Inv::put(inv, 16 * i + 4 * grp + e, 16 * wave + r16, v[e]);
            }
        }
    }
}

// ----------------------------------------------------------------------------------- chain
template <typename IO, int KP>
struct ChainLds {
    using Rows = HeadRows<IO, KP>;
    using Block = ChunkBlock<IO>;
    using E = typename Op<IO>::elem;
    static constexpr bool kTransposed = IO::bytes == 2;
    alignas(16) E q[kC * Rows::STRIDE], k[kC * Rows::STRIDE];
    alignas(16) E kt[kTransposed ? KP * Rows::TSTRIDE : 8];
    alignas(16) E inv[Block::Inv::PLANES * Block::Inv::PLANE], att[Block::Att::PLANES * Block::Att::PLANE];
    alignas(16) float vec[kVecs * kC];
};

struct ChainArgs {
    Call a;
    const char *blocks;
    const float *h0;
    void *o;
    float *h_final, *ck;
};

template <typename IO, int KP>
__global__ __launch_bounds__(kThreads) void chain_kernel(ChainArgs p) {
    using O = Op<IO>;
    using E = typename O::elem;
    using Rows = HeadRows<IO, KP>;
    using Block = ChunkBlock<IO>;
    using Lds = ChainLds<IO, KP>;
    constexpr int KT = KP / 16, PL = O::kPlanes, OUT = PL == 1 ? 1 : 2;
    extern __shared__ __attribute__((aligned(16))) char raw[];
    Lds &s = *reinterpret_cast<Lds *>(raw);
    const Call &a = p.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane % 16, grp = lane / 16;
    const int64_t b = blockIdx.z;
    const int h = blockIdx.y, hk = h / (a.H / a.Hk);
    // lanes past the last channel repeat it and store nothing
    const int vw = (blockIdx.x * (kThreads / 64) + wave) * 16 + r16, v = min(vw, a.V - 1);
    const bool live = vw < a.V;
    const int64_t head = b * a.H + h;
    const char *blocks = p.blocks + head * a.n * Block::kBytes;
    const int64_t q_off = b * a.q_batch + (int64_t)hk * a.K, k_off = b * a.k_batch + (int64_t)hk * a.K;
    const int64_t v_off = b * a.v_batch + (int64_t)h * a.V + v;

    f4 state[KT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = pair_row(kt, grp, i);
            state[kt][i] = p.h0 && k < a.K ? p.h0[(head * a.K + k) * a.V + v] : 0.0f;
        }

    // the next chunk's tiles, on their way while this one is computed
    typename Rows::template Regs<4> rq, rk;
    typename Block::Inv::template Regs<kThreads> rinv;
    typename Block::Att::template Regs<kThreads> ratt;
    float rvec[2];
    RawOne<IO> rv[4][4];
    const auto fetch = [&](int64_t c) {
        const char *block = blocks + c * Block::kBytes;
        Rows::template load<4>(rq, a.q, q_off, a.q_token, c * kC, a.L, a.K);
        Rows::template load<4>(rk, a.k, k_off, a.k_token, c * kC, a.L, a.K);
        Block::Inv::template load<kThreads>(rinv, reinterpret_cast<const E *>(block + Block::kVecBytes));
        Block::Att::template load<kThreads>(
            ratt, reinterpret_cast<const E *>(block + Block::kVecBytes + Block::kInvBytes));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = min((int)threadIdx.x + kThreads * i, kVecs * kC - 1);
            rvec[i] = reinterpret_cast<const float *>(block)[at];
        }
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t t = c * kC + pair_row(tt, grp, i);
                rv[tt][i] = load_one<IO>(a.v, v_off + (t < a.L ? t : a.L - 1) * a.v_token);
            }
    };
    fetch(0);
    for (int64_t c = 0; c < a.n; ++c) {
        __syncthreads();  // the last chunk's tiles have been read
        const bool whole = (c + 1) * kC <= a.L;
        Rows::template cut<4>(rq, c * kC, a.L, a.K);
        Rows::template cut<4>(rk, c * kC, a.L, a.K);
        Rows::template store<4>(rq, s.q);
        Rows::template store<4>(rk, s.k);
        if constexpr (Lds::kTransposed) Rows::template store_transposed<4>(rk, s.kt);
        Block::Inv::template store<kThreads>(rinv, s.inv);
        Block::Att::template store<kThreads>(ratt, s.att);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = threadIdx.x + kThreads * i;
            if (at < kVecs * kC) s.vec[at] = rvec[i];
        }
        f4 val[4];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                val[tt][i] = whole || c * kC + pair_row(tt, grp, i) < a.L ? rv[tt][i].get() : 0.0f;
        __syncthreads();
        if (c + 1 < a.n) fetch(c + 1);

        float *ck = p.ck ? p.ck + (((c * a.B + b) * a.H + h) * (a.K + kC)) * a.V + v : nullptr;
        if (ck && live) store_state<KT>(ck, a.K, a.V, grp, state);

        // K S and Q S
        f4 ks[4] = {}, qs[4] = {};
#pragma unroll
        for (int x = 0; x < KT / 2; ++x) {
            const auto st = O::template sum<PL>(state[2 * x], state[2 * x + 1]);
            typename O::template Sum<OUT> so;
            if constexpr (PL == 1) {
                so = st;
            } else {
                so.p[0] = st.p[0];
                so.p[1] = st.p[1];
            }
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                const int row = pair_row16(tt, r16);
                ks[tt] = O::mul(ks[tt], O::load(s.k + row * Rows::STRIDE + 32 * x + 8 * grp), st);
                qs[tt] = O::mul(qs[tt], O::load(s.q + row * Rows::STRIDE + 32 * x + 8 * grp), so);
            }
        }
        // X = V - enter K S (a state that does not reach a step has no part in it, whatever it holds)
        f4 err[4] = {};
        typename O::template Sum<PL> xs[2];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
            const f4 en = *reinterpret_cast<const f4 *>(s.vec + kVecKEnter * kC + pair_row(tt, grp, 0));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (en[i] != 0.0f) val[tt][i] = __builtin_fmaf(-en[i], ks[tt][i], val[tt][i]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) xs[y] = O::template sum<PL>(val[2 * y], val[2 * y + 1]);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
            for (int y = 0; y <= tt / 2; ++y)
                err[tt] = O::mul(err[tt],
                                 O::template planes<PL>(s.inv + pair_row16(tt, r16) * Block::Inv::STRIDE + 32 * y + 8 * grp,
                                                        Block::Inv::PLANE),
                                 xs[y]);
        if (ck && live)
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) ck[(int64_t)(a.K + pair_row(tt, grp, i)) * a.V] = err[tt][i];
        // S <- through S + (leave K)^T diag(beta) E
        f4 u[4];
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
            u[tt] = err[tt] * *reinterpret_cast<const f4 *>(s.vec + kVecBeta * kC + pair_row(tt, grp, 0));
        {
            typename O::template Sum<PL> ws[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const f4 l0 = *reinterpret_cast<const f4 *>(s.vec + kVecKLeave * kC + pair_row(2 * y, grp, 0));
                const f4 l1 = *reinterpret_cast<const f4 *>(s.vec + kVecKLeave * kC + pair_row(2 * y + 1, grp, 0));
                ws[y] = O::template sum<PL>(u[2 * y] * l0, u[2 * y + 1] * l1);
            }
            const float through = s.vec[kVecThrough * kC];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) state[kt][i] = through != 0.0f ? through * state[kt][i] : 0.0f;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    typename O::Ex left;
                    if constexpr (Lds::kTransposed)
                        left = O::load(s.kt + pair_row16(kt, r16) * Rows::TSTRIDE + 32 * y + 8 * grp);
                    else
                        left = Op<IO>::gather(s.k + (32 * y + 8 * grp) * Rows::STRIDE + pair_row16(kt, r16), Rows::STRIDE);
                    state[kt] = O::mul(state[kt], left, ws[y]);
                }
            }
        }
        // O = scale enter Q S + P diag(beta) E
        if (p.o) {
            typename O::template Sum<OUT> us[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) us[y] = O::template sum<OUT>(u[2 * y], u[2 * y + 1]);
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) {
                const f4 en = *reinterpret_cast<const f4 *>(s.vec + kVecQEnter * kC + pair_row(tt, grp, 0));
#pragma unroll
                for (int i = 0; i < 4; ++i) qs[tt][i] = en[i] != 0.0f ? en[i] * qs[tt][i] : 0.0f;
#pragma unroll
                for (int y = 0; y <= tt / 2; ++y)
                    qs[tt] = O::mul(qs[tt],
                                    O::template planes<OUT>(
                                        s.att + pair_row16(tt, r16) * Block::Att::STRIDE + 32 * y + 8 * grp,
                                        Block::Att::PLANE),
                                    us[y]);
            }
            if (live) {
                const int64_t at = ((b * a.L + c * kC) * a.H + h) * a.V + v;
                const int step = a.H * a.V;
#pragma unroll
                for (int tt = 0; tt < 4; ++tt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = pair_row(tt, grp, i);
                        if (whole || c * kC + t < a.L) store_io<IO>(p.o, at + (int64_t)t * step, qs[tt][i]);
                    }
            }
        }
    }
    if (p.h_final && live) store_state<KT>(p.h_final + head * a.K * a.V + v, a.K, a.V, grp, state);
}

// ------------------------------------------------------------------------------------ step
// One token: a workgroup of four waves owns one head's columns v0 .. v0 + 31, eight threads side by side
// (4 columns each) times 32 rows apart.  The state is read once, held in registers (KP / 32 rows a thread),
// and written once; S^T k and S^T q go through the same two reductions, o = scale (S'^T q + (q.k) u).
constexpr int kStepV = 32, kStepRows = kThreads / (kStepV / 4);

struct StepArgs {
    Call a;
    float *state;
    void *o;
};

template <typename IO, int KP>
__global__ __launch_bounds__(kThreads) void step_kernel(StepArgs p) {
    constexpr int R = KP / kStepRows;
    __shared__ float qs[KP], ks[KP], part[2][4][kStepV], dots[4][3];
    const Call &a = p.a;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = threadIdx.x % (kStepV / 4), row = threadIdx.x / (kStepV / 4);
    const int h = blockIdx.y, hk = h / (a.H / a.Hk);
    const int64_t b = blockIdx.z;
    const int v0 = blockIdx.x * kStepV + 4 * col;
    const bool live = v0 < a.V;
    float *state = p.state + ((b * a.H + h) * a.K) * a.V + v0;
    f4 s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int k = row + kStepRows * r;
        s[r] = live && k < a.K ? *reinterpret_cast<const f4 *>(state + (int64_t)k * a.V) : f4{0, 0, 0, 0};
    }
    // q, k and the sums q.q, k.k, q.k
    float q = 0.0f, k = 0.0f;
    if (threadIdx.x < KP) {
        if ((int)threadIdx.x < a.K) {
            q = load_io<IO>(a.q, b * a.q_batch + (int64_t)hk * a.K + threadIdx.x);
            k = load_io<IO>(a.k, b * a.k_batch + (int64_t)hk * a.K + threadIdx.x);
        }
        qs[threadIdx.x] = q;
        ks[threadIdx.x] = k;
    }
    float qq = q * q, kk = k * k, qk = q * k;
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) {
        qq += __shfl_xor(qq, d, 64);
        kk += __shfl_xor(kk, d, 64);
        qk += __shfl_xor(qk, d, 64);
    }
    if (lane == 0) {
        dots[wave][0] = qq;
        dots[wave][1] = kk;
        dots[wave][2] = qk;
    }
    __syncthreads();
    qq = dots[0][0] + dots[1][0] + dots[2][0] + dots[3][0];
    kk = dots[0][1] + dots[1][1] + dots[2][1] + dots[3][1];
    qk = dots[0][2] + dots[1][2] + dots[2][2] + dots[3][2];
    const float rq = a.l2norm ? 1.0f / sqrtf(qq + kL2Eps) : 1.0f, rk = a.l2norm ? 1.0f / sqrtf(kk + kL2Eps) : 1.0f;
    const int64_t at = b * a.H + h;
    const float g = a.g[at];
    const bool cut = (a.reset && a.reset[b]) || g < kForget;
    const float decay = expf(g), beta = load_io<IO>(a.beta, at);
    f4 sk = {0, 0, 0, 0}, sq = {0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float kr = ks[row + kStepRows * r], qr = qs[row + kStepRows * r];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[r][i] = cut ? 0.0f : decay * s[r][i];
            sk[i] = __builtin_fmaf(kr, s[r][i], sk[i]);
            sq[i] = __builtin_fmaf(qr, s[r][i], sq[i]);
        }
    }
#pragma unroll
    for (int d = kStepV / 4; d < 64; d *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sk[i] += __shfl_xor(sk[i], d, 64);
            sq[i] += __shfl_xor(sq[i], d, 64);
        }
    if (lane < kStepV / 4) {
        *reinterpret_cast<f4 *>(&part[0][wave][4 * col]) = sk;
        *reinterpret_cast<f4 *>(&part[1][wave][4 * col]) = sq;
    }
    __syncthreads();
    if (!live) return;
    sk = sq = f4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        sk += *reinterpret_cast<const f4 *>(&part[0][w][4 * col]);
        sq += *reinterpret_cast<const f4 *>(&part[1][w][4 * col]);
    }
    f4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float val = load_io<IO>(a.v, b * a.v_batch + (int64_t)h * a.V + v0 + i);
        u[i] = beta * __builtin_fmaf(-rk, sk[i], val);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int k = row + kStepRows * r;
        const float kr = rk * ks[k];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[r][i] = __builtin_fmaf(kr, u[i], s[r][i]);
        if (k < a.K) *reinterpret_cast<f4 *>(state + (int64_t)k * a.V) = s[r];
    }
    if (row == 0)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            store_io<IO>(p.o, at * a.V + v0 + i, a.scale * rq * __builtin_fmaf(rk * qk, u[i], sq[i]));
}

template <typename IO, int KP>
hipError_t prepare(const Call &a, bool backward, char *blocks, hipStream_t stream) {
    const dim3 grid((unsigned)a.n, (unsigned)a.H, (unsigned)a.B);
    if (backward)
        prepare_kernel<IO, KP, true><<<grid, kThreads, 0, stream>>>(a, blocks);
    else
        prepare_kernel<IO, KP, false><<<grid, kThreads, 0, stream>>>(a, blocks);
    return hipGetLastError();
}

template <typename IO, int KP>
hipError_t chain(const ChainArgs &p, hipStream_t stream) {
    const unsigned per = 16 * (kThreads / 64);
    const dim3 grid(((unsigned)p.a.V + per - 1) / per, (unsigned)p.a.H, (unsigned)p.a.B);
    chain_kernel<IO, KP><<<grid, kThreads, sizeof(ChainLds<IO, KP>), stream>>>(p);
    return hipGetLastError();
}

template <typename IO, int KP>
hipError_t step(const StepArgs &p, hipStream_t stream) {
    const dim3 grid(((unsigned)p.a.V + kStepV - 1) / kStepV, (unsigned)p.a.H, (unsigned)p.a.B);
    step_kernel<IO, KP><<<grid, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

size_t block_bytes(int io_dtype) {
    return io_dtype == SSM_BF16 ? ChunkBlock<io_bf16>::kBytes : ChunkBlock<io_f32>::kBytes;
}

hipError_t launch_prepare(const Call &a, int io_dtype, bool backward, char *blocks, hipStream_t stream) {
    if (io_dtype == SSM_BF16)
        return a.K <= 64 ? prepare<io_bf16, 64>(a, backward, blocks, stream)
                         : prepare<io_bf16, 128>(a, backward, blocks, stream);
    return a.K <= 64 ? prepare<io_f32, 64>(a, backward, blocks, stream)
                     : prepare<io_f32, 128>(a, backward, blocks, stream);
}

hipError_t launch_chain(const Call &a, int io_dtype, const char *blocks, const float *h0, void *o, float *h_final,
                        float *ck, hipStream_t stream) {
    const ChainArgs p{a, blocks, h0, o, h_final, ck};
    if (io_dtype == SSM_BF16) return a.K <= 64 ? chain<io_bf16, 64>(p, stream) : chain<io_bf16, 128>(p, stream);
    return a.K <= 64 ? chain<io_f32, 64>(p, stream) : chain<io_f32, 128>(p, stream);
}

}  // namespace delta

namespace {

template <typename A>
delta::Call call_of(const A &a) {
    delta::Call c = {};
    c.q = a.q;
    c.k = a.k;
    c.v = a.v;
    c.g = a.g;
    c.beta = a.beta;
    c.reset = a.reset;
    c.B = a.batch;
    c.L = a.seqlen;
    c.n = (a.seqlen + delta::kC - 1) / delta::kC;
    c.Hk = (int)a.kheads;
    c.H = (int)a.heads;
    c.K = (int)a.kdim;
    c.V = (int)a.vdim;
    c.scale = a.scale;
    c.l2norm = a.l2norm;
    c.q_token = a.q_token ? a.q_token : a.kheads * a.kdim;
    c.k_token = a.k_token ? a.k_token : a.kheads * a.kdim;
    c.v_token = a.v_token ? a.v_token : a.heads * a.vdim;
    c.q_batch = a.q_token ? a.q_batch : a.seqlen * c.q_token;
    c.k_batch = a.k_token ? a.k_batch : a.seqlen * c.k_token;
    c.v_batch = a.v_token ? a.v_batch : a.seqlen * c.v_token;
    return c;
}

}  // namespace

size_t gated_delta_workspace_bytes(const ssm_gated_delta_args_t &a) {
    const int64_t n = (a.seqlen + delta::kC - 1) / delta::kC;
    return (size_t)(a.batch * a.heads * n) * delta::block_bytes(a.io_dtype);
}

hipError_t launch_gated_delta_fwd(const ssm_gated_delta_args_t &a, hipStream_t stream) {
    const delta::Call c = call_of(a);
    char *blocks = static_cast<char *>(a.workspace);
    const hipError_t e = delta::launch_prepare(c, a.io_dtype, false, blocks, stream);
    if (e != hipSuccess) return e;
    return delta::launch_chain(c, a.io_dtype, blocks, a.h0, a.o, a.h_final, a.checkpoints, stream);
}

size_t gated_delta_bwd_workspace_bytes(const ssm_gated_delta_bwd_args_t &a) { return delta::backward_bytes(a); }

hipError_t launch_gated_delta_bwd(const ssm_gated_delta_bwd_args_t &a, hipStream_t stream) {
    return delta::launch_backward(call_of(a), a, stream);
}

hipError_t launch_gated_delta_step(const ssm_gated_delta_step_args_t &a, hipStream_t stream) {
    delta::StepArgs p = {};
    p.a.q = a.q;
    p.a.k = a.k;
    p.a.v = a.v;
    p.a.g = a.g;
    p.a.beta = a.beta;
    p.a.reset = a.reset;
    p.a.B = a.batch;
    p.a.Hk = (int)a.kheads;
    p.a.H = (int)a.heads;
    p.a.K = (int)a.kdim;
    p.a.V = (int)a.vdim;
    p.a.scale = a.scale;
    p.a.l2norm = a.l2norm;
    p.a.q_batch = a.q_batch ? a.q_batch : a.kheads * a.kdim;
    p.a.k_batch = a.k_batch ? a.k_batch : a.kheads * a.kdim;
    p.a.v_batch = a.v_batch ? a.v_batch : a.heads * a.vdim;
    p.state = a.state;
    p.o = a.o;
    if (a.io_dtype == SSM_BF16)
        return a.kdim <= 64 ? delta::step<io_bf16, 64>(p, stream) : delta::step<io_bf16, 128>(p, stream);
    return a.kdim <= 64 ? delta::step<io_f32, 64>(p, stream) : delta::step<io_f32, 128>(p, stream);
}

}  // namespace ssm
