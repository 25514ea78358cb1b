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
// then carries the states from chunk to chunk, each workgroup 16 or 32 value channels apart from the others.
// Heads whose decays grow are done again step by step (gated_delta_grow.hip).
#include "delta_tile.h"

#include <algorithm>

namespace ssm {
namespace delta {
namespace {

// ---------------------------------------------------------------------------------- chunks
template <typename IO, int KP>
struct PrepareLds {
    using Rows = HeadRows<IO, KP>;
    alignas(16) typename Op<IO>::elem k[kC * Rows::STRIDE];
    union {
        alignas(16) typename Op<IO>::elem q[kC * Rows::STRIDE];
        alignas(16) float a[kC][kC + 4];  // B diag(beta), when the queries are in registers
    };
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
// powers of B would not, so equal keys in a row cost no digits.  8 x 2048 steps of 12 heads of 128, bf16: 73 us,
// bound by the substitution's latency (a third of a chunk's 20000 cycles) at three workgroups a CU.
template <typename IO, int KP, bool BWD>
__global__ __launch_bounds__(kThreads) void prepare_kernel(Call a, char *blocks, uint32_t *marks) {
    using O = Op<IO>;
    using E = typename O::elem;
    using Rows = HeadRows<IO, KP>;
    using Block = ChunkBlock<IO, KP, BWD>;
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
    if (threadIdx.x == 0) marks[(b * a.H + h) * a.n + c] = s.gates.grows;
    float *vec = reinterpret_cast<float *>(block);
    E *inv = reinterpret_cast<E *>(block + Block::kInv), *att = reinterpret_cast<E *>(block + Block::kAtt);
    if constexpr (BWD) {
        static_assert(sizeof(Gates) % 4 == 0, "");
        for (int i = threadIdx.x; i < (int)sizeof(Gates) / 4; i += kThreads)
            reinterpret_cast<uint32_t *>(block + Block::kGates)[i] = reinterpret_cast<const uint32_t *>(&s.gates)[i];
    }
    // keys and queries transposed, a lane's eight steps a piece
    for (int i = threadIdx.x; i < KP * kC / 8; i += kThreads) {
        const int k = i / 128 * 16 + i % 16, t = i / 64 % 2 * 32 + i / 16 % 4 * 8;
        alignas(16) E x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = s.k[(t + j) * Rows::STRIDE + k];
        __builtin_memcpy(block + Block::kKt + i * 8 * sizeof(E), x, 8 * sizeof(E));
        if constexpr (BWD) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = s.q[(t + j) * Rows::STRIDE + k];
            __builtin_memcpy(block + Block::kQt + i * 8 * sizeof(E), x, 8 * sizeof(E));
        }
    }
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
    __syncthreads();
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
            put_planes4<IO, Block::ATT, Block::PLANE>(att + tiled(u, 16 * wave + 4 * grp), qk);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                put_planes<IO, Block::ATT, Block::PLANE>(att + tiled(16 * wave + 4 * grp + i, u), qk[i]);
        }
    }
    __syncthreads();
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float v[4] = {i == r16 ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < i; k += 4) {
            const f4 left = *reinterpret_cast<const f4 *>(&s.a[16 * wave + i][16 * wave + k]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k + e < i) v[e] = __builtin_fmaf(-left[e], x[k + e], v[e]);
        }
        x[i] = (v[0] + v[1]) + (v[2] + v[3]);
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
                put_planes4<IO, Block::INV, Block::PLANE>(inv + tiled(16 * wave + r16, 16 * i + 4 * grp), v);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    put_planes<IO, Block::INV, Block::PLANE>(inv + tiled(16 * i + 4 * grp + e, 16 * wave + r16), v[e]);
            }
        }
    }
}

// ----------------------------------------------------------------------------------- chain
template <typename IO, int KP, int NC>
struct ChainLds {
    static constexpr int PL = Op<IO>::kPlanes, OUT = PL == 1 ? 1 : 2;
    Slab<IO, 16 * NC, KP, PL> state;  // column by column, as right operands
    Slab<IO, 16 * NC, kC, PL> x, w;   // X; leave diag(beta) E
    Slab<IO, 16 * NC, kC, OUT> u;     // diag(beta) E
};

struct ChainArgs {
    Call a;
    const char *blocks;
    const float *h0;
    void *o;
    float *h_final, *ck;
    float *parts;  // (heads, segments - 1): Z, K x V floats, and T transposed, K x K
    int64_t per;   // chunks of a segment
    int segments;
    bool wide;  // 32 value channels a workgroup in segments
    int slices;
};

// Four waves carry 16 NC value channels of one head along the chunks.  Wave w has the steps 16 w .. + 15 of
// the chunk in every product over steps and the rows KP/4 w .. of the state.  What it needs of the keys,
// queries and the chunk's matrices no other wave of the workgroup reads, so it comes from memory straight
// into registers, reloaded for the next chunk as soon as it has been used; only states, X and E go round
// through LDS, split into their planes once, by the wave that owns them.  Three barriers a chunk.
// What bounds it is a chunk's chain of products, each behind a barrier and a read of LDS: 2.5 us a chunk where
// a CU has one workgroup, of which 0.35 wait for loads.  8 x 2048 steps of 12 heads of 128, bf16: 175 us, 252
// with checkpoints (302 MB).
//
// A long sequence of few heads runs in segments.  The state that leaves a segment is T S + Z for the state S
// entering it; first (FIRST) all segments but the last form, without outputs, their Z (from a state of zeros,
// the first one's from h0) and, as K more columns without values, their T (from the identity); join_kernel
// turns these into the states entering the segments, and the chains run again from there.  32768 steps of 12
// heads of 128, bf16, ten segments: 337 us, 31 and 278; the whole call 790, in one piece 1410.
template <typename IO, int KP, int NC, bool FIRST>
__global__ __launch_bounds__(kThreads, 2) void chain_kernel(ChainArgs p) {
    using O = Op<IO>;
    using E = typename O::elem;
    using Block = ChunkBlock<IO, KP, false>;
    using Lds = ChainLds<IO, KP, NC>;
    constexpr int KX = KP / 32, ST = KP / 64, PL = Lds::PL, OUT = Lds::OUT;
    extern __shared__ __attribute__((aligned(16))) char raw[];
    Lds &s = *reinterpret_cast<Lds *>(raw);
    const Call &a = p.a;
    const int running = FIRST ? p.segments - 1 : p.segments;
    const ChainPlace place = chain_place(a.B * a.H * running, p.slices);
    if (!place.any) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane % 16, grp = lane / 16;
    const int64_t head = place.head / running, b = head / a.H;
    const int segment = (int)(place.head % running);
    const int64_t begin = segment * p.per, end = min(begin + p.per, a.n);
    const int h = (int)(head % a.H), hk = h / (a.H / a.Hk);
    const int row = 16 * wave + r16, mine = 16 * wave + 4 * grp;  // left operands' row; results' first row
    const char *blocks = p.blocks + head * a.n * Block::kBytes;
    const char *q_base = bytes(static_cast<const char *>(a.q), b * a.q_batch + (int64_t)hk * a.K, IO::bytes);
    const char *k_base = bytes(static_cast<const char *>(a.k), b * a.k_batch + (int64_t)hk * a.K, IO::bytes);
    const char *v_base = bytes(static_cast<const char *>(a.v), b * a.v_batch + (int64_t)h * a.V, IO::bytes);
    char *o_base = static_cast<char *>(p.o) + (b * a.L * a.H + h) * a.V * IO::bytes;
    const uint32_t q_step = (uint32_t)a.q_token * IO::bytes, k_step = (uint32_t)a.k_token * IO::bytes;
    const uint32_t v_step = (uint32_t)a.v_token * IO::bytes, o_step = (uint32_t)(a.H * a.V) * IO::bytes;
    // lanes past the last channels repeat them and store nothing
    const int value_slices = (a.V + 16 * NC - 1) / (16 * NC);
    const bool matrix = FIRST && place.slice >= value_slices;  // columns of T
    if (matrix && segment == 0) return;
    const int width = matrix ? a.K : a.V, vw = channel<NC>(place.slice - (matrix ? value_slices : 0), r16);
    const uint32_t v0 = min(vw, width - NC);
    const bool live = vw < width;
    const auto part = [&](int i) { return p.parts + (head * (p.segments - 1) + i) * a.K * (int64_t)(a.V + a.K); };
    const float *from = p.h0 ? p.h0 + head * a.K * a.V : nullptr;
    if (segment > 0) from = FIRST ? nullptr : part(segment - 1);

    f4 state[ST][NC];
#pragma unroll
    for (int j = 0; j < ST; ++j)
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const int k0 = 16 * (ST * wave + j) + 4 * grp;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                {
                state[j][n][i] = from && k0 + i < a.K ? from[(k0 + i) * a.V + v0 + n] : 0.0f;
                if (matrix) state[j][n][i] = k0 + i == (int)v0 + n ? 1.0f : 0.0f;
            }
            s.state.put4(16 * n + r16, k0, state[j][n]);
        }

    typename O::Ex kf[KX], qf[KX], ktf[ST][2];
    typename O::template Sum<PL> inv[2];
    typename O::template Sum<OUT> att[2];
    f4 k_enter, k_leave, q_enter, beta;
    float through;
    Elements<IO, NC> val[4];
    // (no load has a condition: one that has is waited for where its branch ends)
    // a step of the chunk that is there
    const auto step_of = [&](int64_t c, int t) { return (uint32_t)min((int64_t)t, a.L - 1 - c * kC); };
    const auto load_qk = [&](int64_t c) {
        const char *kc = k_base + c * kC * (int64_t)k_step, *qc = q_base + c * kC * (int64_t)q_step;
        const uint32_t t = step_of(c, row);
#pragma unroll
        for (int x = 0; x < KX; ++x) {
            const uint32_t off = (32 * x + 8 * grp < a.K ? 32 * x + 8 * grp : 0) * IO::bytes;
            kf[x] = O::load(&at<E>(kc, t * k_step + off));
            if constexpr (!FIRST) qf[x] = O::load(&at<E>(qc, t * q_step + off));
        }
    };
    const auto load_vec = [&](int64_t c) {
        const char *vec = blocks + c * Block::kBytes;
        k_enter = at<f4>(vec, (kVecKEnter * kC + mine) * 4);
        k_leave = at<f4>(vec, (kVecKLeave * kC + mine) * 4);
        q_enter = at<f4>(vec, (kVecQEnter * kC + mine) * 4);
        beta = at<f4>(vec, (kVecBeta * kC + mine) * 4);
        through = at<float>(vec, kVecThrough * kC * 4);
    };
    const auto load_val = [&](int64_t c) {
        const char *vc = v_base + c * kC * (int64_t)v_step;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            val[i] = Elements<IO, NC>::load(vc, step_of(c, mine + i) * v_step + (matrix ? 0 : v0) * IO::bytes);
    };
    constexpr int TILE = 512 * IO::bytes;
    const uint32_t in_tile = lane * 8 * IO::bytes;
    // (the waves of the upper half have no second block of columns: they load the first twice)
    const int tile0 = 2 * wave * TILE, tile1 = tile0 + wave / 2 * TILE;
    const auto load_inv = [&](int64_t c) {
        const char *m = blocks + c * Block::kBytes + Block::kInv;
        inv[0] = O::template planes<PL>(&at<E>(m + tile0, in_tile), Block::PLANE);
        inv[1] = O::template planes<PL>(&at<E>(m + tile1, in_tile), Block::PLANE);
    };
    const auto load_att = [&](int64_t c) {
        if constexpr (FIRST) return;
        const char *m = blocks + c * Block::kBytes + Block::kAtt;
        att[0] = O::template planes<OUT>(&at<E>(m + tile0, in_tile), Block::PLANE);
        att[1] = O::template planes<OUT>(&at<E>(m + tile1, in_tile), Block::PLANE);
    };
    const auto load_kt = [&](int64_t c) {
        const char *m = blocks + c * Block::kBytes + Block::kKt + 2 * ST * wave * TILE;
#pragma unroll
        for (int j = 0; j < ST; ++j)
#pragma unroll
            for (int y = 0; y < 2; ++y) ktf[j][y] = O::load(&at<E>(m + (2 * j + y) * TILE, in_tile));
    };
    const uint32_t v_row = (uint32_t)a.V * 4;  // a state's row in bytes
    load_qk(begin);
    load_vec(begin);
    load_val(begin);
    load_inv(begin);
    load_kt(begin);
    load_att(begin);
    __syncthreads();
    for (int64_t c = begin; c < end; ++c) {
        const int64_t next = min(c + 1, end - 1);
        const bool whole = (c + 1) * kC <= a.L;
        char *ck = reinterpret_cast<char *>(p.ck) + (c * a.B * a.H + head) * (a.K + kC) * (int64_t)v_row;
        if (!whole || a.K != KP)  // steps past the end and channels past K, which were loaded from elsewhere
#pragma unroll
            for (int x = 0; x < KX; ++x)
                if (c * kC + row >= a.L || 32 * x + 8 * grp >= a.K) kf[x] = qf[x] = typename O::Ex{};
        // K S and Q S
        f4 ks[NC] = {}, o[NC] = {};
#pragma unroll
        for (int x = 0; x < KX; ++x)
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const auto st = s.state.template get<PL>(16 * n + r16, 32 * x + 8 * grp);
                ks[n] = O::mul(ks[n], kf[x], st);
                if constexpr (!FIRST) o[n] = O::mul(o[n], qf[x], O::template first<OUT>(st));
            }
        load_qk(next);
        // X = V - enter K S (a state that does not reach a step has no part in it, whatever it holds; one that
        // holds infinities or NaNs and ends in this chunk shows in its own outputs through Q S, and must not
        // meet, in the products over steps, the zeros that keep it from the steps behind its end)
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            f4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = !matrix && (whole || c * kC + mine + i < a.L) ? val[i].get(n) : 0.0f;
                const bool seen = k_enter[i] != 0.0f && (through != 0.0f || ks[n][i] - ks[n][i] == 0.0f);
                x[i] = seen ? __builtin_fmaf(-k_enter[i], ks[n][i], x[i]) : x[i];
                o[n][i] = q_enter[i] != 0.0f ? q_enter[i] * o[n][i] : 0.0f;
            }
            s.x.put4(16 * n + r16, mine, x);
        }
        load_val(next);
        if (!FIRST && p.ck) store_rows<ST, NC>(ck, v_row, a.K, 16 * ST * wave + 4 * grp, a.K == KP, v0, live, state);
        __syncthreads();
        // (I + B diag(beta)) E = X
        f4 errs[NC];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            f4 err = O::mul(f4{0, 0, 0, 0}, inv[0], s.x.get(16 * n + r16, 8 * grp));
            if (wave >= 2) err = O::mul(err, inv[1], s.x.get(16 * n + r16, 32 + 8 * grp));
            const f4 u = beta * err;
            s.w.put4(16 * n + r16, mine, k_leave * u);
            if constexpr (!FIRST) s.u.put4(16 * n + r16, mine, u);
            errs[n] = err;
        }
        if (!FIRST && p.ck && live)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[NC];
#pragma unroll
                for (int n = 0; n < NC; ++n) x[n] = errs[n][i];
                store_floats<NC>(ck + (a.K + i) * (int64_t)v_row, mine * v_row + v0 * 4, x);
            }
        load_inv(next);
        const float pass = through;
        load_vec(next);
        __syncthreads();
        // S <- through S + (leave K)^T diag(beta) E
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            const auto w0 = s.w.get(16 * n + r16, 8 * grp), w1 = s.w.get(16 * n + r16, 32 + 8 * grp);
#pragma unroll
            for (int j = 0; j < ST; ++j) {
                f4 &st = state[j][n];
#pragma unroll
                for (int i = 0; i < 4; ++i) st[i] = pass != 0.0f ? pass * st[i] : 0.0f;
                st = O::mul(O::mul(st, ktf[j][0], w0), ktf[j][1], w1);
                s.state.put4(16 * n + r16, 16 * (ST * wave + j) + 4 * grp, st);
            }
        }
        load_kt(next);
        // O = scale enter Q S + P diag(beta) E
        if (!FIRST && p.o) {
            char *oc = o_base + (c * kC + 16 * wave) * (int64_t)o_step;
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                o[n] = O::mul(o[n], att[0], s.u.get(16 * n + r16, 8 * grp));
                if (wave >= 2) o[n] = O::mul(o[n], att[1], s.u.get(16 * n + r16, 32 + 8 * grp));
            }
            if (live)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (whole || c * kC + mine + i < a.L) {
                        float x[NC];
#pragma unroll
                        for (int n = 0; n < NC; ++n) x[n] = o[n][i];
                        store_elements<IO, NC>(oc + i * (int64_t)o_step, 4 * grp * o_step + v0 * IO::bytes, x);
                    }
        }
        load_att(next);
        __syncthreads();
    }
    if (matrix) {  // transposed
#pragma unroll
        for (int j = 0; j < ST; ++j)
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const int k0 = 16 * (ST * wave + j) + 4 * grp;
                if (live && k0 < a.K)
                    *reinterpret_cast<f4 *>(part(segment) + a.K * a.V + (v0 + n) * a.K + k0) = state[j][n];
            }
    } else if constexpr (FIRST)
        store_rows<ST, NC>(reinterpret_cast<char *>(part(segment)), v_row, a.K, 16 * ST * wave + 4 * grp, a.K == KP, v0,
                           live, state);
    else if (p.h_final && segment == p.segments - 1)
        store_rows<ST, NC>(reinterpret_cast<char *>(p.h_final) + head * a.K * (int64_t)v_row, v_row, a.K,
                           16 * ST * wave + 4 * grp, a.K == KP, v0, live, state);
}

// The states entering the segments, each put in the place of the Z before it: kJoinV value channels of a head
// a workgroup, for each thread four rows and 16 of the columns of T S, summed over the eight threads of a row
// through LDS.  A segment's T is loaded while the one before it is worked on.  What T does not take up, or S
// does not hold, has no part in T S (T is 0 behind a reset, and S may hold infinities or NaNs): sums that come
// out as NaN are formed again without the terms that have a zero.  (Rows of T behind K repeat others, where S
// is put as 0.)  About 1 us a segment for a few heads: T, 64 KB, comes from memory once a workgroup.
constexpr int kJoinV = 4;

__global__ __launch_bounds__(kThreads, 2) void join_kernel(ChainArgs p) {
    constexpr int KM = SSM_DELTA_MAX_KDIM, COLS = KM / 8;
    static_assert(kThreads == KM / 4 * 8 && kThreads == KM * kJoinV / 2, "threads of a row, outputs of a thread");
    __shared__ f4 s[KM], sums[8][KM];
    const Call &a = p.a;
    const int slices = a.V / kJoinV;  // V is a multiple of 8
    const int64_t head = blockIdx.x / slices, size = a.K * (int64_t)(a.V + a.K);
    const int v0 = (int)(blockIdx.x % slices) * kJoinV;
    float *part = p.parts + head * (p.segments - 1) * size;
    const int quad = threadIdx.x % (KM / 4), eighth = threadIdx.x / (KM / 4);
    const float *column = part + a.K * a.V + min(4 * quad, a.K - 4);
    const int row = threadIdx.x / 2, half = threadIdx.x % 2 * 2, at = min(row, a.K - 1) * a.V + v0 + half;
    f4 t[COLS], m[COLS];
    f2 z;
    const auto load = [&](int g) {
#pragma unroll
        for (int j = 0; j < COLS; ++j)
            t[j] = *reinterpret_cast<const f4 *>(column + g * size + min(COLS * eighth + j, a.K - 1) * a.K);
        z = *reinterpret_cast<const f2 *>(part + g * size + at);
    };
    const auto put = [&](f2 x) {
        if (row >= a.K) x = f2{0, 0};
        float *to = reinterpret_cast<float *>(&s[row]) + half;
        to[0] = x[0];
        to[1] = x[1];
    };
    put(*reinterpret_cast<const f2 *>(part + at));
    load(1);
    __syncthreads();
    for (int g = 1; g < p.segments - 1; ++g) {
#pragma unroll
        for (int j = 0; j < COLS; ++j) m[j] = t[j];
        f2 out = z;
        load(min(g + 1, p.segments - 2));
        f4 sum[4];  // a row's channels each
        const auto add_up = [&](auto with_zeros) {
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[r] = f4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < COLS; ++j) {
                const f4 x = s[COLS * eighth + j];
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int n = 0; n < kJoinV; ++n)
                        if (with_zeros.value || (m[j][r] != 0.0f && x[n] != 0.0f))
                            sum[r][n] = __builtin_fmaf(m[j][r], x[n], sum[r][n]);
            }
        };
        add_up(std::true_type{});
        f4 all = sum[0] + sum[1] + sum[2] + sum[3];
        if (!(all[0] + all[1] + all[2] + all[3] < __builtin_inff())) add_up(std::false_type{});
#pragma unroll
        for (int r = 0; r < 4; ++r) sums[eighth][4 * quad + r] = sum[r];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) out += *reinterpret_cast<const f2 *>(reinterpret_cast<const float *>(&sums[e][row]) + half);
        put(out);
        if (row < a.K) *reinterpret_cast<f2 *>(part + g * size + at) = out;
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------ step
// One token: a workgroup of four waves owns one head's columns v0 .. v0 + 31, eight threads side by side
// (4 columns each) times 32 rows apart.  The state is read once, held in registers (KP / 32 rows a thread),
// and written once; S^T k and S^T q go through the same two reductions, o = scale (S'^T q + (q.k) u).  Bound by
// HBM: 256 sequences of 40 heads of 128 x 128 in 268 us, 5.0 TB/s.
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
hipError_t prepare(const Call &a, bool backward, char *workspace, hipStream_t stream) {
    const dim3 grid((unsigned)a.n, (unsigned)a.H, (unsigned)a.B);
    uint32_t *marks = reinterpret_cast<uint32_t *>(workspace);
    char *blocks = workspace + marks_bytes(a.B * a.H * a.n);
    if (backward)
        prepare_kernel<IO, KP, true><<<grid, kThreads, 0, stream>>>(a, blocks, marks);
    else
        prepare_kernel<IO, KP, false><<<grid, kThreads, 0, stream>>>(a, blocks, marks);
    return hipGetLastError();
}

template <typename IO, int KP, int NC, bool FIRST>
hipError_t chain_pass(ChainArgs p, hipStream_t stream) {
    p.slices = (p.a.V + 16 * NC - 1) / (16 * NC) + (FIRST ? (p.a.K + 16 * NC - 1) / (16 * NC) : 0);
    const unsigned grid = chain_grid(p.a.B * p.a.H * (p.segments - FIRST), p.slices);
    chain_kernel<IO, KP, NC, FIRST><<<grid, kThreads, sizeof(ChainLds<IO, KP, NC>), stream>>>(p);
    return hipGetLastError();
}

template <typename IO, int KP>
hipError_t chain(const ChainArgs &p, hipStream_t stream) {
    if (p.segments > 1) {
        hipError_t e = p.wide ? chain_pass<IO, KP, 2, true>(p, stream) : chain_pass<IO, KP, 1, true>(p, stream);
        if (e != hipSuccess) return e;
        if (p.segments > 2)
            join_kernel<<<(unsigned)(p.a.B * p.a.H * (p.a.V / kJoinV)), kThreads, 0, stream>>>(p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        return p.wide ? chain_pass<IO, KP, 2, false>(p, stream) : chain_pass<IO, KP, 1, false>(p, stream);
    }
    // 32 channels a workgroup where every CU gets one all the same (8 x 2048 x 12 heads: 175 us, 215 with 16;
    // where checkpoints are written as well 257 and 314)
    return wide_slices(p.a) ? chain_pass<IO, KP, 2, false>(p, stream) : chain_pass<IO, KP, 1, false>(p, stream);
}

template <typename IO, int KP>
hipError_t step(const StepArgs &p, hipStream_t stream) {
    const dim3 grid(((unsigned)p.a.V + kStepV - 1) / kStepV, (unsigned)p.a.H, (unsigned)p.a.B);
    step_kernel<IO, KP><<<grid, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

size_t block_bytes(int io_dtype, int64_t kdim, bool backward) {
    const auto of = [&](auto io) {
        using IO = decltype(io);
        if (kdim <= 64) return backward ? ChunkBlock<IO, 64, true>::kBytes : ChunkBlock<IO, 64, false>::kBytes;
        return backward ? ChunkBlock<IO, 128, true>::kBytes : ChunkBlock<IO, 128, false>::kBytes;
    };
    return io_dtype == SSM_BF16 ? of(io_bf16{}) : of(io_f32{});
}

hipError_t launch_prepare(const Call &a, int io_dtype, bool backward, char *workspace, hipStream_t stream) {
    if (io_dtype == SSM_BF16)
        return a.K <= 64 ? prepare<io_bf16, 64>(a, backward, workspace, stream)
                         : prepare<io_bf16, 128>(a, backward, workspace, stream);
    return a.K <= 64 ? prepare<io_f32, 64>(a, backward, workspace, stream)
                     : prepare<io_f32, 128>(a, backward, workspace, stream);
}

struct Segments {
    int count;
    bool wide;
};

// Segments of a sequence of n chunks: as many as run at once with outputs, two workgroups a CU, of at least eight
// chunks, as each costs a step of join_kernel and its state once more.  The pass without outputs has up to three
// workgroups a CU of 16 channels, which run at once, or six of 32, of which two do (held to two, 32768 steps of 12
// heads take 886 us and not 789, 16384 of 20 heads 715 and 643, 8192 of 12 238 and 225, 4096 of 12 139 and 142).
// Where there would be fewer than eight segments, workgroups take 32 channels, which leaves room for more.
// bf16, K = V = 128, whole calls, us, as they run and in one piece (in slices of 16 alone):
//   32768 steps of one head 160 (32 segments) and 1035, of 4 heads 334 (13) and 1167, of 12 heads 787 (10 of 32
//   channels) and 1410 (988); 16384 steps of 8 heads 268 and 614 (309), of 20 heads 644 and 794 (852); 4096 steps
//   of 4 heads 79 and 161, of 12 heads 143 and 172 (137), of 16 heads 163 and 179 (161); 2048 of 12 heads 99 and 96.
// Not taken: 1024 steps of 12 heads in three segments 73, in two 59, in one piece 60; 4096 steps of 24 heads in five
// 226, in one piece 191.
static Segments segments_of(int64_t heads, int64_t n, int64_t K, int64_t V) {
    const auto long_enough = [&](int64_t s) { return s <= n / 8 && s * s <= 2 * n; };
    const auto fits = [&](int64_t s, int width) {
        const int64_t values = heads * ((V + width - 1) / width), matrices = heads * ((K + width - 1) / width);
        return long_enough(s) && values * s <= 512 && values * (s - 1) + matrices * (s - 2) <= 48 * width;
    };
    if (n < 32 || !fits(3, 16)) return {1, false};
    int64_t s = 3;
    while (fits(s + 1, 16)) ++s;
    const bool wide = s < 8 && long_enough(s + 1);
    if (wide)
        while (fits(s + 1, 32)) ++s;
    const int64_t per = (n + s - 1) / s;
    return {(int)((n + per - 1) / per), wide};
}

size_t chain_bytes(int io_dtype, int64_t heads, int64_t n, int64_t K, int64_t V) {
    return marks_bytes(heads * n) + up256((size_t)(heads * n) * block_bytes(io_dtype, K, false)) +
           up256((size_t)(heads * (segments_of(heads, n, K, V).count - 1) * K * (V + K)) * sizeof(float));
}

hipError_t launch_chain(const Call &a, int io_dtype, char *workspace, const float *h0, void *o, float *h_final, float *ck,
                        hipStream_t stream) {
    const int64_t heads = a.B * a.H;
    const Segments split = segments_of(heads, a.n, a.K, a.V);
    const char *blocks = workspace + marks_bytes(heads * a.n);
    float *parts = reinterpret_cast<float *>(workspace + marks_bytes(heads * a.n) +
                                             up256((size_t)(heads * a.n) * block_bytes(io_dtype, a.K, false)));
    const ChainArgs p{a, blocks, h0, o, h_final, ck, parts, (a.n + split.count - 1) / split.count, split.count, split.wide, 0};
    hipError_t e;
    if (io_dtype == SSM_BF16)
        e = a.K <= 64 ? chain<io_bf16, 64>(p, stream) : chain<io_bf16, 128>(p, stream);
    else
        e = a.K <= 64 ? chain<io_f32, 64>(p, stream) : chain<io_f32, 128>(p, stream);
    if (e != hipSuccess) return e;
    return launch_grow(a, io_dtype, reinterpret_cast<const uint32_t *>(workspace), h0, o, h_final, ck, stream);
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
    return delta::chain_bytes(a.io_dtype, a.batch * a.heads, n, a.kdim, a.vdim);
}

hipError_t launch_gated_delta_fwd(const ssm_gated_delta_args_t &a, hipStream_t stream) {
    const delta::Call c = call_of(a);
    char *workspace = static_cast<char *>(a.workspace);
    const hipError_t e = delta::launch_prepare(c, a.io_dtype, false, workspace, stream);
    if (e != hipSuccess) return e;
    return delta::launch_chain(c, a.io_dtype, workspace, a.h0, a.o, a.h_final, a.checkpoints, stream);
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
