// gated_delta_grow.hip -- heads of the gated delta rule whose decays grow (ssm_gated_delta_fwd, _bwd) on
// gfx950, one step after another.  A chunk's own equations (gated_delta.hip) subtract numbers as large as the
// largest product of its decays, e^{G_t - G_s}, from one another; where keys write a state over again and again
// it stays far smaller, and what is left of the difference is rounding: 64 steps of g = 0.1 with one key are
// off by 1e-4 of the largest output, of g = 0.3 by 15 times that output.  prepare_kernel marks the chunks in
// which such a product exceeds e^kGrowth = e (so that a chunk's rounding errors grow by no more), and these
// kernels, which run behind the others, do the whole of a head with such a chunk again by the definition:
//   S' = e^g S,  e = v - S'^T k,  S = S' + beta k e^T,  o = scale S^T q
// Backwards, from the last step (dS: the gradient of S behind it):
//   dq = scale S do,  dS += scale q do^T,  du = dS^T k,  dbeta = e.du,  dv = beta du,
//   dk = beta dS e - S' dv,  dS -= k dv^T,  dg = <dS, S'>,  dS <- e^g dS
// Heads without growth, the usual ones, cost the look at their marks: 2 to 5 us a call.
#include "delta_tile.h"
#include "wide_io.h"

namespace ssm {
namespace delta {
namespace {

// A wave holds four channels of a state in registers: 16 lanes a channel, eight rows a lane.
constexpr int kRows = 8, kWaves = kThreads / 64, kGroup = 4 * kWaves;  // channels of a workgroup
static_assert(16 * kRows == SSM_DELTA_MAX_KDIM, "rows of 16 lanes");

struct Place {
    int wave, lane, row, v;  // the lane's first row and its channel
    int rows;                // how many of its rows there are: all or none
    bool live;
    __device__ Place(const Call &a, int v0) {
        lane = threadIdx.x % 64;
        wave = threadIdx.x / 64;
        row = lane % 16 * kRows;
        rows = row < a.K ? kRows : 0;
        v = v0 + 4 * wave + lane / 16;
        live = v < a.V;
    }
    __device__ __forceinline__ bool first() const { return lane % 16 == 0; }  // of a channel's lanes
};

// One step of a head: its key and query (normed), gates and reset.
template <typename IO>
struct Step {
    float q[kRows], k[kRows], decay, beta;
    bool cut;
    __device__ __forceinline__ static void unit(const Call &a, const void *base, int64_t at, int rows, float (&x)[kRows]) {
        const Raw<IO, kRows> raw = load_raw<IO, kRows>(base, at, rows);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            x[i] = raw[i];
            s = __builtin_fmaf(x[i], x[i], s);
        }
        if (!a.l2norm) return;
        const float r = 1.0f / sqrtf(sum16(s) + kL2Eps);
#pragma unroll
        for (int i = 0; i < kRows; ++i) x[i] *= r;
    }
    __device__ __forceinline__ Step(const Call &a, const Place &p, int64_t b, int h, int hk, int64_t t, bool query) {
        unit(a, a.k, b * a.k_batch + t * a.k_token + (int64_t)hk * a.K + p.row, p.rows, k);
        if (query) unit(a, a.q, b * a.q_batch + t * a.q_token + (int64_t)hk * a.K + p.row, p.rows, q);
        const int64_t at = (b * a.L + t) * a.H + h;
        const float g = a.g[at];
        cut = (a.reset && a.reset[b * a.L + t]) || g < kForget;
        decay = expf(g);
        beta = load_io<IO>(a.beta, at);
    }
};

__device__ __forceinline__ float dot(const float (&x)[kRows], const float (&y)[kRows]) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) s = __builtin_fmaf(x[i], y[i], s);
    return sum16(s);
}
__device__ __forceinline__ float sum4(float x) {  // over the four channels of a wave
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}
template <typename IO>
__device__ __forceinline__ void forget(const Step<IO> &s, float (&S)[kRows]) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) S[i] = s.cut ? 0.0f : s.decay * S[i];
}
__device__ __forceinline__ void add(const float (&x)[kRows], float y, float (&S)[kRows]) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) S[i] = __builtin_fmaf(x[i], y, S[i]);
}

// Whether one of `n` marks is set.
__device__ __forceinline__ bool marked(const uint32_t *marks, int64_t n) {
    bool any = false;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) any |= marks[i] != 0;
    return __syncthreads_or(any);
}

struct GrowArgs {
    Call a;
    const uint32_t *marks;
    const float *h0;
    void *o;
    float *h_final, *ck;
};

// A head's 16 channels a workgroup; waves have channels of their own and never wait for one another.  Bound by
// the latency of a step's loads and sums, 1.1 us a step: 2048 steps of one head of 128 x 128, bf16, 2.3 ms, of 8
// rows of 12 heads 4.6 ms.
template <typename IO>
__global__ __launch_bounds__(kThreads) void grow_kernel(GrowArgs p) {
    const Call &a = p.a;
    const int h = blockIdx.y, hk = h / (a.H / a.Hk);
    const int64_t b = blockIdx.z, head = b * a.H + h;
    if (!marked(p.marks + head * a.n, a.n)) return;
    const Place at(a, blockIdx.x * kGroup);
    const int64_t column = (head * a.K + at.row) * a.V + at.v;
    float S[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) S[i] = p.h0 && at.live && at.rows ? p.h0[column + i * a.V] : 0.0f;
    for (int64_t t = 0; t < a.L; ++t) {
        float *ck = p.ck + ((t / kC * a.B * a.H + head) * (a.K + kC)) * a.V + at.v;
        if (p.ck && t % kC == 0 && at.live && at.rows)
#pragma unroll
            for (int i = 0; i < kRows; ++i) ck[(at.row + i) * a.V] = S[i];
        const Step<IO> s(a, at, b, h, hk, t, true);
        const float v = at.live ? load_io<IO>(a.v, b * a.v_batch + t * a.v_token + (int64_t)h * a.V + at.v) : 0.0f;
        forget(s, S);
        const float e = v - dot(s.k, S);
        add(s.k, s.beta * e, S);
        const float o = a.scale * dot(s.q, S);
        if (!at.live || !at.first()) continue;
        if (p.ck) ck[(a.K + t % kC) * a.V] = e;
        if (p.o) store_io<IO>(p.o, ((b * a.L + t) * a.H + h) * a.V + at.v, o);
    }
    if (p.ck && at.live && at.first())  // no errors behind the last step
        for (int64_t t = a.L; t < a.n * kC; ++t)
            p.ck[(((a.n - 1) * a.B * a.H + head) * (a.K + kC) + a.K + t % kC) * a.V + at.v] = 0.0f;
    if (p.h_final && at.live && at.rows)
#pragma unroll
        for (int i = 0; i < kRows; ++i) p.h_final[column + i * a.V] = S[i];
}

struct GrowBackArgs {
    Call a;
    const uint32_t *marks;
    const float *ck, *dh_final;
    const void *dout;
    void *dq, *dk, *dv, *dbeta;
    float *dg, *dh0;
    // sums over channels and heads: of dq and dk (64 x K each) at the start of the chunk's block of the key
    // head's first head, of dbeta (64) in the (head, chunk)'s first sums of E.dU; both have been read by now
    char *blocks;
    int64_t block_bytes;
    float *dbeta_sum;
};

constexpr int kSub = 8;  // steps of a stretch: a chunk's states are formed again from every eighth

struct GrowBackLds {
    float every[kWaves][kC / kSub][kRows][64], within[kWaves][kSub][kRows][64];
    float part[2][kWaves][2 * SSM_DELTA_MAX_KDIM + 2];  // a step's dq, dk, dbeta, dg of each wave's channels
};

// All heads of a key head, 16 channels at a time, from the last chunk to the first.  A chunk's states come from
// its checkpoint and errors: forwards through the chunk, keeping every eighth, and again through eight steps
// ahead of going back through them.  A step's sums over the channels go round through LDS in a fixed order; a
// barrier a step (the next step's sums have places of their own).  Latency again, 3.9 us for a step and 16
// channels: 2048 steps of one head of 128 x 128, bf16, 63 ms, of 8 rows of 12 heads 79 ms.
template <typename IO>
__global__ __launch_bounds__(kThreads) void grow_back_kernel(GrowBackArgs p) {
    extern __shared__ __attribute__((aligned(16))) char raw[];
    GrowBackLds &s = *reinterpret_cast<GrowBackLds *>(raw);
    const Call &a = p.a;
    const int hk = blockIdx.x, share = a.H / a.Hk;
    const int64_t b = blockIdx.y, head0 = b * a.H + (int64_t)hk * share;
    if (!marked(p.marks + head0 * a.n, share * a.n)) return;
    const auto sums = [&](int64_t c) { return reinterpret_cast<float *>(p.blocks + (head0 * a.n + c) * p.block_bytes); };
    int turn = 0;
    for (int h = hk * share; h < (hk + 1) * share; ++h) {
        const int64_t head = b * a.H + h;
        for (int v0 = 0; v0 < a.V; v0 += kGroup) {
            const Place at(a, v0);
            const bool fresh = h == hk * share && v0 == 0;  // the sums' first terms
            const int64_t column = (head * a.K + at.row) * a.V + at.v;
            const bool there = at.live && at.rows;
            float dS[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) dS[i] = p.dh_final && there ? p.dh_final[column + i * a.V] : 0.0f;
            for (int64_t c = a.n - 1; c >= 0; --c) {
                const float *ck = p.ck + ((c * a.B * a.H + head) * (a.K + kC)) * a.V + at.v;
                const int steps = (int)min((int64_t)kC, a.L - c * kC);
                float S[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) S[i] = there ? ck[(at.row + i) * a.V] : 0.0f;
                const auto error = [&](int t) { return at.live ? ck[(a.K + t) * a.V] : 0.0f; };
                const auto advance = [&](int t, int keep) {
                    const Step<IO> x(a, at, b, h, hk, c * kC + t, false);
                    forget(x, S);
                    if (keep >= 0)
#pragma unroll
                        for (int i = 0; i < kRows; ++i) s.within[at.wave][keep][i][at.lane] = S[i];
                    add(x.k, x.beta * error(t), S);
                };
                for (int t = 0; t < steps; ++t) {
                    if (t % kSub == 0)
#pragma unroll
                        for (int i = 0; i < kRows; ++i) s.every[at.wave][t / kSub][i][at.lane] = S[i];
                    advance(t, -1);
                }
                for (int t = steps - 1; t >= 0; --t) {
                    if (t == steps - 1 || t % kSub == kSub - 1) {
                        const int from = t / kSub * kSub;
#pragma unroll
                        for (int i = 0; i < kRows; ++i) S[i] = s.every[at.wave][t / kSub][i][at.lane];
                        for (int u = from; u <= t; ++u) advance(u, u - from);
                    }
                    const int64_t step = c * kC + t;
                    const Step<IO> x(a, at, b, h, hk, step, true);
                    const float e = error(t);
                    const int64_t o_at = ((b * a.L + step) * a.H + h) * a.V + at.v;
                    const float d = at.live ? a.scale * load_io<IO>(p.dout, o_at) : 0.0f;
                    float old[kRows], dq[kRows], dk[kRows];
#pragma unroll
                    for (int i = 0; i < kRows; ++i) old[i] = S[i] = s.within[at.wave][t % kSub][i][at.lane];
                    add(x.k, x.beta * e, S);
                    add(x.q, d, dS);
                    const float du = dot(x.k, dS), dv = x.beta * du;
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        dq[i] = sum4(S[i] * d);
                        dk[i] = sum4(__builtin_fmaf(x.beta * e, dS[i], -old[i] * dv));
                    }
                    add(x.k, -dv, dS);
                    const float dbeta = sum4(e * du), dg = sum4(dot(dS, old));
                    forget(x, dS);
                    if (at.live && at.first()) store_io<IO>(p.dv, o_at, dv);
                    float(&part)[kWaves][2 * SSM_DELTA_MAX_KDIM + 2] = s.part[turn];
                    turn ^= 1;
                    if (at.lane < 16) {
#pragma unroll
                        for (int i = 0; i < kRows; ++i) {
                            part[at.wave][at.row + i] = dq[i];
                            part[at.wave][SSM_DELTA_MAX_KDIM + at.row + i] = dk[i];
                        }
                        if (at.lane == 0) {
                            part[at.wave][2 * SSM_DELTA_MAX_KDIM] = dbeta;
                            part[at.wave][2 * SSM_DELTA_MAX_KDIM + 1] = x.cut ? 0.0f : dg;
                        }
                    }
                    __syncthreads();
                    const auto total = [&](int i) { return (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]); };
                    const auto put = [](float &to, bool set, float x) { to = set ? x : to + x; };
                    const int i = threadIdx.x, k = i % SSM_DELTA_MAX_KDIM;
                    if (k < a.K) put(sums(c)[(i / SSM_DELTA_MAX_KDIM * kC + t) * a.K + k], fresh, total(i));
                    if (i == 0) put(p.dbeta_sum[(head * a.n + c) * kC + t], v0 == 0, total(2 * SSM_DELTA_MAX_KDIM));
                    if (i == 1) put(p.dg[(b * a.L + step) * a.H + h], v0 == 0, total(2 * SSM_DELTA_MAX_KDIM + 1));
                }
            }
            if (p.dh0 && there)
#pragma unroll
                for (int i = 0; i < kRows; ++i) p.dh0[column + i * a.V] = dS[i];
        }
        __syncthreads();
        for (int64_t t = threadIdx.x; t < a.L; t += kThreads)
            store_io<IO>(p.dbeta, (b * a.L + t) * a.H + h, p.dbeta_sum[head * a.n * kC + t]);
    }
    // through the norms, a step a wave: dx = r (dxhat - xhat (xhat . dxhat))
    const Place at(a, 0);
    for (int64_t t = at.wave; t < a.L; t += kWaves)
        for (int which = 0; which < 2; ++which) {
            const int64_t from = which ? b * a.k_batch + t * a.k_token : b * a.q_batch + t * a.q_token;
            const float *sum = sums(t / kC) + (which * kC + t % kC) * a.K + at.row;
            float x[kRows], d[kRows], squares = 0.0f;
            const Raw<IO, kRows> x0 = load_raw<IO, kRows>(which ? a.k : a.q, from + (int64_t)hk * a.K + at.row, at.rows);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                x[i] = x0[i];
                squares = __builtin_fmaf(x[i], x[i], squares);
                d[i] = at.rows ? sum[i] : 0.0f;
            }
            if (a.l2norm) {
                const float r = 1.0f / sqrtf(sum16(squares) + kL2Eps);
#pragma unroll
                for (int i = 0; i < kRows; ++i) x[i] *= r;
                const float along = dot(x, d);
#pragma unroll
                for (int i = 0; i < kRows; ++i) d[i] = r * (d[i] - x[i] * along);
            }
            if (at.lane < 16 && at.rows)
                store_raw<IO>(which ? p.dk : p.dq, ((b * a.L + t) * a.Hk + hk) * a.K + at.row, kRows, d);
        }
}

}  // namespace

hipError_t launch_grow(const Call &a, int io_dtype, const uint32_t *marks, const float *h0, void *o, float *h_final,
                       float *ck, hipStream_t stream) {
    const GrowArgs p{a, marks, h0, o, h_final, ck};
    const dim3 grid((unsigned)((a.V + kGroup - 1) / kGroup), (unsigned)a.H, (unsigned)a.B);
    if (io_dtype == SSM_BF16)
        grow_kernel<io_bf16><<<grid, kThreads, 0, stream>>>(p);
    else
        grow_kernel<io_f32><<<grid, kThreads, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_grow_back(const Call &c, const ssm_gated_delta_bwd_args_t &a, const uint32_t *marks, const float *ck,
                            char *blocks, float *dbeta_sum, hipStream_t stream) {
    const GrowBackArgs p{c, marks, ck, a.dh_final, a.dout, a.dq, a.dk, a.dv, a.dbeta, a.dg, a.dh0, blocks,
                         (int64_t)block_bytes(a.io_dtype, a.kdim, true), dbeta_sum};
    const dim3 grid((unsigned)c.Hk, (unsigned)c.B);
    if (a.io_dtype == SSM_BF16)
        grow_back_kernel<io_bf16><<<grid, kThreads, sizeof(GrowBackLds), stream>>>(p);
    else
        grow_back_kernel<io_f32><<<grid, kThreads, sizeof(GrowBackLds), stream>>>(p);
    return hipGetLastError();
}

}  // namespace delta
}  // namespace ssm
