// delta_tile.h -- operands, tiles and per-chunk gates of the gated delta rule's kernels (gfx950).
//
// A chunk is 64 steps.  All products run on 16 x 16 result tiles of the matrix cores, contracted 32 at
// a time: lane l holds row (A) or column (B) l % 16 and the eight consecutive contraction indices
// 8 (l / 16) .. + 7; the result has column l % 16 and, in register i, row 4 (l / 16) + i.  Where a result
// is the right operand of the next product its tiles come in pairs whose rows are dealt out so that
// the two results of a lane ARE the eight values the next product wants of it (pair_row): states, value
// errors and gradients go from one product to the next without leaving their registers.
//
// Precision.  q, k, v, do in bf16 are exact operands.  What was computed in fp32 enters a bf16 product as
// the sum of three bf16 numbers (8 significant bits each, 24 in all: the value itself to 2^-24), an exact
// operand times such a sum as three products and two sums as the six of the nine that reach 2^-24.
// Where a result only feeds a bf16 output, two numbers (16 bits) and three products do.  fp32 inputs run
// the same kernels on the fp32 matrix instructions.
#pragma once

#include "ssm_device.h"
#include "ssm_internal.h"

namespace ssm {
namespace delta {

constexpr int kC = 64;          // steps of a chunk (SSM_DELTA_CHUNK)
constexpr int kThreads = 256;
constexpr float kForget = -104.0f;  // e^g is 0 in fp32 from here on: such a step is a reset
constexpr float kL2Eps = 1e-6f;

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// Row of a result's register i in tile `tile` of a run of pairs, for lane group `grp` (lane / 16).
__device__ __forceinline__ constexpr int pair_row(int tile, int grp, int i) {
    return 32 * (tile / 2) + 8 * grp + 4 * (tile & 1) + i;
}
// The same for row r = 0..15 of that tile (rows of the left operand).
__device__ __forceinline__ constexpr int pair_row16(int tile, int r) { return pair_row(tile, r / 4, r % 4); }

// The operands of one contraction over 32, for fp32 and bf16 tensors.
template <typename IO>
struct Op;

template <>
struct Op<io_f32> {
    using elem = float;
    static constexpr int kPlanes = 1;  // fp32 numbers are kept as they are
    struct Ex {
        float v[8];
    };
    template <int P>
    using Sum = Ex;
    static __device__ __forceinline__ Ex load(const float *p) {
        const f4 a = *reinterpret_cast<const f4 *>(p), b = *reinterpret_cast<const f4 *>(p + 4);
        return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    }
    // eight elements `stride` apart
    static __device__ __forceinline__ Ex gather(const float *p, int stride) {
        Ex r;
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = p[i * stride];
        return r;
    }
    template <int P>
    static __device__ __forceinline__ Ex planes(const float *p, int) {
        return load(p);
    }
    template <int P>
    static __device__ __forceinline__ Ex sum(f4 a, f4 b) {
        return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    }
    static __device__ __forceinline__ Ex exact(f4 a, f4 b) { return sum<1>(a, b); }
    static __device__ __forceinline__ f4 mul(f4 c, const Ex &a, const Ex &b) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
        return c;
    }
};

template <>
struct Op<io_bf16> {
    using elem = __bf16;
    static constexpr int kPlanes = 3;
    struct Ex {
        b8 v;
    };
    template <int P>
    struct Sum {
        b8 p[P];  // largest first
    };
    static __device__ __forceinline__ Ex load(const __bf16 *p) { return {*reinterpret_cast<const b8 *>(p)}; }
    // `P` planes of a matrix, `stride` elements apart
    template <int P>
    static __device__ __forceinline__ Sum<P> planes(const __bf16 *p, int stride) {
        Sum<P> r;
#pragma unroll
        for (int i = 0; i < P; ++i) r.p[i] = *reinterpret_cast<const b8 *>(p + i * stride);
        return r;
    }
    static __device__ __forceinline__ b8 narrow(const float (&x)[8]) {
        b8 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const b2 t = __builtin_convertvector((f2){x[2 * i], x[2 * i + 1]}, b2);
            r[2 * i] = t[0];
            r[2 * i + 1] = t[1];
        }
        return r;
    }
    template <int P>
    static __device__ __forceinline__ Sum<P> sum(f4 a, f4 b) {
        float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        Sum<P> r;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            r.p[p] = narrow(x);
            if (p + 1 < P)
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] -= (float)r.p[p][i];
        }
        return r;
    }
    // values that are bf16 numbers
    static __device__ __forceinline__ Ex exact(f4 a, f4 b) {
        const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        return {narrow(x)};
    }
    static __device__ __forceinline__ f4 one(f4 c, b8 a, b8 b) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f4 mul(f4 c, const Ex &a, const Ex &b) { return one(c, a.v, b.v); }
    template <int P>
    static __device__ __forceinline__ f4 mul(f4 c, const Ex &a, const Sum<P> &b) {
#pragma unroll
        for (int p = P - 1; p >= 0; --p) c = one(c, a.v, b.p[p]);
        return c;
    }
    template <int P>
    static __device__ __forceinline__ f4 mul(f4 c, const Sum<P> &a, const Ex &b) {
#pragma unroll
        for (int p = P - 1; p >= 0; --p) c = one(c, a.p[p], b.v);
        return c;
    }
    // smallest terms first; those below the last plane's weight are left out
    template <int P>
    static __device__ __forceinline__ f4 mul(f4 c, const Sum<P> &a, const Sum<P> &b) {
#pragma unroll
        for (int s = P - 1; s >= 0; --s)
#pragma unroll
            for (int i = s; i >= 0; --i) c = one(c, a.p[i], b.p[s - i]);
        return c;
    }
};

template <typename IO>
__device__ __forceinline__ float widen(typename Op<IO>::elem v) {
    return (float)v;
}

// One call's tensors as its kernels see them.  Strides in elements; a head's K (or V) channels are
// consecutive, its heads too.
struct Call {
    const void *q, *k, *v, *beta;
    const float *g;
    const uint8_t *reset;
    int64_t q_batch, q_token, k_batch, k_token, v_batch, v_token;
    int64_t B, L, n;  // n: chunks of a row
    int Hk, H, K, V;
    float scale;
    int l2norm;
};

// What a chunk's kernels need of its gates; rows past the end have beta 0 and decay 1.
struct Gates {
    double G[kC];   // running sum of the log decays
    int doc[kC];    // resets up to and with each step
    float beta[kC], enter[kC], leave[kC];
    float rq[kC], rk[kC];
    float through;
};

// Wave 0 fills G, doc, beta, enter, leave and through.  A barrier has to follow.
template <typename IO>
__device__ __forceinline__ void load_gates(const Call &a, int64_t b, int h, int64_t t0, Gates &s) {
    if (threadIdx.x >= 64) return;
    const int t = threadIdx.x;
    const bool in = t0 + t < a.L;
    const int64_t at = (b * a.L + t0 + t) * a.H + h;
    float g = in ? a.g[at] : 0.0f;
    const bool cut = in && ((a.reset && a.reset[b * a.L + t0 + t]) || g < kForget);
    double G = cut ? 0.0 : (double)g;
    int doc = cut;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const double up = __shfl_up(G, d, 64);
        const int ud = __shfl_up(doc, d, 64);
        if (t >= d) {
            G += up;
            doc += ud;
        }
    }
    const double end = __shfl(G, 63, 64);
    const int last = __shfl(doc, 63, 64);
    s.G[t] = G;
    s.doc[t] = doc;
    s.beta[t] = in ? load_io<IO>(a.beta, at) : 0.0f;
    s.enter[t] = doc == 0 ? expf((float)G) : 0.0f;
    s.leave[t] = doc == last ? expf((float)(end - G)) : 0.0f;
    if (t == 0) s.through = last == 0 ? expf((float)end) : 0.0f;
}

// D_ts = product of the decays behind step s up to t, 0 where t does not see s (s <= t).
__device__ __forceinline__ float decay(const Gates &s, int t, int u) {
    return u <= t && s.doc[t] == s.doc[u] ? expf((float)(s.G[t] - s.G[u])) : 0.0f;
}

// 64 rows of K channels (rows from t0 on of one head) between memory, registers and LDS, 16 bytes a
// piece: lane = row, so that a transposed copy is written without conflicts.  Loads have no condition (a
// conditional one is waited for where its branch ends, and the next chunk's are to stay in flight).
template <typename IO, int KP>
struct HeadRows {
    using E = typename Op<IO>::elem;
    static constexpr int PER = 16 / IO::bytes;           // elements of a piece
    static constexpr int STRIDE = KP + PER;               // LDS row, in elements
    static constexpr int TSTRIDE = kC + PER;              // row of the transposed copy
    template <int WAVES>
    struct Regs {
        u4 r[KP / PER / WAVES];
    };
    template <int WAVES>
    static __device__ __forceinline__ void load(Regs<WAVES> &r, const void *base, int64_t off, int64_t token, int64_t t0,
                                                int64_t L, int K) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        const int64_t t = t0 + lane < L ? t0 + lane : L - 1;
        const char *row = static_cast<const char *>(base) + (off + t * token) * IO::bytes;
#pragma unroll
        for (int i = 0; i < KP / PER / WAVES; ++i) {
            const int c = (wave * (KP / PER / WAVES) + i) * PER;
            r.r[i] = *reinterpret_cast<const u4 *>(row + (c < K ? c : 0) * IO::bytes);
        }
    }
    // The steps past the end and the channels past K, which were loaded from elsewhere, as 0.
    template <int WAVES>
    static __device__ __forceinline__ void cut(Regs<WAVES> &r, int64_t t0, int64_t L, int K) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        if (t0 + kC <= L && K == KP) return;
#pragma unroll
        for (int i = 0; i < KP / PER / WAVES; ++i) {
            const int c = (wave * (KP / PER / WAVES) + i) * PER;
            if (t0 + lane >= L || c >= K) r.r[i] = u4{0, 0, 0, 0};
        }
    }
    template <int WAVES>
    static __device__ __forceinline__ void store(const Regs<WAVES> &r, E *lds) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < KP / PER / WAVES; ++i) {
            const int c = (wave * (KP / PER / WAVES) + i) * PER;
            *reinterpret_cast<u4 *>(lds + lane * STRIDE + c) = r.r[i];
        }
    }
    template <int WAVES>
    static __device__ __forceinline__ void store_transposed(const Regs<WAVES> &r, E *lds) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < KP / PER / WAVES; ++i) {
            const int c = (wave * (KP / PER / WAVES) + i) * PER;
            E e[PER];
            __builtin_memcpy(e, &r.r[i], 16);
#pragma unroll
            for (int j = 0; j < PER; ++j) lds[(c + j) * TSTRIDE + lane] = e[j];
        }
    }
};

// A 64 x 64 matrix of a chunk in the workspace: fp32, or bf16 planes.
template <typename IO, int P>
struct ChunkMatrix {
    using E = typename Op<IO>::elem;
    static constexpr int PLANES = IO::bytes == 2 ? P : 1;
    static constexpr int PER = 16 / IO::bytes;
    static constexpr int STRIDE = kC + PER, PLANE = kC * STRIDE;  // in LDS
    static constexpr int ELEMS = PLANES * kC * kC;                // in the workspace
    static constexpr int PIECES = ELEMS / PER;
    template <int THREADS>
    struct Regs {
        u4 r[PIECES / THREADS];
    };
    template <int THREADS>
    static __device__ __forceinline__ void load(Regs<THREADS> &r, const E *from) {
#pragma unroll
        for (int i = 0; i < PIECES / THREADS; ++i)
            r.r[i] = reinterpret_cast<const u4 *>(from)[threadIdx.x + THREADS * i];
    }
    template <int THREADS>
    static __device__ __forceinline__ void store(const Regs<THREADS> &r, E *lds) {
#pragma unroll
        for (int i = 0; i < PIECES / THREADS; ++i) {
            const int at = threadIdx.x + THREADS * i, row = at / (kC / PER), c = at % (kC / PER);
            *reinterpret_cast<u4 *>(lds + row * STRIDE + c * PER) = r.r[i];
        }
    }
    // four values of one row of the matrix (or column, where it is kept transposed), at row and col .. + 3
    static __device__ __forceinline__ void put4(E *to, int row, int col, f4 v) {
        if constexpr (IO::bytes == 4) {
            *reinterpret_cast<f4 *>(to + row * kC + col) = v;
        } else {
#pragma unroll
            for (int p = 0; p < PLANES; ++p) {
                b4 q;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    q[i] = (__bf16)v[i];
                    v[i] -= (float)q[i];
                }
                *reinterpret_cast<b4 *>(to + p * kC * kC + row * kC + col) = q;
            }
        }
    }
    static __device__ __forceinline__ void put(E *to, int row, int col, float v) {
#pragma unroll
        for (int p = 0; p < PLANES; ++p) {
            const E q = (E)v;
            to[p * kC * kC + row * kC + col] = q;
            v -= (float)q;
        }
    }
};

// What the chunks hand to the chains, one block per (row, head, chunk): the row vectors, the inverse and
// the attention matrix, both transposed for the backward chain.
enum { kVecKEnter, kVecKLeave, kVecQEnter, kVecBeta, kVecThrough, kVecs };

template <typename IO>
struct ChunkBlock {
    using Inv = ChunkMatrix<IO, 3>;
    using Att = ChunkMatrix<IO, 2>;   // forward: for the outputs alone
    using AttT = ChunkMatrix<IO, 3>;  // backward
    static constexpr size_t kVecBytes = kVecs * kC * sizeof(float);
    static constexpr size_t kInvBytes = Inv::ELEMS * IO::bytes;
    static constexpr size_t kBytes = kVecBytes + kInvBytes + AttT::ELEMS * IO::bytes;
};

// A state's column (rows of `to`, V apart) from a wave's registers.
template <int KT>
__device__ __forceinline__ void store_state(float *to, int K, int V, int grp, const f4 (&s)[KT]) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = pair_row(kt, grp, i);
            if (K == 16 * KT || k < K) to[k * V] = s[kt][i];
        }
}

// An element as it lies in memory, kept so until it is used.
template <typename IO>
struct RawOne {
    typename IO::storage v;
    __device__ __forceinline__ float get() const {
        if constexpr (IO::bytes == 2)
            return bf16_bits_to_f32(v);
        else
            return v;
    }
};
template <typename IO>
__device__ __forceinline__ RawOne<IO> load_one(const void *p, int64_t i) {
    return {static_cast<const typename IO::storage *>(p)[i]};
}

// Enqueue the chunks' kernel (gated_delta.hip); `blocks`: ChunkBlock<IO>::kBytes a chunk.
hipError_t launch_prepare(const Call &a, int io_dtype, bool backward, char *blocks, hipStream_t stream);
size_t block_bytes(int io_dtype);
// The forward chain; o, h_final and ck may be NULL.
hipError_t launch_chain(const Call &a, int io_dtype, const char *blocks, const float *h0, void *o, float *h_final,
                        float *ck, hipStream_t stream);
// The backward of a call (gated_delta_bwd.hip).
hipError_t launch_backward(const Call &c, const ssm_gated_delta_bwd_args_t &a, hipStream_t stream);
size_t backward_bytes(const ssm_gated_delta_bwd_args_t &a);

}  // namespace delta
}  // namespace ssm
