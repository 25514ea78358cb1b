// delta_tile.h -- operands, tiles and per-chunk gates of the gated delta rule's kernels (gfx950).
//
// A chunk is 64 steps.  All products run on 16 x 16 result tiles of the matrix cores, contracted 32 at
// a time: lane l holds row (A) or column (B) l % 16 and the eight consecutive contraction indices
// 8 (l / 16) .. + 7; the result has column l % 16 and, in register i, row 4 (l / 16) + i.
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
constexpr float kGrowth = 1.0f;  // a chunk in which decays multiply to more than e^kGrowth is marked (gated_delta_grow.hip)

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

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
    static __device__ __forceinline__ Ex first(const Ex &a) {
        return a;
    }
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
    template <int P, int Q>
    static __device__ __forceinline__ Sum<P> first(const Sum<Q> &a) {
        Sum<P> r;
#pragma unroll
        for (int i = 0; i < P; ++i) r.p[i] = a.p[i];
        return r;
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

// Sum over the 16 lanes of a row of results, in each of them: rotations within the row (ror 8, 4, 2, 1) in the
// vector unit, where shuffles would go through LDS.
template <int CTRL>
__device__ __forceinline__ float rotated(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum16(float x) {
    x += rotated<0x128>(x);
    x += rotated<0x124>(x);
    x += rotated<0x122>(x);
    return x + rotated<0x121>(x);
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
    int grows;      // whether a product of decays in the chunk exceeds e^kGrowth
};

// Wave 0 fills G, doc, beta, enter, leave, through and grows.  A barrier has to follow.
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
    // the largest G_t - G_s of a document (its entering state stands at 0)
    bool grows = false;
    if (__any(g > 0.0f)) {
        double low = doc == 0 ? fmin(G, 0.0) : G;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const double up = __shfl_up(low, d, 64);
            const int ud = __shfl_up(doc, d, 64);
            if (t >= d && ud == doc) low = fmin(low, up);
        }
        grows = __any(G - low > (double)kGrowth);
    }
    if (t == 0) {
        s.through = last == 0 ? expf((float)end) : 0.0f;
        s.grows = grows;
    }
}

// D_ts = product of the decays behind step s up to t, 0 where t does not see s (s <= t).
__device__ __forceinline__ float decay(const Gates &s, int t, int u) {
    return u <= t && s.doc[t] == s.doc[u] ? expf((float)(s.G[t] - s.G[u])) : 0.0f;
}

// 64 rows of K channels (rows from t0 on of one head) between memory, registers and LDS, 16 bytes a piece:
// lane = row.  Loads have no condition (a conditional one is waited for where its branch ends, and the next
// chunk's are to stay in flight).
template <typename IO, int KP>
struct HeadRows {
    using E = typename Op<IO>::elem;
    static constexpr int PER = 16 / IO::bytes;           // elements of a piece
    static constexpr int STRIDE = KP + PER;               // LDS row, in elements
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
};

// Planes of a matrix whose rows are `STRIDE` elements apart and whose planes are `PLANE` apart: the value
// itself in fp32, the sum of `P` bf16 numbers else.  Four consecutive values of a row, or one.
template <typename IO, int P, int PLANE>
__device__ __forceinline__ void put_planes4(typename Op<IO>::elem *to, f4 v) {
    if constexpr (IO::bytes == 4) {
        *reinterpret_cast<f4 *>(to) = v;
    } else {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            b4 q;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const b2 w = __builtin_convertvector((f2){v[2 * i], v[2 * i + 1]}, b2);
                q[2 * i] = w[0];
                q[2 * i + 1] = w[1];
            }
            if (p + 1 < P)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] -= (float)q[i];
            *reinterpret_cast<b4 *>(to + p * PLANE) = q;
        }
    }
}
template <typename IO, int P, int PLANE>
__device__ __forceinline__ void put_planes(typename Op<IO>::elem *to, float v) {
#pragma unroll
    for (int p = 0; p < (IO::bytes == 2 ? P : 1); ++p) {
        const typename Op<IO>::elem q = (typename Op<IO>::elem)v;
        to[p * PLANE] = q;
        v -= (float)q;
    }
}

// ROWS x WIDTH numbers in LDS as `P` planes (one in fp32), rows padded by 16 bytes.
template <typename IO, int ROWS, int WIDTH, int P>
struct Slab {
    using E = typename Op<IO>::elem;
    static constexpr int PLANES = IO::bytes == 2 ? P : 1;
    static constexpr int STRIDE = WIDTH + 16 / IO::bytes, PLANE = ROWS * STRIDE;
    alignas(16) E e[PLANES * PLANE];
    __device__ __forceinline__ void put4(int row, int col, f4 v) {
        put_planes4<IO, PLANES, PLANE>(e + row * STRIDE + col, v);
    }
    __device__ __forceinline__ void put(int row, int col, float v) {
        put_planes<IO, PLANES, PLANE>(e + row * STRIDE + col, v);
    }
    // the first N planes of the eight numbers at row, col
    template <int N = PLANES>
    __device__ __forceinline__ auto get(int row, int col) const {
        return Op<IO>::template planes<N>(e + row * STRIDE + col, PLANE);
    }
    __device__ __forceinline__ auto get_exact(int row, int col) const { return Op<IO>::load(e + row * STRIDE + col); }
};

// Element (row, col) of a matrix of 64 columns kept as the left operands of its 16 x 32 tiles, 64 lanes of
// eight elements each: a wave loads a tile as one run of memory.
__device__ __forceinline__ constexpr int tiled(int row, int col) {
    return ((row / 16 * 2 + col / 32) * 64 + row % 16 + col % 32 / 8 * 16) * 8 + col % 8;
}

// What the chunks hand to the chains, one block per (row, head, chunk) in the workspace: vectors over the
// steps; the inverse and the attention matrix (transposed for the backward chain), planes of 64 x 64; the
// keys, and for the backward the queries, transposed (KP x 64).  All matrices tiled.  For the backward the
// chunk's gates as well.
enum { kVecKEnter, kVecKLeave, kVecQEnter, kVecBeta, kVecThrough, kVecs };

template <typename IO, int KP, bool BWD>
struct ChunkBlock {
    using E = typename Op<IO>::elem;
    static constexpr int PLANE = kC * kC;
    static constexpr int INV = IO::bytes == 2 ? 3 : 1;            // planes of the inverse
    static constexpr int ATT = IO::bytes == 2 ? (BWD ? 3 : 2) : 1;  // forward: for the outputs alone
    static constexpr size_t kInv = kVecs * kC * sizeof(float);    // byte offsets
    static constexpr size_t kAtt = kInv + (size_t)INV * PLANE * IO::bytes;
    static constexpr size_t kKt = kAtt + (size_t)ATT * PLANE * IO::bytes;
    static constexpr size_t kQt = kKt + (size_t)KP * kC * IO::bytes;
    static constexpr size_t kGates = kQt + (size_t)KP * kC * IO::bytes;  // backward: the gates, for the gradients
    static constexpr size_t kBytes = BWD ? kGates + (sizeof(Gates) + 15) / 16 * 16 : kQt;
};

// The chains' workgroups: one head's 16 NC value channels each, heads dealt out to the 8 XCDs (workgroups
// go to them in turn), so that the workgroups that read the same chunks share an L2.
struct ChainPlace {
    int64_t head;
    int slice;
    bool any;
};
__device__ __forceinline__ ChainPlace chain_place(int64_t heads, int slices) {
    const int64_t turn = blockIdx.x / 8;
    ChainPlace p;
    p.head = turn / slices * 8 + blockIdx.x % 8;
    p.slice = (int)(turn % slices);
    p.any = p.head < heads;
    return p;
}
inline unsigned chain_grid(int64_t heads, int slices) { return (unsigned)((heads + 7) / 8 * 8 * slices); }
// Whether slices of 32 value channels leave a workgroup for each CU.
inline bool wide_slices(const Call &a) { return a.B * a.H * ((a.V + 31) / 32) >= 256; }

// A tensor's place for a whole wave and a lane's distance from it in bytes: one address register a lane.
template <typename T>
__device__ __forceinline__ T &at(const void *base, uint32_t off) {
    return *reinterpret_cast<T *>(const_cast<char *>(static_cast<const char *>(base)) + off);
}
template <typename T>
__device__ __forceinline__ const char *bytes(const T *p, int64_t elements, int64_t size) {
    return reinterpret_cast<const char *>(p) + elements * size;
}

// A lane's first value channel in a chain's workgroup: two of them lie side by side, so that they are loaded and
// stored together (V is even: both are there or neither).
template <int NC>
__device__ __forceinline__ int channel(int slice, int r16) {
    return NC * (16 * slice + r16);
}
typedef f2 f2_a4 __attribute__((aligned(4)));
typedef uint32_t u1_a2 __attribute__((aligned(2)));

// NC neighbouring floats, or elements, at a lane's channels.
template <int NC>
__device__ __forceinline__ void store_floats(void *row, uint32_t off, const float (&x)[NC]) {
    if constexpr (NC == 2)
        at<f2_a4>(row, off) = f2{x[0], x[1]};
    else
        at<float>(row, off) = x[0];
}
template <typename IO, int NC>
__device__ __forceinline__ void store_elements(void *row, uint32_t off, const float (&x)[NC]) {
    if constexpr (IO::bytes == 4)
        store_floats<NC>(row, off, x);
    else if constexpr (NC == 2)
        at<u1_a2>(row, off) = pack_bf16x2(x[0], x[1]);
    else
        store_io<IO>(&at<char>(row, off), 0, x[0]);
}

// A wave's rows of a state (from k0 on, V floats each) into memory.
template <int ST, int NC>
__device__ __forceinline__ void store_rows(char *to, uint32_t v_row, int K, int k0, bool every, uint32_t v0, bool live,
                                           const f4 (&s)[ST][NC]) {
    if (!live) return;
#pragma unroll
    for (int j = 0; j < ST; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (every || k0 + 16 * j + i < K) {
                float x[NC];
#pragma unroll
                for (int n = 0; n < NC; ++n) x[n] = s[j][n][i];
                store_floats<NC>(to + (16 * j + i) * (int64_t)v_row, k0 * v_row + v0 * 4, x);
            }
}

// NC neighbouring elements as they lie in memory, kept so until they are used.
template <typename IO, int NC>
struct Elements {
    typedef typename IO::storage one;
    one v[NC];
    static __device__ __forceinline__ Elements load(const void *row, uint32_t off) {
        Elements r;
        if constexpr (NC == 2 && IO::bytes == 2) {
            const uint32_t w = at<u1_a2>(row, off);
            __builtin_memcpy(&r.v, &w, 4);
        } else if constexpr (NC == 2) {
            const f2 w = at<f2_a4>(row, off);
            r.v[0] = w[0];
            r.v[1] = w[1];
        } else {
            r.v[0] = at<one>(row, off);
        }
        return r;
    }
    __device__ __forceinline__ float get(int n) const {
        if constexpr (IO::bytes == 2)
            return bf16_bits_to_f32(v[n]);
        else
            return v[n];
    }
};

// A call's workspace begins with a mark for each chunk of each head (marks_bytes), then the chunks' blocks
// (block_bytes each).
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }
inline size_t marks_bytes(int64_t chunks) { return up256((size_t)chunks * sizeof(uint32_t)); }
// Enqueue the chunks' kernel (gated_delta.hip).
hipError_t launch_prepare(const Call &a, int io_dtype, bool backward, char *workspace, hipStream_t stream);
size_t block_bytes(int io_dtype, int64_t kdim, bool backward);
// The forward chain, and the heads that grow; o, h_final and ck may be NULL.  `workspace`: chain_bytes.
hipError_t launch_chain(const Call &a, int io_dtype, char *workspace, const float *h0, void *o, float *h_final, float *ck,
                        hipStream_t stream);
size_t chain_bytes(int io_dtype, int64_t heads, int64_t n, int64_t kdim, int64_t vdim);
// Heads with a marked chunk again, step by step (gated_delta_grow.hip); key heads of one backwards.
hipError_t launch_grow(const Call &a, int io_dtype, const uint32_t *marks, const float *h0, void *o, float *h_final,
                       float *ck, hipStream_t stream);
hipError_t launch_grow_back(const Call &c, const ssm_gated_delta_bwd_args_t &a, const uint32_t *marks, const float *ck,
                            char *blocks, float *dbeta_sum, hipStream_t stream);
// The backward of a call (gated_delta_bwd.hip).
hipError_t launch_backward(const Call &c, const ssm_gated_delta_bwd_args_t &a, hipStream_t stream);
size_t backward_bytes(const ssm_gated_delta_bwd_args_t &a);

}  // namespace delta
}  // namespace ssm
