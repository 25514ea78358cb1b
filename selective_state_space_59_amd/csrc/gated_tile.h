// gated_tile.h -- what the forward and backward tile kernels of the gated recurrence share
// (gfx950): 16-byte loads and stores at any element alignment, the combination of runs of
// steps, and the hand-over of states between the tiles of a sequence.
#pragma once

#include "gated_device.h"
#include "wide_io.h"

namespace ssm {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x2_t u32x2_a2 __attribute__((aligned(2)));

// A lane holds W words (4 bytes) of each of its rows: 4, or 2 for the decode step's bf16.
template <int W>
struct Words {
    static_assert(W == 4 || W == 2, "16 or 8 bytes a lane");
    uint32_t w[W];
};

template <int W>
__device__ __forceinline__ Words<W> load_words(const char *p) {
    Words<W> r;
    if constexpr (W == 4) {
        const u32x4_t v = *reinterpret_cast<const u32x4_a2 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = v[i];
    } else {
        const u32x2_t v = *reinterpret_cast<const u32x2_a2 *>(p);
        r.w[0] = v[0];
        r.w[1] = v[1];
    }
    return r;
}

template <int W>
__device__ __forceinline__ void store_words(char *p, const Words<W> &q) {
    if constexpr (W == 4)
        *reinterpret_cast<u32x4_a2 *>(p) = u32x4_t{q.w[0], q.w[1], q.w[2], q.w[3]};
    else
        *reinterpret_cast<u32x2_a2 *>(p) = u32x2_t{q.w[0], q.w[1]};
}

// How a tile lies over a workgroup: THREADS lanes, W words of R consecutive rows each; the lanes
// of a row cover kRowBytes.  128 bytes give a layer of 1536 channels 24 blocks a row, and the lanes
// of a row one whole line; pieces of 256 or 512 bytes, with as many times fewer and larger
// workgroups, ran the 8 x 2048 x 1536 bf16 forward in 82 and 99 us where 128 took 71 (in tiles of
// 128 steps, ahead of the steps that took it to 52).
constexpr int kRowBytes = 128;

template <typename IO, int W_, int R_, int THREADS_>
struct Tile {
    static constexpr int W = W_, R = R_, THREADS = THREADS_;
    static constexpr int V = 4 * W / IO::bytes;           // channels of a lane
    static constexpr int LANES = kRowBytes / (4 * W);     // lanes of a row
    static constexpr int CB = kRowBytes / IO::bytes;      // channels of a workgroup
    static constexpr int G = THREADS / LANES;             // lane groups, one behind the other in time
    static constexpr int T = G * R;                       // steps
};

// Calls f(std::integral_constant<int, steps>) with the steps of a sequence's tiles: FULL, or, where it
// ends sooner, the least of 32, 64, ... that hold it (one tile, no chain).  A longer tile would load and
// compute steps that are not there: training steps in bf16 RATE, 256 x 16 x 5120 184 us against 819 in
// full tiles, 64 x 48 x 2048 52 against 96, 64 x 100 x 2048 92 against 106.
template <int FULL, int STEPS = 32, typename F>
void with_steps(int64_t seqlen, F &&f) {
    if constexpr (STEPS < FULL)
        if (seqlen > STEPS) return with_steps<FULL, STEPS * 2>(seqlen, f);
    f(std::integral_constant<int, STEPS>{});
}

// What the channel count asks of a lane's loads; a variant of its own for each, because a branch
// per tensor makes the compiler wait for one tensor before it loads the next (3 x 1237 x 331 fp32,
// backward: 26 us with such a branch, 12 us without).
enum Edge {
    kWhole,   // a multiple of a lane's channels: lanes are full or past the end
    kRagged,  // at least one lane's channels: the last lane of a row loads the row's last V channels
              // and shifts them into place
    kTiny     // fewer: element by element
};

template <typename IO, int W>
constexpr int lane_channels = 4 * W / IO::bytes;

inline Edge edge_of(int64_t dim, int V) { return dim % V == 0 ? kWhole : dim > V ? kRagged : kTiny; }

template <typename F>
void with_edge(Edge e, F &&f) {
    if (e == kWhole)
        f(std::integral_constant<int, kWhole>{});
    else if (e == kRagged)
        f(std::integral_constant<int, kRagged>{});
    else
        f(std::integral_constant<int, kTiny>{});
}

// A lane's channels d0 .. d0 + V - 1, of which nv are there; it loads from `load` on, `shift`
// channels earlier (lanes past the end load what is there and use none of it).
struct Cols {
    int d0, nv, load, shift;
};
template <int EDGE>
__device__ __forceinline__ Cols cols_of(int d0, int D, int V) {
    Cols c = {d0, min(V, D - d0), d0, 0};
    if constexpr (EDGE != kTiny) c.load = min(d0, D - V);
    if constexpr (EDGE == kRagged) c.shift = c.nv > 0 ? d0 - c.load : 0;
    return c;
}

// One word group by elements (nv of them, the others 0).
template <typename IO, int W>
__device__ __forceinline__ Words<W> load_elements(const char *p, int nv) {
    Words<W> q = {};
#pragma unroll
    for (int e = 0; e < lane_channels<IO, W>; ++e)
        if (e < nv) {
            if constexpr (IO::bytes == 2)
                q.w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[e] << (16 * (e & 1));
            else
                q.w[e] = reinterpret_cast<const uint32_t *>(p)[e];
        }
    return q;
}

// R rows of a lane, `off[j]` bytes behind the wave-uniform `base`.
template <typename IO, int EDGE, int W, int R>
__device__ __forceinline__ void load_rows(const char *base, const uint32_t (&off)[R], int nv, Words<W> (&q)[R]) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if constexpr (EDGE == kTiny)
            q[j] = load_elements<IO, W>(base + off[j], nv);
        else
            q[j] = load_words<W>(base + off[j]);
    }
}

// Drops the first `shift` (< V) channels of a ragged lane's rows.
template <typename IO, int W, int R>
__device__ __forceinline__ void shift_rows(Words<W> (&q)[R], int shift) {
    if (shift == 0) return;
    constexpr int PER = 4 / IO::bytes;  // channels of a word
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if (PER == 2 && (shift & 1))
#pragma unroll
            for (int i = 0; i < W; ++i) q[j].w[i] = q[j].w[i] >> 16 | (i + 1 < W ? q[j].w[i + 1] << 16 : 0);
#pragma unroll
        for (int by = 1; by < W; by *= 2)
            if (shift / PER & by)
#pragma unroll
                for (int i = 0; i < W; ++i) q[j].w[i] = i + by < W ? q[j].w[i + by] : 0;
    }
}

// V channels of one row where they may be fewer (a single row: nothing to wait for in between).
template <typename IO, int W>
__device__ __forceinline__ Words<W> load_some(const char *p, int nv) {
    return nv >= lane_channels<IO, W> ? load_words<W>(p) : load_elements<IO, W>(p, nv);
}

template <typename IO, int W>
__device__ __forceinline__ void store_row(char *p, int nv, const Words<W> &q) {
    constexpr int V = 4 * W / IO::bytes;
    if (nv >= V) {
        store_words(p, q);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < nv) {
                if constexpr (IO::bytes == 2)
                    reinterpret_cast<uint16_t *>(p)[e] = (uint16_t)(q.w[e / 2] >> (16 * (e & 1)));
                else
                    reinterpret_cast<uint32_t *>(p)[e] = q.w[e];
            }
    }
}

template <typename IO, int W>
__device__ __forceinline__ float lane_elem(const Words<W> &q, int v) {
    if constexpr (IO::bytes == 2) return __uint_as_float(v & 1 ? q.w[v / 2] & 0xffff0000u : q.w[v / 2] << 16);
    return __uint_as_float(q.w[v]);
}

template <typename IO, int W>
__device__ __forceinline__ Words<W> lane_pack(const float (&f)[4 * W / IO::bytes]) {
    Words<W> q;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if constexpr (IO::bytes == 2)
            q.w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        else
            q.w[i] = __float_as_uint(f[i]);
    }
    return q;
}

// V floats of a lane to LDS.
template <int V>
__device__ __forceinline__ void lds_put(float *p, const float (&f)[V]) {
    static_assert(V % 4 == 0, "16 bytes at a time");
#pragma unroll
    for (int v = 0; v < V; v += 4) *reinterpret_cast<float4 *>(p + v) = make_float4(f[v], f[v + 1], f[v + 2], f[v + 3]);
}

// A run of steps maps the state h entering it to p h + l (p the product of its decays, l its
// states from 0), or to l alone once it holds a reset: p is then NaN, which every later product
// keeps, and a select drops the entering state whatever it holds.  (A NaN decay makes l NaN too,
// so it is not lost.)  With RATE an entering 0 gives l also where p is an infinity: decays above 1
// take no input, so every state may be 0 while their product leaves the range.  (The rows of a tile
// have a branch for it: a select on every element took the 1M-token forward from 1685 to 1725 us.
// SIGMOID, whose p is at most 1, does without: the second test took its packed backward from 180 to
// 186 us.)
template <int MODE>
__device__ __forceinline__ float run_apply(float p, float l, float h) {
    const bool alone = MODE == SSM_GATE_RATE ? (p != p) | (h == 0.0f) : p != p;
    return alone ? l : __builtin_fmaf(p, h, l);
}

// ---- states between the tiles of one (batch row, channel block): a chain
//
// Each tile leaves one 8-byte record per channel: first its own (p, l), as soon as it has read
// its inputs, then the state after it.  A tile reads the records before it, backwards, until it
// meets a state.  A record is one atomic word, so it needs no flag and no fence: the high word
// tells what it holds, with two NaN patterns that p is never stored as.
constexpr uint32_t kRecEmpty = 0xffffffffu, kRecState = 0xfffffffeu;
constexpr int kLook = 8;  // records looked at together (4: 1M tokens 6% slower; 16: more registers, no faster)

typedef unsigned long long u64_t;

__device__ __forceinline__ void rec_put(u64_t *r, uint32_t hi, float lo) {
    __hip_atomic_store(r, ((u64_t)hi << 32) | __float_as_uint(lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state entering tile k (k > 0) of a chain whose records are `stride` apart; rec: this
// lane's channel in tile k's place.  The states are always formed oldest first,
// state_i = apply(run_i, state_{i-1}), so the result does not depend on how far back the nearest
// state was found.
//
// Every wait ends: a tile's number in its chain is a ticket drawn when its workgroup already
// runs, so the tiles before it belong to workgroups that run or have ended, the first never
// waits, and a tile leaves its state without waiting for a later one.
template <int MODE>
__device__ __forceinline__ float chain_enter(const u64_t *rec, int64_t stride, int k) {
    for (;;) {
        u64_t v[kLook];
#pragma unroll
        for (int j = 0; j < kLook; ++j)
            v[j] = j < k ? __hip_atomic_load(rec - (int64_t)(j + 1) * stride, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT)
                         : ~(u64_t)0;
        float h = 0.0f;
        bool known = false;  // h is the state after the record at hand
#pragma unroll
        for (int j = kLook - 1; j >= 0; --j) {
            const uint32_t hi = (uint32_t)(v[j] >> 32);
            const float lo = __uint_as_float((uint32_t)v[j]);
            known = hi == kRecState || (known && hi != kRecEmpty);
            h = hi == kRecState ? lo : run_apply<MODE>(__uint_as_float(hi), lo, h);
        }
        if (__all(known)) return h;
        __builtin_amdgcn_s_sleep(1);
    }
}

// p as a record's high word: one NaN pattern for every NaN.
__device__ __forceinline__ uint32_t rec_hi(float p) { return p != p ? 0x7fc00000u : __float_as_uint(p); }

// The chain of workgroup i of chains * tiles (the tile within it is the ticket it draws).
// Workgroups go to the XCDs in turn.  A short chain's tiles are dealt out one chain after the
// other; a long chain's run over all XCDs, eight at a time, so that no chain waits for one XCD that
// is behind.  Dealt out against spread, bf16 RATE forward, 16384 steps of 1536 channels (131072 in the
// last): 8 tiles a chain 52.0 and 54.2 us, 16 52.1 and 53.1, 32 53.4 and 53.7, 64 54.8 and 55.1, 128
// 105.9 and 97.9 (32768 steps), 512 383 and 342; of 5120 channels 16 tiles 166 and 158, 64 169 and 159,
// so wide layers would gain from a spread of 16 and 32 tiles too.  The backward (tiles of 128
// steps): even up to 64 tiles, 1134 and 1028 us a training step of 131072.
// Either way every chain gets `tiles`.
constexpr int kLongChain = 64;

__device__ __forceinline__ int chain_of(unsigned i, int chains, int tiles) {
    constexpr int kXcds = 8;
    const unsigned whole = (unsigned)(tiles / kXcds * kXcds) * chains;
    if (tiles < kLongChain || i >= whole) return i % chains;
    return i / kXcds % chains;
}

// Workspace of a chained launch: the records, then one ticket counter per chain.
struct ChainPlan {
    int64_t chains, tiles, cb;
    size_t rec_bytes() const { return (size_t)(chains * tiles * cb) * 8; }
    size_t bytes() const { return tiles > 1 ? (rec_bytes() + (size_t)chains * 4 + 255) & ~(size_t)255 : 0; }
};

// Empties the records and counters (a kernel, so that it can be captured).
hipError_t launch_chain_init(const ChainPlan &p, void *workspace, hipStream_t stream);

}  // namespace ssm
