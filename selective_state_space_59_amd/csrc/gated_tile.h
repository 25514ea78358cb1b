// gated_tile.h -- what the forward and backward tile kernels of the gated recurrence share
// (gfx950): 16-byte loads and stores at any element alignment, the combination of runs of
// steps, and the hand-over of states between the tiles of a sequence.
#pragma once

#include "gated_device.h"
#include "wide_io.h"

namespace ssm {

constexpr int kLanesPerRow = 8;  // 8 lanes x 16 bytes: a 128-byte piece of a row
constexpr int kGatedThreads = 256;
constexpr int kRowGroups = kGatedThreads / kLanesPerRow;  // lane groups stacked in time

template <typename IO>
struct TileShape {
    static constexpr int V = 16 / IO::bytes;        // channels of a lane
    static constexpr int CB = V * kLanesPerRow;     // channels of a workgroup: 64 (bf16), 32 (fp32)
};

// R rows of a lane: `off[j]` bytes behind the wave-uniform `base`, `nv` valid channels (the last
// channel block of an odd width takes its elements one by one).
template <typename IO, int R>
__device__ __forceinline__ void load_rows(const char *base, const uint32_t (&off)[R], int nv, u32x4_t (&q)[R]) {
    constexpr int V = TileShape<IO>::V;
    if (nv == V) {
#pragma unroll
        for (int j = 0; j < R; ++j) q[j] = *reinterpret_cast<const u32x4_a2 *>(base + off[j]);
    } else {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            u32x4_t v = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e < nv) {
                    if constexpr (IO::bytes == 2)
                        v[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(base + off[j])[e] << (16 * (e & 1));
                    else
                        v[e] = reinterpret_cast<const uint32_t *>(base + off[j])[e];
                }
            q[j] = v;
        }
    }
}

template <typename IO>
__device__ __forceinline__ float lane_elem(const u32x4_t &q, int v) {
    if constexpr (IO::bytes == 2) return __uint_as_float(v & 1 ? q[v / 2] & 0xffff0000u : q[v / 2] << 16);
    return __uint_as_float(q[v]);
}

template <typename IO>
__device__ __forceinline__ u32x4_t lane_pack(const float (&f)[TileShape<IO>::V]) {
    u32x4_t q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (IO::bytes == 2)
            q[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        else
            q[i] = __float_as_uint(f[i]);
    }
    return q;
}

template <typename IO>
__device__ __forceinline__ void store_words(char *p, int nv, const u32x4_t &q) {
    constexpr int V = TileShape<IO>::V;
    if (nv == V) {
        *reinterpret_cast<u32x4_a2 *>(p) = q;
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < nv) {
                if constexpr (IO::bytes == 2)
                    reinterpret_cast<uint16_t *>(p)[e] = (uint16_t)(q[e / 2] >> (16 * (e & 1)));
                else
                    reinterpret_cast<uint32_t *>(p)[e] = q[e];
            }
    }
}

// A run of steps maps the state h entering it to p h + l (p the product of its decays, l its
// states from 0), or to l alone once it holds a reset: p is then NaN, which every later product
// keeps, and a select drops the entering state whatever it holds.  (A NaN decay makes l NaN too,
// so it is not lost.)
__device__ __forceinline__ float run_apply(float p, float l, float h) {
    return p != p ? l : __builtin_fmaf(p, h, l);
}

// ---- states between the tiles of one (batch row, channel block): a chain
//
// Each tile leaves one 8-byte record per channel: first its own (p, l), as soon as it has read
// its inputs, then the state after it.  A tile reads the records before it, backwards, until it
// meets a state.  A record is one atomic word, so it needs no flag and no fence: the high word
// tells what it holds, with two NaN patterns that p is never stored as.
constexpr uint32_t kRecEmpty = 0xffffffffu, kRecState = 0xfffffffeu;
constexpr int kLook = 8;  // records read at once

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
__device__ __forceinline__ float chain_enter(const u64_t *rec, int64_t stride, int k) {
    float h = 0.0f;
    bool found = false;
    while (!found) {
        u64_t v[kLook];
#pragma unroll
        for (int j = 0; j < kLook; ++j)
            v[j] = j < k ? __hip_atomic_load(rec - (int64_t)(j + 1) * stride, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT)
                         : ~(u64_t)0;
        int at = -1;
        bool open = true;
#pragma unroll
        for (int j = 0; j < kLook; ++j) {
            const uint32_t hi = (uint32_t)(v[j] >> 32);
            if (open && hi == kRecState) at = j;
            open = open && hi != kRecState && hi != kRecEmpty;
        }
        if (at >= 0) {
#pragma unroll
            for (int j = kLook - 1; j >= 0; --j) {
                const float lo = __uint_as_float((uint32_t)v[j]), p = __uint_as_float((uint32_t)(v[j] >> 32));
                if (j == at)
                    h = lo;
                else if (j < at)
                    h = run_apply(p, lo, h);
            }
            found = true;
        } else {
            __builtin_amdgcn_s_sleep(1);
        }
    }
    return h;
}

// p as a record's high word: one NaN pattern for every NaN.
__device__ __forceinline__ uint32_t rec_hi(float p) { return p != p ? 0x7fc00000u : __float_as_uint(p); }

// Workspace of a chained launch: the records, then one ticket counter per chain.
struct ChainPlan {
    int64_t chains, tiles, cb;
    size_t rec_bytes() const { return (size_t)(chains * tiles * cb) * 8; }
    size_t bytes() const { return tiles > 1 ? (rec_bytes() + (size_t)chains * 4 + 255) & ~(size_t)255 : 0; }
};

// Empties the records and counters (a kernel, so that it can be captured).
hipError_t launch_chain_init(const ChainPlan &p, void *workspace, hipStream_t stream);

}  // namespace ssm
