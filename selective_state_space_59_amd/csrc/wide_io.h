// wide_io.h -- 16-byte loads and stores at the alignment of an element (gfx950).
#pragma once

#include "ssm_device.h"

namespace ssm {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
// 16 bytes at the alignment of an element: one global_load_dwordx4 / store (the hardware takes
// unaligned addresses), so odd widths and shifted tensors run on the same path.
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));

// E consecutive elements as they lie in memory, in pieces of 16 bytes (8 where they are no more).
template <typename IO, int E>
struct Raw {
    static constexpr int WORDS = E * IO::bytes / 4, N = WORDS < 4 ? WORDS : 4, Q = WORDS / N;
    typedef uint32_t piece_t __attribute__((ext_vector_type(N)));
    typedef piece_t piece_a2 __attribute__((aligned(2)));
    piece_t q[Q];
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (IO::bytes == 2) {
            const uint32_t w = q[e / 2 / N][e / 2 % N];
            return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
        }
        return __uint_as_float(q[e / N][e % N]);
    }
};

// Elements i .. i + E - 1 of p, of which the first n are there (the others read as 0).
template <typename IO, int E>
__device__ __forceinline__ Raw<IO, E> load_raw(const void *p, int64_t i, int n) {
    using RAW = Raw<IO, E>;
    constexpr int N = RAW::N;
    const char *at = static_cast<const char *>(p) + i * IO::bytes;
    RAW r = {};
    if (n >= E) {
#pragma unroll
        for (int k = 0; k < RAW::Q; ++k) r.q[k] = reinterpret_cast<const typename RAW::piece_a2 *>(at)[k];
        return r;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e < n) {
            if constexpr (IO::bytes == 2)
                r.q[e / 2 / N][e / 2 % N] |= (uint32_t)reinterpret_cast<const uint16_t *>(at)[e] << (16 * (e & 1));
            else
                r.q[e / N][e % N] = reinterpret_cast<const uint32_t *>(at)[e];
        }
    return r;
}

template <typename IO, int E>
__device__ __forceinline__ void store_raw(void *p, int64_t i, int n, const float (&f)[E]) {
    using RAW = Raw<IO, E>;
    constexpr int N = RAW::N;
    char *at = static_cast<char *>(p) + i * IO::bytes;
    if (n >= E) {
        RAW r;
#pragma unroll
        for (int w = 0; w < RAW::WORDS; ++w) {
            if constexpr (IO::bytes == 2)
                r.q[w / N][w % N] = pack_bf16x2(f[2 * w], f[2 * w + 1]);
            else
                r.q[w / N][w % N] = __float_as_uint(f[w]);
        }
#pragma unroll
        for (int k = 0; k < RAW::Q; ++k) reinterpret_cast<typename RAW::piece_a2 *>(at)[k] = r.q[k];
        return;
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e < n) store_io<IO>(at, e, f[e]);
}

}  // namespace ssm
