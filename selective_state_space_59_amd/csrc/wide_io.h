// wide_io.h -- 16-byte loads and stores at the alignment of an element (gfx950).
#pragma once

#include "ssm_device.h"

namespace ssm {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
// 16 bytes at the alignment of an element: one global_load_dwordx4 / store (the hardware takes
// unaligned addresses), so odd widths and shifted tensors run on the same path.
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));

// Eight consecutive elements as they lie in memory: 16 bytes of bf16, 32 of fp32.
template <typename IO>
struct Raw8 {
    static constexpr int Q = IO::bytes / 2;
    u32x4_t q[Q];
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (IO::bytes == 2) return __uint_as_float(e & 1 ? q[0][e / 2] & 0xffff0000u : q[0][e / 2] << 16);
        return __uint_as_float(q[e / 4][e % 4]);
    }
};

// Elements i .. i + 7 of p, of which the first n are there (the others read as 0).
template <typename IO>
__device__ __forceinline__ Raw8<IO> load8(const void *p, int64_t i, int n) {
    const char *at = static_cast<const char *>(p) + i * IO::bytes;
    Raw8<IO> r;
    if (n >= 8) {
#pragma unroll
        for (int k = 0; k < Raw8<IO>::Q; ++k) r.q[k] = reinterpret_cast<const u32x4_a2 *>(at)[k];
        return r;
    }
#pragma unroll
    for (int k = 0; k < Raw8<IO>::Q; ++k) r.q[k] = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) {
            if constexpr (IO::bytes == 2)
                r.q[0][e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(at)[e] << (16 * (e & 1));
            else
                r.q[e / 4][e % 4] = reinterpret_cast<const uint32_t *>(at)[e];
        }
    return r;
}

template <typename IO>
__device__ __forceinline__ void store8(void *p, int64_t i, int n, const float (&f)[8]) {
    char *at = static_cast<char *>(p) + i * IO::bytes;
    if (n >= 8) {
        if constexpr (IO::bytes == 2) {
            *reinterpret_cast<u32x4_a2 *>(at) = u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                        pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                reinterpret_cast<u32x4_a2 *>(at)[k] =
                    u32x4_t{__float_as_uint(f[4 * k]), __float_as_uint(f[4 * k + 1]), __float_as_uint(f[4 * k + 2]),
                            __float_as_uint(f[4 * k + 3])};
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) store_io<IO>(at, e, f[e]);
}

}  // namespace ssm
