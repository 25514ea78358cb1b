// matmul_fp8.hip -- the product of two e4m3 matrices with block scales (ssm_matmul_fp8) on gfx950:
//   y[m,n] = sum_j sx[m,j] sw[n/128,j] sum_{k in block j} x[m,k] w[n,k]
// One matrix instruction (16 x 16, 128 deep) sums a block's 128 products of a tile; its result is added to
// the fp32 sums with the two scales.  w is the left operand, so that a lane holds four neighbouring
// columns of y and ONE row, whose scale is then one number a tile.
#include "ssm_device.h"
#include "ssm_internal.h"

#include <algorithm>

namespace ssm {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i8 __attribute__((ext_vector_type(8)));

constexpr int kOne = 0x7f7f7f7f;  // 1.0 in the exponent bytes of the scaled instruction

// 32 bytes of a row as a block's product takes them.  The 8-bit instruction adds the products of a lane in
// groups of eight, aligned to the largest of each: what lies 2^14 below it is lost, less than 7 * 2^-14 of the
// sum of all magnitudes.  For random data that is 1.5e-5 of the result, far below a bf16 result's own rounding
// (2e-3), and more than it only where large terms cancel; for an fp32 result the values are widened to bf16,
// exactly, and summed by the bf16 instruction at half the rate.
template <typename OUT>
struct Operand {
    i8 v;
    Operand() = default;
    __device__ __forceinline__ Operand(i4 a, i4 b) : v{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]} {}
};
template <>
struct Operand<io_f32> {
    b8 v[4];
    Operand() = default;
    __device__ __forceinline__ Operand(i4 a, i4 b) {
        const int w[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const b2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false);
            const b2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true);
            const int e = i % 2 * 4;
            v[i / 2][e] = lo[0];
            v[i / 2][e + 1] = lo[1];
            v[i / 2][e + 2] = hi[0];
            v[i / 2][e + 3] = hi[1];
        }
    }
};

__device__ __forceinline__ int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

__device__ __forceinline__ f4 block_product(const Operand<io_bf16> &w, const Operand<io_bf16> &x) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, f4{0, 0, 0, 0}, 0, 0, 0, kOne, 0, kOne);
}
__device__ __forceinline__ f4 block_product(const Operand<io_f32> &w, const Operand<io_f32> &x) {
    f4 p = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], p, 0, 0, 0);
    return p;
}

template <typename OUT>
__device__ __forceinline__ void store4(const ssm_matmul_fp8_args_t &a, int64_t m, int64_t n, f4 v, bool wide) {
    if (m >= a.m || n >= a.n) return;
    const int64_t at = m * a.n + n;
    if (wide) {
        if constexpr (OUT::bytes == 2)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.y) + at) =
                make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        else
            *reinterpret_cast<f4 *>(static_cast<float *>(a.y) + at) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < a.n) store_io<OUT>(a.y, at + i, v[i]);
}

// ---------------------------------------------------------------------------------- few rows
// Up to 16 MT rows: w is read once, straight into registers.  A workgroup owns 16 rows of w; its waves
// share out the blocks of K and add their sums up in LDS.
constexpr int kSkinnyWaves = 4;

template <typename OUT, int MT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_kernel(ssm_matmul_fp8_args_t a, int blocks, bool wide) {
    __shared__ __attribute__((aligned(16))) f4 part[kSkinnyWaves][MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane % 16, grp = lane / 16;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const char *w = static_cast<const char *>(a.wq) + least(n0 + r16, a.n - 1) * a.k;
    const float *sw = a.w_scales + n0 / 128 * blocks;
    const char *x[MT];
    const float *sx[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t m = least(16 * t + r16, a.m - 1);
        x[t] = static_cast<const char *>(a.xq) + m * a.k;
        sx[t] = a.x_scales + m * blocks;
    }
    // 16 bytes at k, 0 behind the row's end
    const auto piece = [&](const char *row, int64_t k) {
        return k < a.k ? *reinterpret_cast<const i4 *>(row + k) : i4{0, 0, 0, 0};
    };
    f4 acc[MT] = {};
    for (int j = wave; j < blocks; j += kSkinnyWaves) {
        const int64_t k = 128 * (int64_t)j + 16 * grp;
        const Operand<OUT> wv(piece(w, k), piece(w, k + 64));
        const float s = sw[j];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const f4 p = block_product(wv, Operand<OUT>(piece(x[t], k), piece(x[t], k + 64)));
            const float st = s * sx[t][j];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(p[i], st, acc[t][i]);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    for (int t = wave; t < MT; t += kSkinnyWaves) {
        f4 v = part[0][t][lane];
#pragma unroll
        for (int i = 1; i < kSkinnyWaves; ++i) v += part[i][t][lane];
        store4<OUT>(a, 16 * t + r16, n0 + 4 * grp, v, wide);
    }
}

// -------------------------------------------------------------------------------------- tiles
__device__ const i4 kZeros[1] = {};

typedef __attribute__((address_space(3))) void *lds_ptr;
typedef const __attribute__((address_space(1))) void *global_ptr;

constexpr int kRun = 8;

// BM x BN of y a workgroup, WM x WN a wave (WN divides 128).  Both operands of a block of K go straight
// from memory to LDS, 16 bytes a lane, one block ahead of the products.  A row's eight pieces of 16 bytes
// are kept in the order piece ^ (row % 8), by the address each lane loads from, so that the 16 rows of an
// operand are read without bank conflicts.
template <typename OUT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(BM / WM * (BN / WN) * 64) void tile_kernel(ssm_matmul_fp8_args_t a, int blocks, int tiles_m,
                                                                       int tiles_n, bool wide) {
    constexpr int WAVES = BM / WM * (BN / WN), MT = WM / 16, NT = WN / 16;
    constexpr int LOADS = (BM + BN) / 8 / WAVES;  // of 8 rows each
    constexpr int THREADS = 64 * WAVES, NB = (BN + 127) / 128;  // w's blocks a workgroup meets
    __shared__ __attribute__((aligned(1024))) char lds[2][(BM + BN) * 128];
    __shared__ float scales[2][kRun][BM], w_scales[2][kRun][NB];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane % 16, grp = lane / 16;
    // Tiles by XCD (workgroups are dealt out to the 8 in turn): each takes a run of tiles, in columns of up
    // to 8 rows of tiles, so that the tiles it works on at one time share rows of x and w in its L2.
    const int total = tiles_m * tiles_n, xcd = blockIdx.x % 8, each = total / 8, more = total % 8;
    const int id = xcd * each + min(xcd, more) + (int)blockIdx.x / 8;
    const int band = id / (8 * tiles_n), high = min(8, tiles_m - 8 * band), in = id - band * 8 * tiles_n;
    const int64_t m0 = (int64_t)(8 * band + in % high) * BM, n0 = (int64_t)(in / high) * BN;

    // x's loads of a wave come first, then w's: a wave has one kind only (BM and BN are multiples of its rows)
    static_assert(BM % (8 * LOADS) == 0 && BN % (8 * LOADS) == 0, "");
    const bool of_x = wave * LOADS * 8 < BM;
    const int first = wave * LOADS * 8 - (of_x ? 0 : BM);
    const int64_t row0 = of_x ? m0 : n0, left = (of_x ? a.m : a.n) - 1 - row0;
    const char *src = static_cast<const char *>(of_x ? a.xq : a.wq) + row0 * a.k;
    const int piece = 16 * (lane % 8 ^ lane / 8);
    uint32_t off[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) off[j] = (uint32_t)least(first + 8 * j + lane / 8, left) * (uint32_t)a.k + piece;
    const int wm = wave / (BN / WN) * WM, wn = wave % (BN / WN) * WN;
    // The scales go through LDS, kRun blocks of K at a time: a row's lie side by side, and fetching one
    // for each of 16 rows every block cost more than the operands (3000 cycles of a block's 6700).
    constexpr int PER = kRun * BM / THREADS;
    const int s_row = threadIdx.x / (kRun / PER), s_at = threadIdx.x % (kRun / PER) * PER;
    const float *sx = a.x_scales + least(m0 + s_row, a.m - 1) * blocks;
    const int w_at = threadIdx.x % (kRun * NB) / NB;
    const float *sw = a.w_scales + least(n0 / 128 + threadIdx.x % NB, (a.n - 1) / 128) * blocks;
    float ahead[PER], ahead_w;
    const auto load_scales = [&](int j) {
#pragma unroll
        for (int i = 0; i < PER; ++i) ahead[i] = sx[min(j + s_at + i, blocks - 1)];
        ahead_w = sw[min(j + w_at, blocks - 1)];
    };
    const auto keep_scales = [&](int run) {
#pragma unroll
        for (int i = 0; i < PER; ++i) scales[run % 2][s_at + i][s_row] = ahead[i];
        if (threadIdx.x < kRun * NB) w_scales[run % 2][w_at][threadIdx.x % NB] = ahead_w;
    };

    const auto fetch = [&](int j, int buf) {
        const char *from = src + 128 * (int64_t)j;
        char *to = lds[buf] + wave * LOADS * 1024;
        if (128 * (int64_t)(j + 1) <= a.k) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                // (kept a base and a distance: the sums, formed once, would take two registers each)
                uint32_t o = off[i];
                asm volatile("" : "+v"(o));
                __builtin_amdgcn_global_load_lds((global_ptr)(from + o), (lds_ptr)(to + i * 1024), 16, 0, 0);
            }
        } else {  // behind a row's end: zeros
            const bool in = 128 * (int64_t)j + piece < a.k;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                uint32_t o = off[i];
                asm volatile("" : "+v"(o));
                const char *p = in ? from + o : reinterpret_cast<const char *>(kZeros);
                __builtin_amdgcn_global_load_lds((global_ptr)p, (lds_ptr)(to + i * 1024), 16, 0, 0);
            }
        }
    };
    f4 acc[MT][NT] = {};
    fetch(0, 0);
    load_scales(0);
    keep_scales(0);
    for (int j = 0; j < blocks; ++j) {
        const char *buf = lds[j % 2];
        // (ahead of the barrier: the run before the last was read up to the block before)
        if (j % kRun == 0 && j > 0) keep_scales(j / kRun);
        __builtin_amdgcn_s_waitcnt(0);  // this wave's loads have landed; the barrier: everyone's
        __syncthreads();
        if (j % kRun == 0) load_scales(j + kRun);
        if (j + 1 < blocks) fetch(j + 1, (j + 1) % 2);
        float s[MT];
        const float s_w = w_scales[j / kRun % 2][j % kRun][wn / 128];
#pragma unroll
        for (int t = 0; t < MT; ++t) s[t] = scales[j / kRun % 2][j % kRun][wm + 16 * t + r16] * s_w;
        const auto operand = [&](int row) {
            const char *at = buf + row * 128;
            return Operand<OUT>(*reinterpret_cast<const i4 *>(at + 16 * (grp ^ row % 8)),
                                *reinterpret_cast<const i4 *>(at + 16 * ((grp + 4) ^ row % 8)));
        };
        Operand<OUT> x[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) x[t] = operand(wm + 16 * t + r16);
        // Column u's products are under way while those of u - 1 are added: an instruction's result takes as
        // long as the next one needs to run, and a wave waits where it asks for it earlier.
        Operand<OUT> w = operand(BM + wn + r16);
        f4 p[MT];
#pragma unroll
        for (int u = 0; u <= NT; ++u) {
            f4 q[MT];
            if (u < NT) {
#pragma unroll
                for (int t = 0; t < MT; ++t) q[t] = block_product(w, x[t]);
                if (u + 1 < NT) w = operand(BM + wn + 16 * (u + 1) + r16);
            }
            if (u > 0)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][u - 1][i] = __builtin_fmaf(p[t][i], s[t], acc[t][u - 1][i]);
            if (u > 0 && u < NT && OUT::bytes == 2)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix instruction,
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // the four sums of an earlier one
                }
            __builtin_amdgcn_sched_barrier(0);  // (or every operand would be read ahead, beyond the registers)
#pragma unroll
            for (int t = 0; t < MT; ++t) p[t] = q[t];
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u)
            store4<OUT>(a, m0 + wm + 16 * t + r16, n0 + wn + 16 * u + 4 * grp, acc[t][u], wide);
}

template <typename OUT>
void launch(const ssm_matmul_fp8_args_t &a, hipStream_t stream) {
    const int blocks = (int)((a.k + 127) / 128);
    const bool wide = a.n % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % (4 * OUT::bytes) == 0;
    // Few rows.  The skinny kernel's time goes by the rounds of its workgroups (16 rows of w each) over the CUs and
    // by its pieces of 16 rows of x, a tile's hardly by either; so it takes over where it has 512 workgroups' work
    // of 32 rows at most.  us, skinny and tiles, bf16 y (fp32: up to a fifth more on either side), K = 2560 (at
    // 1280 and 5120 the same side wins, but for 17 rows of N = 10240, 6.4 and 7.1 at 1280):
    //   N              2560         4096         5120         8192         10240        16384
    //   17 rows     5.6  11.3    5.7  11.3    7.9  11.4    8.0  11.3   11.6  11.5   14.9  13.4
    //   32 rows     6.2  11.3    6.3  11.4   10.0  11.5   10.0  11.4   14.6  11.7   18.4  13.6
    //   33 rows     7.7  11.3    7.7  11.4   12.1  11.5   12.1  11.4   17.6  11.6   22.4  13.5
    //   64 rows     9.3  11.5    9.3  11.6   15.8  11.6   16.0  11.7   23.1  12.0   29.7  13.9
    // and with 1 row of 10240 x 2560 6.4 and 10.9, of 2560 x 5120 6.2 and 19.5 (20 calls in a graph, which w outlasts
    // in the last cache; where it comes from memory a row of 10240 x 2560 takes 7.4 us, 3.5 TB/s of w).
    if (a.m <= 16 || (a.m <= 64 && (a.n + 15) / 16 <= (a.m <= 32 ? 512 : 256))) {
        const unsigned grid = (unsigned)((a.n + 15) / 16), threads = 64 * kSkinnyWaves;
        if (a.m <= 16) skinny_kernel<OUT, 1><<<grid, threads, 0, stream>>>(a, blocks, wide);
        else if (a.m <= 32) skinny_kernel<OUT, 2><<<grid, threads, 0, stream>>>(a, blocks, wide);
        else skinny_kernel<OUT, 4><<<grid, threads, 0, stream>>>(a, blocks, wide);
        return;
    }
    const auto tiles = [&](int64_t bm, int64_t bn) { return ((a.m + bm - 1) / bm) * ((a.n + bn - 1) / bn); };
    // The largest tile that still gives every CU a workgroup.  16384 x 10240 x 2560 in bf16: tiles of 256 473 us
    // (1810 TFLOP/s), of 128 575; 256 x 10240 x 2560: of 64 17.2 us, of 128 21.8; fp32 results, whose widened operands
    // would not fit the registers beside 256 x 256 of sums, stay with 128.
    if (OUT::bytes == 2 && tiles(256, 256) >= 256) {
        if constexpr (OUT::bytes == 2)
            tile_kernel<OUT, 256, 256, 64, 128><<<(unsigned)tiles(256, 256), 512, 0, stream>>>(
                a, blocks, (int)((a.m + 255) / 256), (int)((a.n + 255) / 256), wide);
    } else if (tiles(128, 128) >= 256) {
        tile_kernel<OUT, 128, 128, 64, 64><<<(unsigned)tiles(128, 128), 256, 0, stream>>>(
            a, blocks, (int)((a.m + 127) / 128), (int)((a.n + 127) / 128), wide);
    } else {
        tile_kernel<OUT, 64, 64, 32, 32><<<(unsigned)tiles(64, 64), 256, 0, stream>>>(
            a, blocks, (int)((a.m + 63) / 64), (int)((a.n + 63) / 64), wide);
    }
}

}  // namespace

hipError_t launch_matmul_fp8(const ssm_matmul_fp8_args_t &a, hipStream_t stream) {
    if (a.out_dtype == SSM_BF16)
        launch<io_bf16>(a, stream);
    else
        launch<io_f32>(a, stream);
    return hipGetLastError();
}

}  // namespace ssm
