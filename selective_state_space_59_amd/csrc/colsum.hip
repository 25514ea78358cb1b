// colsum.hip -- sums over the rows of fp32 partial results, part[k][n][D] -> out_k[D], for the
// gradients of per-channel vectors on gfx950.
//
// The partial rows are few and small beside the pass that wrote them; they are added in a fixed
// order (no atomics), at most 64 in a row per lane, in stages of 256 rows while there are many.
#include <algorithm>

#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr int kStageRows = 256;  // partial rows of a workgroup in a stage
constexpr int kLastRows = 1024;  // most rows of the last stage

struct Outs {
    float *p[3];
};

// Threads: 64 columns x LANES row lanes.  blockIdx: (column block, row chunk, k).
template <int LANES>
__global__ __launch_bounds__(64 * LANES) void colsum_kernel(const float *part, int64_t n, int64_t D, int rows,
                                                            Outs out) {
    __shared__ float s[LANES][64];
    const int c = threadIdx.x & 63, lane = threadIdx.x >> 6, k = blockIdx.z;
    if (!out.p[k]) return;
    const int64_t d = (int64_t)blockIdx.x * 64 + c, lo = (int64_t)blockIdx.y * rows, hi = lo + rows < n ? lo + rows : n;
    float v = 0.0f;
    if (d < D) {
        const float *p = part + (int64_t)k * n * D + d;
#pragma unroll 8
        for (int64_t i = lo + lane; i < hi; i += LANES) v += p[i * D];
    }
    s[lane][c] = v;
    __syncthreads();
    if (lane == 0 && d < D) {
        for (int i = 1; i < LANES; ++i) v += s[i][c];
        out.p[k][(int64_t)blockIdx.y * D + d] = v;
    }
}

}  // namespace

size_t column_sums_scratch_bytes(int64_t n, int64_t D, int K) {
    size_t b = 0;
    while (n > kLastRows) {
        n = (n + kStageRows - 1) / kStageRows;
        b += (size_t)(n * D * K) * 4;
    }
    return (b + 255) & ~(size_t)255;
}

hipError_t launch_column_sums(const float *part, int64_t n, int64_t D, int K, float *const out[], float *scratch,
                              hipStream_t stream) {
    const unsigned cols = (unsigned)((D + 63) / 64);
    while (n > kLastRows) {
        const int64_t chunks = (n + kStageRows - 1) / kStageRows;
        Outs o = {};
        for (int k = 0; k < K; ++k) o.p[k] = out[k] ? scratch + (int64_t)k * chunks * D : nullptr;
        colsum_kernel<4><<<dim3(cols, (unsigned)chunks, (unsigned)K), 256, 0, stream>>>(part, n, D, kStageRows, o);
        part = scratch;
        scratch += chunks * D * K;
        n = chunks;
    }
    Outs o = {};
    for (int k = 0; k < K; ++k) o.p[k] = out[k];
    colsum_kernel<16><<<dim3(cols, 1, (unsigned)K), 1024, 0, stream>>>(part, n, D, kLastRows, o);
    return hipGetLastError();
}

}  // namespace ssm
