// Sums over rows of partial results, the last step of the parameters'
// gradients of the backward calls around the scan: out[j][c] = sum of
// part[row][j][c].  A workgroup takes 64 columns of one j, its 16 wavefronts
// every sixteenth row each, joined in wavefront order: the same order on every
// call, no atomics.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "block_internal.h"
#include "lane_ops.h"

namespace ssm {
namespace {

constexpr int kCols = 64, kWaves = 16;

__global__ __launch_bounds__(kCols * kWaves) void column_sums(ColumnSums a, int64_t first) {
    __shared__ float s[kWaves][kCols];
    const int lane = threadIdx.x % kCols, wave = threadIdx.x / kCols;
    const int64_t c = first + (int64_t)blockIdx.x * kCols + lane;
    const int j = blockIdx.y;
    float sum = 0.0f;
    if (c < a.D) {
        const float* p = a.part + j * a.D + c;
        const int64_t step = a.m * a.D;
#pragma unroll 8
        for (int64_t r = wave; r < a.n; r += kWaves) sum += p[r * step];
    }
    s[wave][lane] = sum;
    lds_barrier();
    if (wave == 0 && c < a.D) {
        sum = s[0][lane];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) sum += s[k][lane];
        if (a.strided) {
            const int K = a.m - 1;
            if (j < K) a.out[0][c * K + j] = sum;
            else if (a.out[1]) a.out[1][c] = sum;
        } else if (float* out = j == 0 ? a.out[0] : (j == 1 ? a.out[1] : a.out[2])) {
            if (j == 0 && a.divide) {
                const float by = a.divide[c];
                sum = by != 0.0f ? sum / by : 0.0f;
            }
            out[c] = sum;
        }
    }
}

}  // namespace

hipError_t launch_column_sums(const ColumnSums& a, hipStream_t stream) {
    return in_slices((a.D + kCols - 1) / kCols, kMaxItems / (kCols * kWaves), [&](int64_t first, int64_t n) {
        column_sums<<<dim3((unsigned)n, (unsigned)a.m), kCols * kWaves, 0, stream>>>(a, first * kCols);
        return hipGetLastError();
    });
}

}  // namespace ssm
