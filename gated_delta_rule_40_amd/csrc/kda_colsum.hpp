// kda_colsum.hpp -- column sums of partial results [n][cols], in a fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// A workgroup sums COLSUM_COLS columns (64 bytes of a row) by COLSUM_WALKS
// strided walks each; the walks' sums are added in two steps of eight.
constexpr int COLSUM_COLS = 16, COLSUM_WALKS = 64, COLSUM_THREADS = COLSUM_COLS * COLSUM_WALKS;

// The sum of column i, in the first COLSUM_COLS threads.
__device__ __forceinline__ float column_sum(const float *src, int32_t n, int64_t cols, int64_t i)
{
    __shared__ float part[COLSUM_WALKS][COLSUM_COLS + 1];
    const int c = threadIdx.x % COLSUM_COLS, walk = threadIdx.x / COLSUM_COLS;
    float s = 0.f;
    if (i < cols)
#pragma unroll 8
        for (int32_t r = walk; r < n; r += COLSUM_WALKS) s += src[r * cols + i];
    part[walk][c] = s;
    __syncthreads();
    if (walk < 8) {
#pragma unroll
        for (int v = 1; v < 8; ++v) s += part[walk + 8 * v][c];
    }
    __syncthreads();
    if (walk < 8) part[walk][c] = s;
    __syncthreads();
    if (walk == 0) {
#pragma unroll
        for (int v = 1; v < 8; ++v) s += part[v][c];
    }
    return s;
}

}  // namespace kda
