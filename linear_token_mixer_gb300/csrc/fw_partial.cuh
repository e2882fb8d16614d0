// fw_partial.cuh -- the sum of partial rows [slices][count] that the blocks of a launch before have written,
// column by column in an order that does not depend on which block wrote first.
#pragma once

#include "fw_decay.cuh"

namespace fw {

// A block: 32 columns by 32 shares of the slices, each share added in order, then the shares in order.
constexpr int kSumCols = 32, kSumShares = 32;

// put(i, z) with the sum z of column i.
template <typename F> __device__ __forceinline__ void sum_slices(const float *ws, int slices, int64_t count, F put) {
    __shared__ float part[kSumShares][kSumCols + 1];
    const int c = threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
    const int64_t i = (int64_t)blockIdx.x * kSumCols + c;
    float z = 0.f;
    if (i < count)
#pragma unroll 8
        for (int s = r; s < slices; s += kSumShares) z += ws[(int64_t)s * count + i];
    part[r][c] = z;
    __syncthreads();
    if (r != 0 || i >= count) return;
    z = 0.f;
#pragma unroll
    for (int k = 0; k < kSumShares; ++k) z += part[k][c];
    put(i, z);
}

inline dim3 sum_grid(int64_t count) { return dim3((unsigned)((count + kSumCols - 1) / kSumCols)); }

}  // namespace fw
