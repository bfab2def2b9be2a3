// column_sum.h -- sums of the columns of a small fp32 matrix [n, cols] of
// partial sums, in a fixed order: the second stage of every gradient that
// sums over tokens.
//
// A workgroup takes 32 columns; 32 groups of lanes take every 32nd row and
// meet in LDS, so that a short chain of loads hides its latency even with
// few columns (512 x 4096: 111 us with one thread a column, 7 us so).  The
// additions are 64-bit: the rows are already sums over many tokens.
#pragma once

#include "sconv_device.h"

namespace sconv {

constexpr int kSumCols = 32, kSumGroups = 32;

template <typename F>
__device__ __forceinline__ void column_sum(const float* partial, int64_t n, int64_t cols, F&& put) {
  __shared__ double part[kSumGroups][kSumCols];
  const int lane = threadIdx.x % kSumCols, group = threadIdx.x / kSumCols;
  const int64_t col = (int64_t)blockIdx.x * kSumCols + lane;
  double acc = 0.0;
  if (col < cols) {
#pragma unroll 4
    for (int64_t r = group; r < n; r += kSumGroups) acc += (double)partial[r * cols + col];
  }
  part[group][lane] = acc;
  __syncthreads();
  if (group != 0 || col >= cols) return;
  acc = 0.0;
#pragma unroll
  for (int g = 0; g < kSumGroups; ++g) acc += part[g][lane];
  put(col, (float)acc);
}

}  // namespace sconv
