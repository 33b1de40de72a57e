// colsum.h -- sums down the rows of a table of partial sums, in a fixed order.
#pragma once

#include "device_math.h"

namespace mscan {

// Where a column's sums go (either pointer may be null).
struct ColStore {
  float *first, *second;
  __device__ __forceinline__ void operator()(int c, float s) const {
    if (first) first[c] = s;
  }
  __device__ __forceinline__ void operator()(int c, float2 s) const {
    if (first) first[c] = s.x;
    if (second) second[c] = s.y;
  }
};

__device__ __forceinline__ void col_add(float& a, float b) { a += b; }
__device__ __forceinline__ void col_add(float2& a, float2 b) { a.x += b.x, a.y += b.y; }

// 16 columns a workgroup, 64 threads down the rows of each: at the usual 1000
// to 2000 rows a thread has some 20 loads, and a few hundred columns are enough
// for dozens of workgroups (64 columns and 16 threads each took 8.5 us for 1024
// rows of 192 columns, this 4.8).
template <typename S, typename F>
__global__ void __launch_bounds__(1024) colsum_kernel(const S* part, int64_t rows, int cols, F store) {
  __shared__ S acc[64][17];
  const int c = threadIdx.x & 15, t = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  S s{};
  if (col < cols) {
#pragma unroll 8
    for (int64_t k = t; k < rows; k += 64) col_add(s, part[k * cols + col]);
  }
  acc[t][c] = s;
  __syncthreads();
  if (t < 8) {  // eight sums of eight, then one of eight
    s = acc[t * 8][c];
#pragma unroll
    for (int k = 1; k < 8; ++k) col_add(s, acc[t * 8 + k][c]);
  }
  __syncthreads();
  if (t < 8) acc[t][c] = s;
  __syncthreads();
  if (t == 0 && col < cols) {
#pragma unroll
    for (int k = 1; k < 8; ++k) col_add(s, acc[k][c]);
    store(col, s);
  }
}

}  // namespace mscan
