// wide_grid.h -- launches of more workgroups than one axis of a grid holds: an
// axis may not have 2^32 threads or more (2^23 workgroups of 512), so the rest
// goes to the second one.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mscan {

// A grid of n workgroups or, past one axis, up to 2^20 - 1 more, which return at once.
inline dim3 wide_grid(int64_t n) {
  constexpr int64_t kAxis = 1 << 20;  // of up to 1024 threads
  return n <= kAxis ? dim3((unsigned)n) : dim3((unsigned)kAxis, (unsigned)((n + kAxis - 1) / kAxis));
}
__device__ __forceinline__ int64_t wide_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

}  // namespace mscan
