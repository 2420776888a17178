// The rows of an expert's run in the sorted order, for the kernels and for the host. Counts, alignments and rows are each below 2^31
// (the C entry checks them); a sum of two of them is not an int.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace nvfp4 {

// `count` up to a multiple of `align`; the caller's rows hold the result, so it is below 2^31 again.
__host__ __device__ __forceinline__ int padded_run(int count, int align) {
  const uint32_t a = (uint32_t)align;
  return (int)(((uint32_t)count + (a - 1)) / a * a);
}

// f(r) for one of 64 lanes' rows of [first, end): first + lane, and every 64th from there.
template <class F>
__host__ __device__ __forceinline__ void each_64th(int first, int end, int lane, F&& f) {
  for (int64_t r = (int64_t)first + lane; r < end; r += 64) f(r);
}

}  // namespace nvfp4
