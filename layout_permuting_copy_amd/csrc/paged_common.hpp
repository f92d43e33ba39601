// Device helpers of the paged key-value cache kernels: cache rows through a block table, lane sums,
// conversions.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.hpp"
#include "paged.hpp"

namespace tc {
namespace dev {

// A sequence's length as the kernels take it: 0 .. most.
__device__ __forceinline__ int paged_len(const int32_t* lens, int b, int most) {
  const int n = lens[b];
  return n < 0 ? 0 : n < most ? n : most;
}

// The page of table entry c of sequence b, or -1 where that names no page of the pool.
__device__ __forceinline__ int paged_page(const PagedTable& t, const PagedPool& p, int b, uint32_t c) {
  const int g = t.p[int64_t(b) * t.sb + int64_t(c) * t.sc];
  return uint32_t(g) < uint32_t(p.pages) ? g : -1;
}

// x of the lane `lane ^ MASK`.
template <int MASK>
__device__ __forceinline__ float lane_xor(float x) {
  return __shfl_xor(x, MASK, 64);
}

}  // namespace dev
}  // namespace tc
