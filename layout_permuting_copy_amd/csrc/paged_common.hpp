// Device helpers of the paged key-value cache kernels: cache rows through a block table, exchanges between
// lanes.
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

// A lane exchange by DPP: x of the lane that CTRL names; lanes that get none, or that the row mask leaves out, have 0.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CTRL, ROWS, 0xf, ROWS == 0xf));
}

// The inclusive sum over the lanes up to this one: within rows of 16 by shifts of 1, 2, 4 and 8, then each row's
// last sum added to the rows above it.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x += dpp<0x111>(x);
  x += dpp<0x112>(x);
  x += dpp<0x114>(x);
  x += dpp<0x118>(x);
  x += dpp<0x142, 0xa>(x);
  x += dpp<0x143, 0xc>(x);
  return x;
}

// The greatest of N neighbouring lanes' x (N = 2 .. 32, a power of two), in each of them: swaps within four lanes, then
// mirrors of 8 and 16 (whose halves hold equal values by then).
template <int N>
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
  const auto take = [&](uint32_t o) { x = x < o ? o : x; };
  if constexpr (N >= 2) take(dpp<0xb1>(x));   // quad: 1 0 3 2
  if constexpr (N >= 4) take(dpp<0x4e>(x));   // quad: 2 3 0 1
  if constexpr (N >= 8) take(dpp<0x141>(x));  // half row mirrored
  if constexpr (N >= 16) take(dpp<0x140>(x)); // row mirrored
  if constexpr (N >= 32) take(__shfl_xor(x, 16, 64));
  return x;
}

}  // namespace dev
}  // namespace tc
