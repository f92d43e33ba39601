// Device helpers of the paged key-value cache's and the attention kernels: cache rows through a block table, exchanges
// between lanes, 16- and 8-bit values.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.hpp"
#include "paged.hpp"

namespace tc {
namespace dev {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kInf = __builtin_inff();

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

// A number as it is, but not as known: what derives from it is computed anew, not kept in registers from before.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
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

// Two fp32 values to two of the 16-bit type, nearest even.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (BF16) {
    bf16x2 v;
    v[0] = __bf16(x);
    v[1] = __bf16(y);
    return __builtin_bit_cast(uint32_t, v);
  } else {
    f16x2 v;
    v[0] = _Float16(x);
    v[1] = _Float16(y);
    return __builtin_bit_cast(uint32_t, v);
  }
}
template <bool BF16>
__device__ __forceinline__ float low_half(uint32_t v) {
  if constexpr (BF16) return __builtin_bit_cast(float, v << 16);
  return float(__builtin_bit_cast(f16x2, v)[0]);
}
template <bool BF16>
__device__ __forceinline__ float high_half(uint32_t v) {
  if constexpr (BF16) return __builtin_bit_cast(float, v & 0xffff0000u);
  return float(__builtin_bit_cast(f16x2, v)[1]);
}

// Two e4m3 codes (the low or high half of w) to two values of the 16-bit type: exact in both.
template <bool BF16, bool HIGH>
__device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
  if constexpr (BF16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
}

// The maximum as the exponents' reference, kept finite: exp2(x - reference) is then 0 for x = -infinity and
// infinite for x = +infinity, so a row of nothing sums to 0 and an infinite logit to infinity (its lse; out,
// infinity over infinity, is NaN).
__device__ __forceinline__ float finite(float top) {
  return __builtin_amdgcn_fmed3f(top, -3.4028234664e38f, 3.4028234664e38f);
}

// x of this lane's pair and of the lane 16 (D = 16) or 32 away, in either order: a register swapped with a copy of
// itself by rows or halves.  The copy has to be a register of its own.
template <int D>
__device__ __forceinline__ void partners(float x, float* p, float* q) {
  uint32_t a = __builtin_bit_cast(uint32_t, x), b = a;
  asm("" : "+v"(b));
  if constexpr (D == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0], b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0], b = r[1];
  }
  *p = __builtin_bit_cast(float, a);
  *q = __builtin_bit_cast(float, b);
}
}  // namespace dev
}  // namespace tc
