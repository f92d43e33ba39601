// New tokens' keys and values into the pages of a cache, as bits or as 8-bit codes with a scale a row.
#include "paged_common.hpp"

namespace tc {
namespace dev {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kAppendThreads = 256;

// Eight 2-byte values at p: one 16-byte load, or element loads where rows are not 16-byte aligned.
template <bool WIDE>
__device__ __forceinline__ u32x4 load8(const unsigned char* p) {
  if constexpr (WIDE) return *reinterpret_cast<const u32x4*>(p);
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = uint32_t(h[2 * i]) | uint32_t(h[2 * i + 1]) << 16;
  return v;
}

template <bool BF16>
__device__ __forceinline__ void to_f32(const u32x4& v, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[2 * i] = __builtin_bit_cast(float, v[i] << 16);
      x[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xffff0000u);
    } else {
      x[2 * i] = float(__builtin_bit_cast(_Float16, uint16_t(v[i])));
      x[2 * i + 1] = float(__builtin_bit_cast(_Float16, uint16_t(v[i] >> 16)));
    }
  }
}

// One row of new values into the pool: `v` are the lane's eight values at element 8 * c of the row
// (active lanes), `dst` the row, `scale` its scale.  A row's lanes are LPR neighbours.
//
// 8-bit rows: scale = amax / 448 and code = x / scale, both divisions correctly rounded, so that the
// codes are those of the definition evaluated in fp32; e4m3 rounds to nearest even, and amax / scale
// stays under 448 * (1 + 2^-22), which still rounds to 448.
template <bool BF16, bool E4M3, int LPR>
__device__ __forceinline__ void store_row(const u32x4& v, int c, bool active, unsigned char* dst, float* scale) {
  if constexpr (!E4M3) {
    if (active) *reinterpret_cast<u32x4*>(dst + 16 * c) = v;
  } else {
    float x[8], m = 0.0f;
    to_f32<BF16>(v, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = __builtin_fabsf(x[i]);
      m = m < a || a != a ? a : m;  // a NaN stays: nothing compares with it
    }
    if (!active) m = 0.0f;
#pragma unroll
    for (int d = 1; d < LPR; d *= 2) {
      const float o = __shfl_xor(m, d, 64);
      m = m < o || o != o ? o : m;
    }
    float s = m / 448.0f;
    if (s < 1.17549435e-38f) s = 1.0f;
    int w0 = 0, w1 = 0;
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] / s, x[1] / s, w0, false);
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] / s, x[3] / s, w0, true);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] / s, x[5] / s, w1, false);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] / s, x[7] / s, w1, true);
    if (active) {
      *reinterpret_cast<u32x2*>(dst + 8 * c) = u32x2{uint32_t(w0), uint32_t(w1)};
      if (c == 0) *scale = s;
    }
  }
}

// Lanes: LPR a (token, head) row, of which head_dim / 8 move eight values each of the key and of the value.
// Every lane stays to the end: the row maximum and the search below are exchanges between lanes.
// Bound: HBM for prompts, the latency of length -> table -> row for single tokens.
template <bool BF16, bool E4M3, bool WIDE, int LPR>
__global__ __launch_bounds__(kAppendThreads) void paged_append_kernel(AppendArgs a, Div32 heads) {
  constexpr int RPW = 64 / LPR;  // rows a wave
  const int lane = threadIdx.x & 63, c = lane % LPR;
  const uint32_t row = (blockIdx.x * (kAppendThreads / 64) + threadIdx.x / 64) * RPW + lane / LPR;
  const uint32_t t = udiv(row, heads);  // rows count heads within tokens; the host keeps them under 2^31
  const int h = int(row - t * heads.d);
  const bool mine = t < uint32_t(a.tokens);
  const bool active = mine && 8 * c < a.head_dim;
  u32x4 k = {}, v = {};
  if (active) {
    k = load8<WIDE>(a.k + int64_t(t) * a.kt + h * a.kh + 16 * c);
    v = load8<WIDE>(a.v + int64_t(t) * a.vt + h * a.vh + 16 * c);
  }
  int b = int(t), pos = -1;
  if (!a.starts) {
    if (mine) pos = a.lens[b] - 1;
  } else {
    // b = how many of starts[1 .. batch] are <= t, counted 64 at a time by the wave for each of its tokens
    b = 0;
    for (int base = 0; base < a.table.batch; base += 64) {
      const int s = base + lane < a.table.batch ? a.starts[base + lane + 1] : 0x7fffffff;
      int last = 0;
#pragma unroll
      for (int r = 0; r < RPW; ++r) {
        const int tr = __builtin_amdgcn_readlane(int(mine ? t : a.tokens - 1), r * LPR);
        const int n = __popcll(__ballot(s <= tr));
        if (lane / LPR == r) b += n;
        last = n;
      }
      if (last < 64) break;  // the wave's last token lies before a later sequence
    }
    if (mine && b < a.table.batch) {
      const int first = a.starts[b], end = a.starts[b + 1];
      if (first <= int(t) && int(t) < end) pos = a.lens[b] - (end - int(t));
    }
  }
  int page = -1;
  uint32_t r = 0;
  if (pos >= 0) {
    const uint32_t col = udiv(uint32_t(pos), a.pool.div);
    r = uint32_t(pos) - col * a.pool.div.d;
    if (col < uint32_t(a.table.cols)) page = paged_page(a.table, a.pool, b, col);
  }
  const bool out = active && page >= 0;
  const PagedPool& p = a.pool;
  unsigned char* kd = nullptr;
  unsigned char* vd = nullptr;
  float *ks = nullptr, *vs = nullptr;
  if (out) {
    kd = p.k + page * p.kp + r * p.kr + h * p.kh;
    vd = p.v + page * p.vp + r * p.vr + h * p.vh;
    if constexpr (E4M3) {
      ks = p.ks + page * p.ksp + r * p.ksr + h * p.ksh;
      vs = p.vs + page * p.vsp + r * p.vsr + h * p.vsh;
    }
    if (a.weights && c == 0 && pos < a.w.cols) a.weights[b * a.w.sb + h * a.w.sh + pos * a.w.sc] = 0.0f;
  }
  store_row<BF16, E4M3, LPR>(k, c, out, kd, ks);
  store_row<BF16, E4M3, LPR>(v, c, out, vd, vs);
}

template <bool BF16, bool E4M3, bool WIDE, int LPR>
void launch(const AppendArgs& a, hipStream_t s) {
  const int64_t per = kAppendThreads / LPR;
  const int64_t wgs = (a.tokens * a.heads + per - 1) / per;
  hipLaunchKernelGGL((paged_append_kernel<BF16, E4M3, WIDE, LPR>), dim3(uint32_t(wgs)), dim3(kAppendThreads), 0, s, a,
                     make_div32(uint32_t(a.heads)));
}

template <bool BF16, bool E4M3, bool WIDE>
void by_lanes(const AppendArgs& a, hipStream_t s) {
  const int lanes = a.head_dim / 8;
  if (lanes <= 2) return launch<BF16, E4M3, WIDE, 2>(a, s);
  if (lanes <= 4) return launch<BF16, E4M3, WIDE, 4>(a, s);
  if (lanes <= 8) return launch<BF16, E4M3, WIDE, 8>(a, s);
  if (lanes <= 16) return launch<BF16, E4M3, WIDE, 16>(a, s);
  return launch<BF16, E4M3, WIDE, 32>(a, s);
}

template <bool E4M3>
void by_type(const AppendArgs& a, int dtype, bool wide, hipStream_t s) {
  if constexpr (!E4M3) return wide ? by_lanes<true, E4M3, true>(a, s) : by_lanes<true, E4M3, false>(a, s);  // bits either way
  else if (dtype == TC_BF16) return wide ? by_lanes<true, E4M3, true>(a, s) : by_lanes<true, E4M3, false>(a, s);
  else return wide ? by_lanes<false, E4M3, true>(a, s) : by_lanes<false, E4M3, false>(a, s);
}

}  // namespace dev

int launch_paged_append(const AppendArgs& a, int dtype, int cache_dtype, bool wide, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (a.tokens * a.heads > (int64_t(1) << 30)) return TC_E_RANGE;
  if (cache_dtype == TC_E4M3)
    dev::by_type<true>(a, dtype, wide, s);
  else
    dev::by_type<false>(a, dtype, wide, s);
  return TC_OK;
}

}  // namespace tc
