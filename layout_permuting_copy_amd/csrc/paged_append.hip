// New tokens' keys and values into the pages of a cache, as bits or as 8-bit codes with a scale a row.
#include "paged_common.hpp"

namespace tc {
namespace dev {

constexpr int kAppendThreads = 256;
constexpr int kAppendStarts = 2048;  // token_starts kept in LDS

// Eight 2-byte values at p: one 16-byte load, or element loads where rows are not 16-byte aligned.
template <bool WIDE>
__device__ __forceinline__ u32x4 load8(const unsigned char* p) {
  if constexpr (WIDE) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
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
// 8-bit rows: scale = amax / 448 and code = x / scale, both quotients correctly rounded, so that the codes are
// those of the definition evaluated in fp32; e4m3 rounds to nearest even, and amax / scale stays under
// 448 * (1 + 2^-22), which still rounds to 448.  The magnitudes are compared as integers, where a NaN is above
// infinity.  The row's quotients share their divisor: with r the rounded reciprocal of scale and q = x r, the
// remainder x - q scale (exact in one fused step) gives the correctly rounded q + r (x - q scale) (Markstein
// 1990), 6 operations instead of the division's 11; tiny scales are first multiplied by 2^64 with their x, which
// keeps the remainder exact, and under an infinite scale the quotients are x r.
template <bool BF16, bool E4M3, int LPR>
__device__ __forceinline__ void store_row(const u32x4& v, int c, bool active, unsigned char* dst, float* scale) {
  if constexpr (!E4M3) {
    if (active) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(dst + 16 * c));
  } else {
    float x[8];
    to_f32<BF16>(v, x);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = __builtin_bit_cast(uint32_t, x[i]) & 0x7fffffffu;
      m = m < a ? a : m;
    }
    m = group_max<LPR>(active ? m : 0u);
    float s = __builtin_bit_cast(float, m) / 448.0f;
    if (s < 1.17549435e-38f) s = 1.0f;
    const float up = s < 0x1p-60f ? 0x1p64f : 1.0f, d = s * up, r = 1.0f / d;
    const bool infinite = __builtin_isinf(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = x[i] * up, q = y * r, rest = infinite ? 0.0f : __builtin_fmaf(-q, d, y);
      x[i] = rest == 0.0f ? q : __builtin_fmaf(rest, r, q);  // (an exact quotient keeps its zero's sign)
    }
    int w0 = 0, w1 = 0;
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], w0, false);
    w0 = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w0, true);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], w1, false);
    w1 = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], w1, true);
    if (active) {
      __builtin_nontemporal_store(u32x2{uint32_t(w0), uint32_t(w1)}, reinterpret_cast<u32x2*>(dst + 8 * c));
      if (c == 0) *scale = s;
    }
  }
}

// A workgroup moves kAppendThreads / LPR (token, head) rows; LPR lanes a row, of which head_dim / 8
// move eight values each of the key and of the value (one row a lane: the prompts in 27 us, two 29, four 31).  The rows are
// on their way while the place of each of the workgroup's tokens is found, once for all its heads: its sequence by a
// binary search of token_starts (in LDS where they fit), then length, page, offset.
// Bound: HBM for prompts (16665 tokens of 8 heads of 128: 137 MB in 25.7 us, 5.3 TB/s; new rows are read and cache rows
// written past the caches), the latency of starts -> length -> table -> row otherwise (32 single tokens 2.7 us, 6994
// tokens of 8 heads of 64 to 8 bits 8.3 us).
template <bool BF16, bool E4M3, bool WIDE, int LPR>
__global__ __launch_bounds__(kAppendThreads) void paged_append_kernel(AppendArgs a, Div32 heads) {
  constexpr int ROWS = kAppendThreads / LPR;
  __shared__ int starts[kAppendStarts];
  __shared__ int place_seq[ROWS], place_page[ROWS], place_pos[ROWS];  // page -1: nowhere
  const int tid = threadIdx.x, c = tid % LPR;
  const uint32_t row0 = blockIdx.x * ROWS, t0 = udiv(row0, heads);  // rows count heads within tokens
  const uint32_t row = row0 + tid / LPR, token = udiv(row, heads);
  const int h = int(row - token * heads.d);
  u32x4 k{}, v{};
  if (token < uint32_t(a.tokens) && 8 * c < a.head_dim) {
    k = load8<WIDE>(a.k + int64_t(token) * a.kt + h * a.kh + 16 * c);
    v = load8<WIDE>(a.v + int64_t(token) * a.vt + h * a.vh + 16 * c);
  }
  const PagedPool& p = a.pool;
  const int batch = a.table.batch;
  const bool listed = a.starts && batch < kAppendStarts;
  if (listed) {
    for (int i = tid; i <= batch; i += kAppendThreads) starts[i] = a.starts[i];
    __syncthreads();
  }
  // the workgroup's tokens, at most ROWS (one head) of them
  static_assert(ROWS <= kAppendThreads);
  if (tid < ROWS) {
    const uint32_t t = t0 + tid;
    int b = int(t), pos = -1, page = -1;
    const auto length = [&](int of) {
      const int n = a.lens[of];
      return n < 0 ? 0 : n;
    };
    if (t < uint32_t(a.tokens) && t <= udiv(row0 + ROWS - 1, heads)) {
      if (!a.starts) {
        pos = length(b) - 1;
      } else {
        // the last b with starts[b] <= t
        int lo = 0, hi = batch;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if ((listed ? starts[mid] : a.starts[mid]) <= int(t)) lo = mid; else hi = mid;
        }
        b = lo;
        const int first = listed ? starts[b] : a.starts[b], end = listed ? starts[b + 1] : a.starts[b + 1];
        if (first <= int(t) && int(t) < end) pos = length(b) - (end - int(t));
      }
      if (pos >= 0) {
        const uint32_t col = udiv(uint32_t(pos), p.div);
        if (col < uint32_t(a.table.cols)) page = paged_page(a.table, p, b, col);
      }
    }
    place_seq[tid] = b;
    place_page[tid] = page;
    place_pos[tid] = pos;
  }
  __syncthreads();
  const int at = int(token - t0), b = place_seq[at], page = place_page[at], pos = place_pos[at];
  const bool out = page >= 0 && 8 * c < a.head_dim;
  unsigned char* kd = nullptr;
  unsigned char* vd = nullptr;
  float *ks = nullptr, *vs = nullptr;
  if (out) {
    const uint32_t r = uint32_t(pos) - udiv(uint32_t(pos), p.div) * p.div.d;
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
int launch(const AppendArgs& a, hipStream_t s) {
  const int64_t per = kAppendThreads / LPR;
  const int64_t wgs = (a.tokens * a.heads + per - 1) / per;
  if (!launchable(wgs, kAppendThreads)) return TC_E_RANGE;
  hipLaunchKernelGGL((paged_append_kernel<BF16, E4M3, WIDE, LPR>), dim3(uint32_t(wgs)), dim3(kAppendThreads), 0, s, a,
                     make_div32(uint32_t(a.heads)));
  return TC_OK;
}

template <bool BF16, bool E4M3, bool WIDE>
int by_lanes(const AppendArgs& a, hipStream_t s) {
  const int lanes = a.head_dim / 8;
  if (lanes <= 2) return launch<BF16, E4M3, WIDE, 2>(a, s);
  if (lanes <= 4) return launch<BF16, E4M3, WIDE, 4>(a, s);
  if (lanes <= 8) return launch<BF16, E4M3, WIDE, 8>(a, s);
  if (lanes <= 16) return launch<BF16, E4M3, WIDE, 16>(a, s);
  return launch<BF16, E4M3, WIDE, 32>(a, s);
}

template <bool E4M3>
int by_type(const AppendArgs& a, int dtype, bool wide, hipStream_t s) {
  if constexpr (!E4M3) return wide ? by_lanes<true, E4M3, true>(a, s) : by_lanes<true, E4M3, false>(a, s);  // bits either way
  else if (dtype == TC_BF16) return wide ? by_lanes<true, E4M3, true>(a, s) : by_lanes<true, E4M3, false>(a, s);
  else return wide ? by_lanes<false, E4M3, true>(a, s) : by_lanes<false, E4M3, false>(a, s);
}

}  // namespace dev

int launch_paged_append(const AppendArgs& a, int dtype, int cache_dtype, bool wide, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (a.tokens * a.heads > (int64_t(1) << 30)) return TC_E_RANGE;
  return cache_dtype == TC_E4M3 ? dev::by_type<true>(a, dtype, wide, s) : dev::by_type<false>(a, dtype, wide, s);
}

}  // namespace tc
