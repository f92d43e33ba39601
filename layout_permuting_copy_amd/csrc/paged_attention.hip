// Attention of one new token a sequence over a paged cache, split over the cache's length and joined.
#include <algorithm>
#include <type_traits>

#include "paged_common.hpp"

namespace tc {
namespace dev {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = 4;
constexpr int kTile = 32;                       // cache rows a wave takes at a time
constexpr int kStep = kTile * kAttnWaves;       // and a workgroup
constexpr int kJoinThreads = 512;
constexpr int kCus = 256;
constexpr float kInf = __builtin_inff();

// Cache bytes: an address whose kind the compiler need not find out.
typedef const __attribute__((address_space(1))) unsigned char* global_bytes;
template <int N, bool STREAM>
__device__ __forceinline__ void load_cache(global_bytes p, uint32_t* w) {
  typedef typename Bytes<N>::T T;
  typedef const __attribute__((address_space(1))) T* P;
  const T v = STREAM ? __builtin_nontemporal_load((P)p) : *(P)p;
  if constexpr (N == 4)
    w[0] = v;
  else
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = v[i];
}

// D = A B + C on 16 x 16 tiles with a contraction of 32.  Lane l (r = l % 16, g = l / 16) holds row r
// of A and column r of B at contraction indices 8 g .. 8 g + 7, and column r of C and D at rows 4 g .. 4 g + 3.
template <bool BF16>
__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
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

// How the call's work is cut: a sequence of n rows has max(1, ceil(n / unit_rows)) units for each of
// its `pairs` (cache heads times tiles of query heads); all units in a row, sequence after sequence and
// pair after pair, are dealt to the workgroups in equal runs (the first `rest` of them one longer).
// A pair that lies in one run is finished by its workgroup; one that is cut leaves partial results, in
// slot 0 of a workgroup whose run starts with it and slot 1 of one whose run ends in it.
struct Cut {
  uint32_t wgs, each, rest;  // workgroups that get units
  __device__ __forceinline__ uint32_t start(uint32_t i) const { return i * each + (i < rest ? i : rest); }
  __device__ __forceinline__ uint32_t owner(uint32_t x) const {
    const uint32_t longer = rest * (each + 1);
    return x < longer ? x / (each + 1) : rest + (x - longer) / each;
  }
};

struct Walk {
  uint32_t total;   // units of all sequences, for one pair
  uint32_t before;  // of the lane's sequences' predecessors
  int per;          // sequences a lane sums: lane * per .. lane * per + per - 1
};

__device__ __forceinline__ uint32_t units_of(int n, const Div32& unit) {
  const uint32_t u = udiv(uint32_t(n) + unit.d - 1, unit);
  return u ? u : 1;
}

// Every wave for itself: the lengths' units summed over the lanes.
__device__ __forceinline__ Walk walk_lengths(const AttentionArgs& a) {
  const int lane = threadIdx.x & 63;
  Walk w;
  w.per = (a.table.batch + 63) / 64;
  uint32_t sum = 0;
  for (int k = 0; k < w.per; ++k) {
    const int b = lane * w.per + k;
    if (b < a.table.batch) sum += units_of(paged_len(a.lens, b, a.max_len), a.unit);
  }
  uint32_t upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(upto, d, 64);
    if (lane >= d) upto += o;
  }
  w.total = uint32_t(__builtin_amdgcn_readlane(int(upto), 63));
  w.before = upto - sum;
  return w;
}

__device__ __forceinline__ Cut cut_of(uint32_t units, uint32_t most, uint32_t least_each) {
  Cut c;
  c.wgs = (units + least_each - 1) / least_each;
  c.wgs = c.wgs < most ? c.wgs : most;
  c.each = units / c.wgs;
  c.rest = units - c.each * c.wgs;
  return c;
}

// A run of units: up to 16 * HT query heads of one cache head over rows of one sequence, then of the
// next.  The workgroup's four waves take tiles of 32 rows in turn, each with its own running maximum, sum
// and output (one pass over the cache), and meet once at the end of a segment.  A wave needs neither LDS
// nor a barrier in its loop:
//
//   S^T = K Q^T    rows of A are cache rows: lane (r, g) loads 16 bytes of row r straight into A's
//                  layout; Q^T stays in registers.
//   O^T = V^T P^T  S^T leaves lane (r, g) with head r and rows 4 g .. 4 g + 3 of each 16-row half, which is
//                  B's layout if the contraction index 8 g + j stands for row 4 g + j of the first half
//                  (j < 4) or 4 g + j - 4 of the second: the softmax's output feeds the product as it is.
//                  For V^T lane (r, g) loads, of those eight rows, the same DP / 16 neighbouring
//                  elements (16 lanes: a whole row) and regroups them by byte permutes.
//
// P is held as the sum of two 16-bit values (its rounding and the rest), two products each: the matrix
// cores are idle nine cycles in ten here, and out is then as exact as fp32 sums of fp32 weights.
// 8-bit rows become 16-bit values in registers (exactly); the key's scale multiplies its row's
// logits, the value's its row's weights.
//
// The next tile's keys are requested once this tile's logits are formed, its values once this tile's are
// used, the pages of the one after next before both, so a wave always has loads in flight.  No load of the
// cache is conditional: rows past the end and rows on no page are read from wherever their index leads inside
// the pool (page 0 for no page), and what comes back is masked, in the tiles that have such rows.
//
// DP: head_dim rounded up to 64, 128 or 256.  FULL: head_dim is DP; else the key elements past it
// are cleared (those of Q are, but 0 times infinity is not 0) and the output elements past it not
// stored.  PAGE16: pages of a multiple of 16 rows, so that a 16-row half lies on one page and its address
// is scalar; otherwise each lane finds its rows.
//
// Bound: HBM (a cache row is read once for all heads of its group).
template <bool BF16, bool E4M3, int DP, int HT, bool PAGE16, bool FULL>
struct Attend {
  static constexpr bool VBF = BF16 || E4M3;       // type of the second product
  static constexpr int EB = E4M3 ? 1 : 2;
  static constexpr int KS = DP / 32;              // contraction steps of the first product
  static constexpr int KC = DP * EB / 64;         // 16-byte chunks a lane loads of a key row
  static constexpr int VF = DP / 16;              // elements a lane loads of a value row: tiles of O^T
  static constexpr int VB = VF * EB;              // their bytes: 4, 8, 16 or 32
  static constexpr int VP = VB == 32 ? 16 : VB;   // bytes a load
  static constexpr int VW = VB / 4;

  // The element of Q that contraction index (step s, group g, j) stands for.
  static __device__ __forceinline__ int q_element(int s, int g, int j) {
    if constexpr (E4M3) return ((s >> 1) * 4 + g) * 16 + (s & 1) * 8 + j;
    return s * 32 + g * 8 + j;
  }
  // The element of row r of tile f of O^T (VB = 32: two halves, so that a load covers whole lines).
  static __device__ __forceinline__ int v_element(int r, int f) {
    if constexpr (VB == 32) return (f >> 3) * (DP / 2) + r * 8 + (f & 7);
    return r * VF + f;
  }

  struct Keys {
    u32x4 x[2][KC];  // rows r of both halves
    float scale;     // of the tile's row lane % 32
  };
  struct Values {
    uint32_t x[8][VW];  // rows 4 g + j of both halves
    float scale;
  };

  int lane, r, g;
  // the segment's pools from its cache head on, its row of the block table; strides
  const unsigned char* k0;
  const unsigned char* v0;
  const float* ks0;
  const float* vs0;
  const int32_t* table;
  int64_t kp, kr, vp, vr, ksp, ksr, vsp, vsr, sc;
  int pool_pages;
  Div32 div;
  int key_bytes;  // of a row
  // the lane's byte offsets.  PAGE16: in the 16 rows of a half, of key row r and value row 4 g; otherwise in a row.
  // Both include the lane's chunk (of a value row past head_dim: the row's first)
  uint32_t kchunk, krow, vrow, vrow2;

  __device__ __forceinline__ void pools(const AttentionArgs& a, int b, int h) {
    const PagedPool& p = a.pool;
    k0 = p.k + h * p.kh;
    v0 = p.v + h * p.vh;
    if constexpr (E4M3) {
      ks0 = p.ks + h * p.ksh;
      vs0 = p.vs + h * p.vsh;
    }
    table = a.table.p + b * a.table.sb;
  }
  __device__ __forceinline__ void init(const AttentionArgs& a) {
    const PagedPool& p = a.pool;
    kp = p.kp, kr = p.kr, vp = p.vp, vr = p.vr;
    if constexpr (E4M3) ksp = p.ksp, ksr = p.ksr, vsp = p.vsp, vsr = p.vsr;
    sc = a.table.sc;
    pool_pages = p.pages;
    div = p.div;
    key_bytes = a.head_dim * EB;
    const int e0 = v_element(r, 0), e1 = e0 + DP / 2;
    kchunk = uint32_t(16 * g);
    vrow = FULL || e0 < a.head_dim ? uint32_t(e0 * EB) : 0u;
    vrow2 = FULL || e1 < a.head_dim ? uint32_t(e1 * EB) : 0u;
    if constexpr (PAGE16) {
      krow = uint32_t(r) * uint32_t(kr) + kchunk;
      vrow += uint32_t(4 * g) * uint32_t(vr);
      vrow2 += uint32_t(4 * g) * uint32_t(vr);
    }
  }

  // The table's entry for the tile's row lane % 32 (past the segment: for its last row).
  __device__ __forceinline__ int load_pages(int t, int t1) const {
    const int at = t + (lane & 31);
    return table[int64_t(udiv(uint32_t(at < t1 ? at : t1 - 1), div)) * sc];
  }
  // Bit i: the tile's row i % 32 does not exist (past the end, on no page).
  __device__ __forceinline__ uint64_t missing_rows(int entry, int t, int t1) const {
    return __ballot(t + (lane & 31) >= t1 || uint32_t(entry) >= uint32_t(pool_pages));
  }
  __device__ __forceinline__ uint32_t row_in_page(int at) const {
    return uint32_t(at) - udiv(uint32_t(at), div) * div.d;
  }
  // A scalar address as it is: the compiler would add the lane's offset to some common part of it ahead of time,
  // in vector registers; the load instruction takes both.
  static __device__ __forceinline__ global_bytes scalar(const unsigned char* p) {
    global_bytes q = (global_bytes)p;
    asm("" : "+s"(q));
    return q;
  }
  // No load depends on a condition: `entry` past the pool (no page) is taken as page 0, rows past the
  // end lie on their page all the same.
  __device__ __forceinline__ int page_of(int entry) const { return uint32_t(entry) < uint32_t(pool_pages) ? entry : 0; }

  __device__ __forceinline__ void load_keys(int entry, int t, Keys& k) const {
    const int pages = page_of(entry);
    const uint32_t mine = PAGE16 ? krow : kchunk;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      global_bytes row;
      if constexpr (PAGE16)
        row = scalar(k0 + (__builtin_amdgcn_readlane(pages, 16 * u) * kp + row_in_page(t + 16 * u) * kr));
      else
        row = (global_bytes)(k0 + (__shfl(pages, 16 * u + r, 64) * kp + row_in_page(t + 16 * u + r) * kr));
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        uint32_t* x = reinterpret_cast<uint32_t*>(&k.x[u][c]);
        if constexpr (FULL)
          load_cache<16, false>(row + mine + 64 * c, x);
        else
          load_cache<16, false>(row + (mine + (64 * c + 16 * g < key_bytes ? 64 * c : -16 * g)), x);
      }
    }
    if constexpr (E4M3) k.scale = ks0[pages * ksp + row_in_page(t + (lane & 31)) * ksr];
  }

  // Values are read past the caches: nothing else needs their lines (keys are not, as a line of a
  // key row is covered by two loads).
  __device__ __forceinline__ void load_values(int entry, int t, Values& v) const {
    const int pages = page_of(entry);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const unsigned char* half = nullptr;
      if constexpr (PAGE16) half = v0 + (__builtin_amdgcn_readlane(pages, 16 * u) * vp + row_in_page(t + 16 * u) * vr);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        global_bytes row;
        if constexpr (PAGE16) {
          row = scalar(half + j * vr);
        } else {
          const int i = 16 * u + 4 * g + j;
          row = (global_bytes)(v0 + (__shfl(pages, i, 64) * vp + row_in_page(t + i) * vr));
        }
        load_cache<VP, true>(row + vrow, v.x[4 * u + j]);
        if constexpr (VB == 32) load_cache<VP, true>(FULL ? row + vrow + DP / 2 * EB : row + vrow2, v.x[4 * u + j] + 4);
      }
    }
    if constexpr (E4M3) v.scale = vs0[pages * vsp + row_in_page(t + (lane & 31)) * vsr];
  }
};

// A lane number as it is: what derives from it at one end of a segment is not kept in registers until the next.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The kernel's arguments, read again from where they lie: what only the end of a segment needs is
// not held in scalar registers through the loop (there are about a hundred, and what spills costs vector registers).
__device__ __forceinline__ const AttentionArgs& arguments_again() {
  auto p = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttentionArgs*)p;
}

constexpr int padded_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
// Workgroups a CU holds (the registers they are compiled for): every workgroup of a call runs at once.
constexpr int resident_workgroups(int dp, bool e4m3, int head_tiles, bool plain) {
  return dp == 256 ? (e4m3 && plain ? 2 : 1) : head_tiles == 2 || !plain ? 2 : 3;
}

template <bool BF16, bool E4M3, int DP, int HT, bool PAGE16, bool FULL>
__global__ __launch_bounds__(kAttnThreads, resident_workgroups(DP, E4M3, HT, PAGE16 && FULL))
void paged_attention_kernel(AttentionArgs args) {
  typedef Attend<BF16, E4M3, DP, HT, PAGE16, FULL> A;
  constexpr int KS = A::KS, VF = A::VF;
  constexpr bool VBF = A::VBF;
  __shared__ float merge_ml[kAttnWaves][2][16];
  __shared__ float merge_o[kAttnWaves][16][DP + 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const AttentionArgs& a = args;
  const uint32_t pairs = uint32_t(a.heads) * uint32_t(a.head_tiles);

  // this workgroup's run of units [x, x1), and where it starts: sequence b, pair, unit of the pair
  const Walk walk = walk_lengths(a);
  const Cut cut = cut_of(walk.total * pairs, gridDim.x, uint32_t(a.least_units));
  if (blockIdx.x >= cut.wgs) return;
  const uint32_t x0 = cut.start(blockIdx.x), x1 = cut.start(blockIdx.x + 1);
  uint32_t x = x0;
  int b, n;
  uint32_t pair, unit, units;
  {
    const int at = __popcll(__ballot(walk.before * pairs <= x && lane * walk.per < a.table.batch)) - 1;
    uint32_t left = x - uint32_t(__builtin_amdgcn_readlane(int(walk.before), at)) * pairs;
    b = at * walk.per;
    for (;; ++b) {
      n = __builtin_amdgcn_readfirstlane(paged_len(a.lens, b, a.max_len));
      units = units_of(n, a.unit);
      if (left < units * pairs || b + 1 >= a.table.batch) break;
      left -= units * pairs;
    }
    pair = left / units;
    unit = left - pair * units;
  }

  A w;
  w.lane = lane, w.r = r, w.g = g;
  w.init(a);
  const float scale_log2e = a.scale_log2e;

  while (x < x1) {
    const uint32_t take = units - unit < x1 - x ? units - unit : x1 - x;
    const int h = int(udiv(pair, a.tiles_div)), g0 = int(pair - uint32_t(h) * a.tiles_div.d) * 16 * HT;
    const AttentionArgs& a = arguments_again();
    w.pools(a, b, h);
    const int t0 = int(unit * a.unit.d);
    const int64_t end = int64_t(unit + take) * a.unit.d;
    const int t1 = end < n ? int(end) : n;  // the segment's rows [t0, t1)

    typename A::Keys k;
    typename A::Values v;
    int t = t0 + wave * kTile;
    // (a wave without rows, or a sequence without any, has no tile)
    const bool any = t < t1;
    int entry = 0, next = 0;
    if (any) entry = w.load_pages(t, t1);

    // Q^T: column r is head g0 + 16 ht + r
    const int lane0 = fresh(lane), r0 = lane0 & 15, q0 = lane0 >> 4;
    u32x4 q[HT][KS];
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      const int head = g0 + 16 * ht + r0;
      const bool real = head < a.group;
      const unsigned char* row = a.q + b * a.qb + (int64_t(h) * a.group + (real ? head : a.group - 1)) * a.qh;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int d = A::q_element(s, q0, 0);
        const bool in = FULL || d < a.head_dim;
        const uint16_t* e = reinterpret_cast<const uint16_t*>(row) + (in ? d : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[ht][s][i] = uint32_t(e[2 * i]) | uint32_t(e[2 * i + 1]) << 16;
        if (!real || !in) q[ht][s] = u32x4{};
      }
    }
    const int group = a.group;
    const int64_t logit_row = a.logit_row;
    float* logits = a.logits ? a.logits + (int64_t(b) * a.heads + h) * group * logit_row : nullptr;
    f32x4 o[HT][VF];
    float m[HT], l[HT];  // of head r: the maximum over the wave's rows, the sum over the lane's
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      m[ht] = -kInf;
      l[ht] = 0.0f;
#pragma unroll
      for (int f = 0; f < VF; ++f) o[ht][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // One tile; with MORE the next one's loads among it.  They are in program order whatever the tile holds, so
    // that every wait is for a fixed number of younger loads.
    const auto tile = [&](auto more) {
      constexpr bool MORE = decltype(more)::value;
      // S^T
      f32x4 acc[2][HT];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) acc[u][ht] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          u32x4 y;
          if constexpr (E4M3) {
            const u32x4& c = k.x[u][s >> 1];
            const uint32_t w0 = c[(s & 1) * 2], w1 = c[(s & 1) * 2 + 1];
            y = u32x4{from_e4m3<BF16, false>(w0), from_e4m3<BF16, true>(w0), from_e4m3<BF16, false>(w1),
                      from_e4m3<BF16, true>(w1)};
            if (!FULL && 64 * (s >> 1) + 16 * g >= a.head_dim) y = u32x4{};
          } else {
            y = k.x[u][s];
            if (!FULL && 32 * s + 8 * g >= a.head_dim) y = u32x4{};
          }
#pragma unroll
          for (int ht = 0; ht < HT; ++ht) acc[u][ht] = mfma<BF16>(y, q[ht][s], acc[u][ht]);
        }
      }
      // base-2 logits
      float s[HT][2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f = scale_log2e;
          if constexpr (E4M3) f *= __shfl(k.scale, 16 * u + 4 * g + j, 64);
#pragma unroll
          for (int ht = 0; ht < HT; ++ht) s[ht][u][j] = acc[u][ht][j] * f;
        }
      const uint64_t missing = w.missing_rows(entry, t, t1);
      if constexpr (MORE) {
        entry = next;
        next = w.load_pages(t + 2 * kStep, t1);
        w.load_keys(entry, t + kStep, k);
      }

      float vs[2][4];
      if constexpr (E4M3) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) vs[u][j] = __shfl(v.scale, 16 * u + 4 * g + j, 64);
      }
      if (missing) {
        // rows that do not exist: logits of -infinity, values of 0 (their weight of 0 does not help against a
        // NaN)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool ok = !(missing >> (16 * u + 4 * g + j) & 1);
#pragma unroll
            for (int ht = 0; ht < HT; ++ht) s[ht][u][j] = ok ? s[ht][u][j] : -kInf;
#pragma unroll
            for (int i = 0; i < A::VW; ++i) v.x[4 * u + j][i] = ok ? v.x[4 * u + j][i] : 0u;
            if constexpr (E4M3) vs[u][j] = ok ? vs[u][j] : 0.0f;
          }
      }
      if (logits) {
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
          const int head = g0 + 16 * ht + r;
          if (head < group) {
            float* row = logits + head * logit_row + t + 4 * g;
#pragma unroll
            for (int u = 0; u < 2; ++u)
              *reinterpret_cast<f32x4*>(row + 16 * u) = f32x4{s[ht][u][0], s[ht][u][1], s[ht][u][2], s[ht][u][3]};
          }
        }
      }

      // online softmax, and P^T in B's layout as two 16-bit parts
      u32x4 hi[HT], lo[HT];
#pragma unroll
      for (int ht = 0; ht < HT; ++ht) {
        float top = m[ht];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) top = __builtin_fmaxf(top, s[ht][u][j]);
        top = __builtin_fmaxf(top, lane_xor<16>(top));
        top = __builtin_fmaxf(top, lane_xor<32>(top));
        const float ref = finite(top);
        if (__ballot(top > m[ht])) {
          const float shrink = __builtin_amdgcn_exp2f(m[ht] - ref);
          l[ht] *= shrink;
#pragma unroll
          for (int f = 0; f < VF; ++f) o[ht][f] *= shrink;
          m[ht] = top;
        }
        float e[8];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            e[4 * u + j] = __builtin_amdgcn_exp2f(s[ht][u][j] - ref);
            l[ht] += e[4 * u + j];
            if constexpr (E4M3) e[4 * u + j] *= vs[u][j];
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi[ht][i] = pack2<VBF>(e[2 * i], e[2 * i + 1]);
          lo[ht][i] = pack2<VBF>(e[2 * i] - low_half<VBF>(hi[ht][i]), e[2 * i + 1] - high_half<VBF>(hi[ht][i]));
        }
      }

      // O^T += V^T P^T
#pragma unroll
      for (int f = 0; f < VF; ++f) {
        u32x4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (E4M3) {
            // bytes f of rows 2 i and 2 i + 1, side by side
            y[i] = from_e4m3<true, false>(perm(v.x[2 * i + 1][f >> 2], v.x[2 * i][f >> 2],
                                               uint32_t((f & 3) | ((f & 3) + 4) << 8)));
          } else {
            y[i] = perm(v.x[2 * i + 1][f >> 1], v.x[2 * i][f >> 1], f & 1 ? 0x07060302u : 0x05040100u);
          }
        }
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
          o[ht][f] = mfma<VBF>(y, hi[ht], o[ht][f]);
          o[ht][f] = mfma<VBF>(y, lo[ht], o[ht][f]);
        }
      }
      if constexpr (MORE) w.load_values(entry, t + kStep, v);
    };
    if (any) {
      next = w.load_pages(t + kStep, t1);
      w.load_keys(entry, t, k);
      w.load_values(entry, t, v);
      for (; t + kStep < t1; t += kStep) tile(std::true_type());
      tile(std::false_type());
    }

    // the four waves' parts of each 16 heads
    const AttentionArgs& e = arguments_again();
    const int tid = fresh(int(threadIdx.x)), lane = tid & 63, r = lane & 15, g = lane >> 4;
    const bool done = take == units;
    const int64_t hq0 = (int64_t(b) * e.heads + h) * e.group;
    const int64_t slot = (int64_t(blockIdx.x) * 2 + (x != x0)) * (16 * HT);
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      l[ht] += lane_xor<16>(l[ht]);
      l[ht] += lane_xor<32>(l[ht]);
      __syncthreads();  // the last parts have been read
      if (g == 0) {
        merge_ml[wave][0][r] = m[ht];
        merge_ml[wave][1][r] = l[ht];
      }
#pragma unroll
      for (int f = 0; f < VF; f += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f32x4*>(&merge_o[wave][r][A::v_element(4 * g + i, f)]) =
              f32x4{o[ht][f][i], o[ht][f + 1][i], o[ht][f + 2][i], o[ht][f + 3][i]};
      __syncthreads();
      const int d0 = tid % (DP / 4) * 4;
      for (int head = tid / (DP / 4); head < 16; head += kAttnThreads / (DP / 4)) {
        const int hg = g0 + 16 * ht + head;
        if (hg >= e.group || (!FULL && d0 >= e.head_dim)) continue;
        float mx = -kInf, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kAttnWaves; ++i) mx = __builtin_fmaxf(mx, merge_ml[i][0][head]);
        const float ref = finite(mx);
        f32x4 all = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kAttnWaves; ++i) {
          const float f = __builtin_amdgcn_exp2f(merge_ml[i][0][head] - ref);
          sum += merge_ml[i][1][head] * f;
          all += *reinterpret_cast<const f32x4*>(&merge_o[i][head][d0]) * f;
        }
        if (!done) {
          const int64_t s = slot + 16 * ht + head;
          if (d0 == 0) {
            e.part_ml[2 * s] = mx;
            e.part_ml[2 * s + 1] = sum;
          }
          *reinterpret_cast<f32x4*>(e.part_o + s * e.head_dim + d0) = all;
          continue;
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint16_t* out = reinterpret_cast<uint16_t*>(e.out + b * e.ob + (int64_t(h) * e.group + hg) * e.oh) + d0;
        const uint32_t w0 = pack2<BF16>(all[0] * inv, all[1] * inv), w1 = pack2<BF16>(all[2] * inv, all[3] * inv);
        out[0] = uint16_t(w0);
        out[1] = uint16_t(w0 >> 16);
        out[2] = uint16_t(w1);
        out[3] = uint16_t(w1 >> 16);
        if (d0 == 0) {
          if (e.lse) e.lse[b * e.lb + (int64_t(h) * e.group + hg) * e.lh] = (mx + __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
          if (e.final_ml) {
            e.final_ml[2 * (hq0 + hg)] = mx;
            e.final_ml[2 * (hq0 + hg) + 1] = sum;
          }
        }
      }
    }

    x += take;
    unit += take;
    if (unit == units) {
      unit = 0;
      if (++pair == pairs) {
        pair = 0;
        ++b;
        if (x < x1) {
          n = __builtin_amdgcn_readfirstlane(paged_len(e.lens, b, e.max_len));
          units = units_of(n, e.unit);
        }
      }
    }
  }
}

// The parts of one query head of a pair that was cut, joined: their maxima give each part's factor,
// sums and outputs are added in a fixed order.  One workgroup a (sequence, query head): 32 lanes of four or eight
// elements, 16 parts at a time.
template <bool BF16>
__global__ __launch_bounds__(kJoinThreads) void paged_join_kernel(AttentionArgs a, uint32_t grid, Div32 q_heads) {
  constexpr int G = kJoinThreads / 32;
  __shared__ float part[G][kPagedMaxHeadDim];
  __shared__ float sums[G];
  const int b = int(udiv(blockIdx.x, q_heads)), hh = int(blockIdx.x) - b * int(q_heads.d);
  const uint32_t h = uint32_t(hh) / uint32_t(a.group), in_group = uint32_t(hh) - h * uint32_t(a.group);
  const uint32_t pairs = uint32_t(a.heads) * uint32_t(a.head_tiles), tile = in_group / uint32_t(a.tile_heads);
  const int n = __builtin_amdgcn_readfirstlane(paged_len(a.lens, b, a.max_len));
  const uint32_t units = units_of(n, a.unit);
  const Walk walk = walk_lengths(a);
  const Cut cut = cut_of(walk.total * pairs, grid, uint32_t(a.least_units));
  uint32_t before = uint32_t(__builtin_amdgcn_readlane(int(walk.before), b / walk.per));
  for (int k = b / walk.per * walk.per; k < b; ++k) before += units_of(paged_len(a.lens, k, a.max_len), a.unit);
  const uint32_t x0 = before * pairs + (h * uint32_t(a.head_tiles) + tile) * units;
  const uint32_t i0 = cut.owner(x0), i1 = cut.owner(x0 + units - 1);
  if (i0 == i1) return;
  // part k: of workgroup i0 + k, in its second slot where its run does not start with this pair
  const int parts = int(i1 - i0) + 1, first_slot = cut.start(i0) == x0 ? 0 : 1;
  const int64_t row0 = in_group - tile * uint32_t(a.tile_heads);
  const auto row = [&](int k) { return (int64_t(i0 + k) * 2 + (k == 0 ? first_slot : 0)) * a.tile_heads + row0; };
  float top = -kInf;
  for (int k = threadIdx.x & 63; k < parts; k += 64) top = __builtin_fmaxf(top, a.part_ml[2 * row(k)]);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
  const float ref = finite(top);
  const int lane4 = threadIdx.x & 31, grp = threadIdx.x >> 5;
  f32x4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
  float sum = 0.0f;
#pragma unroll 4
  for (int k = grp; k < parts; k += G) {
    const int64_t at = row(k);
    const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * at] - ref);
    sum += a.part_ml[2 * at + 1] * f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int d = 4 * lane4 + 128 * c;
      if (d < a.head_dim) acc[c] += *reinterpret_cast<const f32x4*>(a.part_o + at * a.head_dim + d) * f;
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) *reinterpret_cast<f32x4*>(&part[grp][4 * lane4 + 128 * c]) = acc[c];
  if (lane4 == 0) sums[grp] = sum;
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= a.head_dim) return;
  float total = 0.0f, y = 0.0f;
#pragma unroll
  for (int k = 0; k < G; ++k) {
    total += sums[k];
    y += part[k][d];
  }
  y = total == 0.0f ? 0.0f : y * (1.0f / total);
  reinterpret_cast<uint16_t*>(a.out + b * a.ob + hh * a.oh)[d] = uint16_t(pack2<BF16>(y, 0.0f));
  if (d == 0) {
    if (a.lse) a.lse[b * a.lb + hh * a.lh] = (top + __builtin_amdgcn_logf(total)) * 0.6931471805599453f;
    if (a.final_ml) {
      a.final_ml[2 * int64_t(blockIdx.x)] = top;
      a.final_ml[2 * int64_t(blockIdx.x) + 1] = total;
    }
  }
}

// weights_out[i] = weights[i] + the sum over a cache head's query heads of exp2(logit - maximum) / sum.
// One workgroup a kWeightRows rows of one (sequence, cache head).
constexpr int kWeightRows = 1024;
__global__ __launch_bounds__(256) void paged_weights_kernel(AttentionArgs a, Div32 heads, Div32 chunks) {
  const uint32_t bh = udiv(blockIdx.x, chunks), chunk = blockIdx.x - bh * chunks.d;
  const int b = int(udiv(bh, heads)), h = int(bh - uint32_t(b) * heads.d);
  const int n = paged_len(a.lens, b, a.max_len);
  const int i0 = int(chunk) * kWeightRows;
  if (i0 >= n) return;
  const float* w = a.weights + b * a.w.sb + h * a.w.sh;
  float* wo = a.weights_out + b * a.wo.sb + h * a.wo.sh;
  float sum[kWeightRows / 256] = {};
  for (int g = 0; g < a.group; ++g) {
    const int64_t hq = int64_t(bh) * a.group + g;
    const float ref = finite(a.final_ml[2 * hq]), total = a.final_ml[2 * hq + 1];
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    const float* x = a.logits + hq * a.logit_row;
#pragma unroll
    for (int k = 0; k < kWeightRows / 256; ++k) {
      const int i = i0 + 256 * k + int(threadIdx.x);
      if (i < n) sum[k] += __builtin_amdgcn_exp2f(x[i] - ref) * inv;
    }
  }
#pragma unroll
  for (int k = 0; k < kWeightRows / 256; ++k) {
    const int i = i0 + 256 * k + int(threadIdx.x);
    if (i < n) wo[i * a.wo.sc] = w[i * a.w.sc] + sum[k];
  }
}

template <bool BF16, bool E4M3, int DP, int HT, bool PAGE16, bool FULL>
void attend(const AttentionArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((paged_attention_kernel<BF16, E4M3, DP, HT, PAGE16, FULL>), dim3(uint32_t(a.workgroups)),
                     dim3(kAttnThreads), 0, s, a);
}

// PAGE16's lane offsets are 32-bit: 16 rows of either pool have to fit.
bool pages_of_16(const PagedPool& p) {
  const int64_t most = int64_t(1) << 27;
  return p.page_size % 16 == 0 && p.kr < most && p.vr < most;
}

template <bool BF16, bool E4M3, int DP, int HT>
void by_page(const AttentionArgs& a, hipStream_t s) {
  if (!pages_of_16(a.pool)) return attend<BF16, E4M3, DP, HT, false, false>(a, s);
  return a.head_dim == DP ? attend<BF16, E4M3, DP, HT, true, true>(a, s) : attend<BF16, E4M3, DP, HT, true, false>(a, s);
}

template <bool BF16, bool E4M3, int DP>
void by_group(const AttentionArgs& a, hipStream_t s) {
  if constexpr (DP <= 128)
    if (a.tile_heads == 32) return by_page<BF16, E4M3, DP, 2>(a, s);
  return by_page<BF16, E4M3, DP, 1>(a, s);
}

template <bool BF16, bool E4M3>
void by_dim(const AttentionArgs& a, hipStream_t s) {
  if (a.head_dim <= 64) return by_group<BF16, E4M3, 64>(a, s);
  if (a.head_dim <= 128) return by_group<BF16, E4M3, 128>(a, s);
  return by_group<BF16, E4M3, 256>(a, s);
}

}  // namespace dev

int64_t paged_logit_row(int64_t max_len) { return (max_len + dev::kStep - 1) / dev::kStep * dev::kStep; }

PagedCut paged_cut(int64_t batch, int64_t heads, int64_t group, int64_t head_dim, int64_t max_len) {
  PagedCut c{};
  // 32 heads at once for larger groups, where their outputs fit the registers
  c.tile_heads = group > 16 && head_dim <= 128 ? 32 : 16;
  c.head_tiles = (group + c.tile_heads - 1) / c.tile_heads;
  const int64_t pairs = batch * heads * c.head_tiles;
  c.unit_rows = dev::kStep;
  c.least_units = 2;
  if (max_len <= 512) {
    c.unit_rows = std::max<int64_t>(dev::kStep, (max_len + dev::kStep - 1) / dev::kStep * dev::kStep);
    c.least_units = 1;
  }
  const int64_t most = pairs * std::max<int64_t>(1, (max_len + c.unit_rows - 1) / c.unit_rows);
  c.cuts = most > pairs;
  const int64_t resident = dev::resident_workgroups(dev::padded_dim(int(head_dim)), true, int(c.tile_heads / 16), true);
  c.workgroups = std::min<int64_t>((most + c.least_units - 1) / c.least_units, resident * dev::kCus);
  c.units = most;
  return c;
}

int launch_paged_attention(const AttentionArgs& in, int dtype, int cache_dtype, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  AttentionArgs a = in;
  const int64_t rows = int64_t(a.table.batch) * a.heads;
  const int64_t chunks = (int64_t(a.max_len) + dev::kWeightRows - 1) / dev::kWeightRows;
  if (rows * chunks >= int64_t(1) << 31) return TC_E_RANGE;
  const int dp = dev::padded_dim(a.head_dim);
  a.workgroups = std::min(a.workgroups, dev::kCus * dev::resident_workgroups(dp, cache_dtype == TC_E4M3, a.tile_heads / 16,
                                                                             dev::pages_of_16(a.pool) && a.head_dim == dp));
  const bool bf16 = dtype == TC_BF16, e4m3 = cache_dtype == TC_E4M3;
  if (bf16)
    e4m3 ? dev::by_dim<true, true>(a, s) : dev::by_dim<true, false>(a, s);
  else
    e4m3 ? dev::by_dim<false, true>(a, s) : dev::by_dim<false, false>(a, s);
  if (a.part_o) {
    const uint32_t hq = uint32_t(rows) * uint32_t(a.group);
    const Div32 qh = make_div32(uint32_t(a.heads) * uint32_t(a.group));
    if (bf16)
      hipLaunchKernelGGL(dev::paged_join_kernel<true>, dim3(hq), dim3(dev::kJoinThreads), 0, s, a, uint32_t(a.workgroups), qh);
    else
      hipLaunchKernelGGL(dev::paged_join_kernel<false>, dim3(hq), dim3(dev::kJoinThreads), 0, s, a, uint32_t(a.workgroups), qh);
  }
  if (a.weights_out && chunks > 0)
    hipLaunchKernelGGL(dev::paged_weights_kernel, dim3(uint32_t(rows * chunks)), dim3(256), 0, s, a,
                       make_div32(uint32_t(a.heads)), make_div32(uint32_t(chunks)));
  return TC_OK;
}

}  // namespace tc
