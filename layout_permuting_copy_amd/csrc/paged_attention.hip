// Attention of one new token a sequence over a paged cache, split over the cache's length and joined.
#include <algorithm>
#include <type_traits>

#include "paged_common.hpp"

namespace tc {
namespace dev {

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = 4;
constexpr int kTile = 32;                       // cache rows a wave takes at a time
constexpr int kStep = kTile * kAttnWaves;       // and a workgroup
constexpr int kJoinThreads = 256;
constexpr int kCus = 256;

// N bytes of a buffer resource at a lane's offset, `more` bytes on: zeros past its range, which takes the place of a condition
// on the load (every wait then is for a fixed number of younger loads).  STREAM: read past the caches.
template <int N, bool STREAM>
__device__ __forceinline__ void load_buffer(Rsrc rsrc, uint32_t off, int more, uint32_t* w) {
  constexpr int policy = STREAM ? kPolNT : 0;
  if constexpr (N == 16) {
    const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, int(off), more, policy));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 8) {
    const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rsrc, int(off), more, policy));
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, int(off), more, policy);
  }
}
constexpr uint32_t kBeyond = 0x80000000u;  // an offset past every range (ranges end below 2^31)
__device__ __forceinline__ Rsrc rows_rsrc(const unsigned char* base, bool live) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char*>(base), 0, live ? int(kBeyond - 1) : 0, kRsrcWord3);
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

// The maximum or sum over the four lanes that differ in bits 4 and 5 (the groups g).
__device__ __forceinline__ float max_of_groups(float x) {
  float p, q;
  partners<16>(x, &p, &q);
  x = __builtin_fmaxf(p, q);
  partners<32>(x, &p, &q);
  return __builtin_fmaxf(p, q);
}
__device__ __forceinline__ float sum_of_groups(float x) {
  float p, q;
  partners<16>(x, &p, &q);
  x = p + q;
  partners<32>(x, &p, &q);
  return p + q;
}

// How the call's work is cut: a sequence of n rows has max(1, ceil(n / unit_rows)) units; the units of all
// sequences, one after another, are dealt in equal runs (the first `rest` of them one longer), and a run goes to as
// many workgroups as there are pairs (a cache head and a tile of its query heads), next to each other in the grid: the
// heads of one row are read at about the same time.  A sequence within one run is finished there; one that is
// cut leaves partial results, in slot 0 of the workgroups whose run starts with it and slot 1 of those
// whose run ends in it.
struct Cut {
  uint32_t runs, each, rest;
  __device__ __forceinline__ uint32_t start(uint32_t i) const { return i * each + (i < rest ? i : rest); }
  __device__ __forceinline__ uint32_t owner(uint32_t x) const {
    const uint32_t longer = rest * (each + 1);
    return x < longer ? x / (each + 1) : rest + (x - longer) / each;
  }
};

struct Walk {
  uint32_t total;   // units of all sequences
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
  const uint32_t upto = wave_scan(sum);
  w.total = uint32_t(__builtin_amdgcn_readlane(int(upto), 63));
  w.before = upto - sum;
  return w;
}

__device__ __forceinline__ Cut cut_of(uint32_t units, uint32_t most, uint32_t least_each) {
  Cut c;
  c.runs = (units + least_each - 1) / least_each;
  c.runs = c.runs < most ? c.runs : most;
  c.each = units / c.runs;
  c.rest = units - c.each * c.runs;
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
// P is held as the sum of 16-bit values (its rounding, the rest's rounding, ...), a product each, the matrix cores being
// mostly idle.  Three bf16 values hold all 24 bits of an fp32 weight; two would leave 2^-18 of it, which shows where
// values cancel (the third costs 0.2 us of 6.3 of 131 rows, 0.5 of 88 of the batch, 1.2 of 187 of the 8-bit rows).  Two fp16
// values hold 22 bits: what they leave is no more than the rounding of a logit of 4 does (a third would cost 0.4 of 24.5
// us).  fp16 parts end at 2^-25, which many light rows beside a heavy one would notice: weights (and sums) are 2^15 times as
// large there until the waves meet.
// 8-bit rows become 16-bit values in registers (exactly); the key's scale multiplies its row's
// logits, the value's its row's weights.
//
// The next tile's keys are requested once this tile's logits are formed, its values once this tile's are
// used, the pages of the one after next before both, so a wave always has loads in flight.  No load of the
// cache is conditional: rows past the end and rows on no page are read from wherever their index leads inside
// the pool (page 0 for no page), and what comes back is masked, in the tiles that have such rows.  The loop
// holds the only copy of its code (its first turn requests and computes nothing, its last computes and
// requests nothing): a short call's time goes into fetching instructions.
//
// DP: head_dim rounded up to 64, 128 or 256.  FULL: head_dim is DP; else the key elements past it are
// zeros (those of Q are, but 0 times infinity is not 0) and the output elements past it not stored.
// PAGE, the rows known to lie on one page: 16 (a half: its address is scalar, its loads go through a
// buffer resource), 4 (a lane's value rows of a half) or 1.
//
// Bound: HBM (a cache row is read once for all heads of its group, up to 16 of them above 128 elements and 32 below;
// FETCH_SIZE counts each byte once.  Larger groups take their tiles of heads from the cache each: one sequence of 65536 rows of
// 256, groups of 16 and 20: 95 and 121 us; 131072 rows of 128, 32 and 40: 102 and 143).  Measured: one
// sequence of 131072 rows, 8 heads of 128 bf16 elements under 64 query heads: 537 MB in 82.8 us (6.5 TB/s, where
// a plain read of 1 GiB reaches 6.1 through the caches and 7.0 past them); 32 of 16384 8-bit rows: 1.11 GB in 176 us
// (6.3 TB/s); 64 of mixed lengths up to 4096 in pages that hold a row's heads together: 468 MB in 83 us (5.6).  Short
// calls are a chain of trips to memory: 131 rows take 6.5 us in a graph, where an empty kernel takes 1.6.  Tried and not
// kept: two tiles ahead of the one computed (the short call 7.1 us, the others level), the next sequence's first
// tile requested before a segment's end (level), fixed splits of 256 to 2048 rows with a join of all (64 sequences:
// 106 to 143 us).
template <bool BF16, bool E4M3, int DP, int HT, int PAGE, bool FULL>
struct Attend {
  static constexpr bool VBF = BF16 || E4M3;       // type of the second product
  static constexpr int EB = E4M3 ? 1 : 2;
  static constexpr int KS = DP / 32;              // contraction steps of the first product
  static constexpr int KC = DP * EB / 64;         // 16-byte chunks a lane loads of a key row
  static constexpr int VF = DP / 16;              // elements a lane loads of a value row: tiles of O^T
  static constexpr int VB = VF * EB;              // their bytes: 4, 8, 16 or 32
  static constexpr int VP = VB == 32 ? 16 : VB;   // bytes a load
  static constexpr int VW = VB / 4;
  static constexpr int PARTS = VBF ? 3 : 2;   // 16-bit values that hold a weight
  static constexpr int RAISE = VBF ? 0 : 15;      // weights are held times 2 to this (at most 2^15, 65504 is fp16's last)

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
  // the lane's byte offsets.  PAGE 16: in the 16 rows of a half, of key row r and value row 4 g; otherwise in a row.
  // Both include the lane's chunk; of a row's chunk past head_dim: beyond the range, or the row's first
  uint32_t kchunk[FULL ? 1 : KC], vchunk, vchunk2;

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
    const int bytes = a.head_dim * EB, e0 = v_element(r, 0) * EB, e1 = e0 + DP / 2 * EB;
    const uint32_t krow = PAGE == 16 ? uint32_t(r) * uint32_t(kr) : 0u, vrow = PAGE == 16 ? uint32_t(4 * g) * uint32_t(vr) : 0u;
    const uint32_t none = PAGE == 16 ? kBeyond : 0u;
#pragma unroll
    for (int c = 0; c < (FULL ? 1 : KC); ++c) kchunk[c] = FULL || 64 * c + 16 * g < bytes ? krow + 64 * c + 16 * g : none;
    vchunk = FULL || e0 < bytes ? vrow + e0 : none;
    vchunk2 = FULL || e1 < bytes ? vrow + e1 : none;
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
  // `entry` past the pool (no page) is taken as page 0; rows past the end lie on their page all the same.
  __device__ __forceinline__ int page_of(int entry) const { return uint32_t(entry) < uint32_t(pool_pages) ? entry : 0; }
  // A row of the pool for a lane (PAGE < 16); where nothing is to be loaded, the pool's first row for every lane.
  __device__ __forceinline__ const unsigned char* row_of(const unsigned char* base, int64_t sp, int64_t sr, int pages, int t,
                                                        int i, bool live) const {
    const int64_t off = __shfl(pages, i, 64) * sp + row_in_page(t + i) * sr;
    return base + (live ? off : 0);
  }
  __device__ __forceinline__ float load_scale(const float* base, int64_t sp, int64_t sr, int pages, int t, bool live) const {
    const int64_t off = pages * sp + row_in_page(t + (lane & 31)) * sr;
    return base[live ? off : 0];
  }

  // The tile at t of table entries `entry`; not live: no memory is read (PAGE 16), or little.
  __device__ __forceinline__ void load_keys(int entry, int t, bool live, Keys& k) const {
    const int pages = page_of(entry);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if constexpr (PAGE == 16) {
        const Rsrc half = rows_rsrc(k0 + (__builtin_amdgcn_readlane(pages, 16 * u) * kp + row_in_page(t + 16 * u) * kr), live);
#pragma unroll
        for (int c = 0; c < KC; ++c)
          load_buffer<16, false>(half, kchunk[FULL ? 0 : c], FULL ? 64 * c : 0, reinterpret_cast<uint32_t*>(&k.x[u][c]));
      } else {
        const unsigned char* row = row_of(k0, kp, kr, pages, t, 16 * u + r, live);
#pragma unroll
        for (int c = 0; c < KC; ++c)
          load_words<16>(row + (FULL ? kchunk[0] + 64 * c : kchunk[FULL ? 0 : c]), reinterpret_cast<uint32_t*>(&k.x[u][c]));
      }
    }
    if constexpr (E4M3) k.scale = load_scale(ks0, ksp, ksr, pages, t, live);
  }

  // Values are read past the caches: nothing else needs their lines (131072 rows: 103 -> 93 us).  Keys are not, as a
  // line of a key row is covered by two loads (past the caches: 8 sequences with weights 33 -> 38 us).
  __device__ __forceinline__ void load_values(int entry, int t, bool live, Values& v) const {
    const int pages = page_of(entry);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if constexpr (PAGE == 16) {
        const unsigned char* half = v0 + (__builtin_amdgcn_readlane(pages, 16 * u) * vp + row_in_page(t + 16 * u) * vr);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const Rsrc row = rows_rsrc(half + j * vr, live);
          load_buffer<VP, true>(row, vchunk, 0, v.x[4 * u + j]);
          if constexpr (VB == 32) load_buffer<VP, true>(row, FULL ? vchunk : vchunk2, FULL ? DP / 2 * EB : 0, v.x[4 * u + j] + 4);
        }
      } else {
        const unsigned char* row = nullptr;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (PAGE == 1 || j == 0)
            row = row_of(v0, vp, vr, pages, t, 16 * u + 4 * g + j, live);
          else
            row += live ? vr : 0;
          gload<VP, 1>(row + vchunk, v.x[4 * u + j]);
          if constexpr (VB == 32) gload<VP, 1>(row + vchunk2, v.x[4 * u + j] + 4);
        }
      }
    }
    if constexpr (E4M3) v.scale = load_scale(vs0, vsp, vsr, pages, t, live);
  }
};

// The kernel's arguments, read again from where they lie: what only the end of a segment needs is
// not held in scalar registers through the loop (there are about a hundred, and what spills costs vector registers).
__device__ __forceinline__ const AttentionArgs& arguments_again() {
  auto p = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttentionArgs*)p;
}

constexpr int padded_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
// Workgroups a CU gets at once, and the registers they are compiled for.  Fewer, longer runs cut fewer sequences and come
// out more even, as long as they keep the memory busy: one workgroup's four waves do with rows of 256 bytes and more
// (64 KB on their way; 64 sequences of mixed lengths in 16-bit rows of 128: 88 us with one a CU, 93 with two or three; 8
// of 16384 8-bit rows of 256: 99 with one, 101 with two, in pages of 24 107 and 110), narrower rows want two (8-bit rows of
// 128: 200 us with one, 187 with two, 194 with three).  Two tiles of heads without FULL and PAGE 16 need more
// registers than two workgroups have.
constexpr int resident_workgroups(int dp, bool e4m3, int head_tiles, bool plain) {
  const int bytes = dp * (e4m3 ? 1 : 2);
  return bytes < 256 && (head_tiles == 1 || plain) ? 2 : 1;
}

template <bool BF16, bool E4M3, int DP, int HT, int PAGE, bool FULL>
__global__ __launch_bounds__(kAttnThreads, resident_workgroups(DP, E4M3, HT, PAGE == 16 && FULL))
void paged_attention_kernel(AttentionArgs args) {
  typedef Attend<BF16, E4M3, DP, HT, PAGE, FULL> A;
  constexpr int KS = A::KS, VF = A::VF;
  constexpr bool VBF = A::VBF;
  __shared__ float merge_ml[kAttnWaves][2][16];
  __shared__ float merge_o[kAttnWaves][16][DP + 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const AttentionArgs& a = args;
  const uint32_t run = udiv(blockIdx.x, a.pairs_div), pair = blockIdx.x - run * a.pairs_div.d;
  const int tile = int(udiv(pair, a.heads_div)), h = int(pair) - tile * int(a.heads_div.d), g0 = tile * 16 * HT;

  // this workgroup's run of units [x0, x1), and where it starts: sequence b, unit of it
  int b, n;
  uint32_t x0, x1, unit, units;
  Cut cut;
  if (!a.parts) {  // nothing is cut: every sequence is one unit and one run
    cut = Cut{};
    x0 = run;
    x1 = run + 1;
    b = int(run);
    unit = 0;
    units = 1;
    n = __builtin_amdgcn_readfirstlane(paged_len(a.lens, b, a.max_len));
  } else {
    const Walk walk = walk_lengths(a);
    cut = cut_of(walk.total, uint32_t(a.runs), uint32_t(a.least_units));
    if (!a.parts_of_sequences && pair == 0 && threadIdx.x == 0) a.parts[run].count = 0;
    if (run >= cut.runs) return;
    x0 = cut.start(run);
    x1 = cut.start(run + 1);
    const int at = __popcll(__ballot(walk.before <= x0 && lane * walk.per < a.table.batch)) - 1;
    unit = x0 - uint32_t(__builtin_amdgcn_readlane(int(walk.before), at));
    b = at * walk.per;
    for (;; ++b) {
      n = __builtin_amdgcn_readfirstlane(paged_len(a.lens, b, a.max_len));
      units = units_of(n, a.unit);
      if (unit < units || b + 1 >= a.table.batch) break;
      unit -= units;
    }
  }
  uint32_t x = x0;

  A w;
  w.lane = lane, w.r = r, w.g = g;
  w.init(a);
  const float scale_log2e = a.scale_log2e;

  while (x < x1) {
    const uint32_t take = units - unit < x1 - x ? units - unit : x1 - x;
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
    int entry = 0;
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
    const int group = a.group, head_dim = a.head_dim;
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

    // t: the next tile; the one before it is computed while its loads are on their way
    bool live = any, have = false;
    uint64_t missing = 0;  // of the tile computed
    while (live || have) {
      float s[HT][2][4];
      if (have) {
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
              if (PAGE < 16 && !FULL && 64 * (s >> 1) + 16 * g >= head_dim) y = u32x4{};
            } else {
              y = k.x[u][s];
              if (PAGE < 16 && !FULL && 32 * s + 8 * g >= head_dim) y = u32x4{};
            }
#pragma unroll
            for (int ht = 0; ht < HT; ++ht) acc[u][ht] = mfma<BF16>(y, q[ht][s], acc[u][ht]);
          }
        }
        // base-2 logits
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float f = scale_log2e;
            if constexpr (E4M3) f *= __shfl(k.scale, 16 * u + 4 * g + j, 64);
#pragma unroll
            for (int ht = 0; ht < HT; ++ht) s[ht][u][j] = acc[u][ht][j] * f;
          }
      }
      const int now = entry;
      entry = w.load_pages(t + kStep, t1);
      w.load_keys(now, t, live, k);
      if (have) {
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
              float* row = logits + head * logit_row + (t - kStep) + 4 * g;
#pragma unroll
              for (int u = 0; u < 2; ++u)
                *reinterpret_cast<f32x4*>(row + 16 * u) = f32x4{s[ht][u][0], s[ht][u][1], s[ht][u][2], s[ht][u][3]};
            }
          }
        }

        // online softmax, and P^T in B's layout as 16-bit parts
        u32x4 part[HT][A::PARTS];
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
          float top = m[ht];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) top = __builtin_fmaxf(top, s[ht][u][j]);
          top = max_of_groups(top);
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
              // (raised after the difference, which rounds to no more than 0: ref - 15 would be any of its neighbours from 2^24 on)
              e[4 * u + j] = __builtin_amdgcn_exp2f(s[ht][u][j] - ref) * float(1 << A::RAISE);
              l[ht] += e[4 * u + j];
              if constexpr (E4M3) e[4 * u + j] *= vs[u][j];
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = e[2 * i], y = e[2 * i + 1];
#pragma unroll
            for (int k = 0; k < A::PARTS; ++k) {
              const uint32_t w = part[ht][k][i] = pack2<VBF>(x, y);
              x -= low_half<VBF>(w);
              y -= high_half<VBF>(w);
            }
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
#pragma unroll
            for (int k = 0; k < A::PARTS; ++k) o[ht][f] = mfma<VBF>(y, part[ht][k], o[ht][f]);
          }
        }
      }
      w.load_values(now, t, live, v);
      missing = w.missing_rows(now, t, t1);
      have = live;
      t += kStep;
      live = t < t1;
    }

    // the four waves' parts of each 16 heads
    const AttentionArgs& e = arguments_again();
    const int tid = fresh(int(threadIdx.x)), lane = tid & 63, r = lane & 15, g = lane >> 4;
    const bool done = take == units;
    const int64_t hq0 = (int64_t(b) * e.heads + h) * e.group;
    const int64_t slot = (int64_t(blockIdx.x) * 2 + (x != x0)) * (16 * HT);
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
      l[ht] = sum_of_groups(l[ht]);
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
      constexpr int at_once = kAttnThreads / (DP / 4);
#pragma unroll
      for (int head0 = 0; head0 < 16; head0 += at_once) {
        const int head = head0 + tid / (DP / 4);
        const int hg = g0 + 16 * ht + head;
        if (hg >= e.group || (!FULL && d0 >= e.head_dim)) continue;
        float mx = -kInf, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kAttnWaves; ++i) mx = __builtin_fmaxf(mx, merge_ml[i][0][head]);
        const float ref = finite(mx);
        f32x4 all = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kAttnWaves; ++i) {
          const float f = __builtin_amdgcn_exp2f(merge_ml[i][0][head] - ref) * (1.0f / float(1 << A::RAISE));
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

    if (e.parts && unit == 0 && pair == 0 && tid == 0 && (e.parts_of_sequences || !done)) {
      // the sequence starts in this run: the runs up to its last unit have its other parts
      const int count = done ? 0 : int(cut.owner(x + units - 1) - run) + 1;
      e.parts[e.parts_of_sequences ? b : int(run)] = PagedParts{b, int32_t(run), count, x != x0};
    }
    x += take;
    unit += take;
    if (unit == units && x < x1) {
      unit = 0;
      ++b;
      n = __builtin_amdgcn_readfirstlane(paged_len(e.lens, b, e.max_len));
      units = units_of(n, e.unit);
    }
  }
}

// The parts of one query head of a sequence that was cut, joined: their maxima give each part's factor, sums and
// outputs are added in a fixed order.  Grid: (sequence or run, query head); those with nothing to join end at
// once.  32 lanes of four or eight elements, 8 parts at a time and 8 such rounds of loads on their way: the call's
// time is its launch and three trips to memory (32 parts of 64 heads: 4.9 us; with one round at a time, 10 us).
template <bool BF16>
__global__ __launch_bounds__(kJoinThreads) void paged_join_kernel(AttentionArgs a) {
  constexpr int G = kJoinThreads / 32, R = 64 / G;
  __shared__ float part[G][kPagedMaxHeadDim];
  const PagedParts p = a.parts[blockIdx.x];
  if (p.count == 0) return;
  const int hh = int(blockIdx.y), h = hh / a.group, in_group = hh - h * a.group, tile = in_group / a.tile_heads;
  // part k: of run p.run + k, in its second slot where its run did not start with this sequence
  const int64_t step = int64_t(a.pairs_div.d) * 2 * a.tile_heads;
  const int64_t row0 = (int64_t(p.run) * a.pairs_div.d + tile * a.heads + h) * 2 * a.tile_heads + (in_group - tile * a.tile_heads);
  const int64_t first = p.slot ? a.tile_heads : 0;
  const int lane = threadIdx.x & 63, lane4 = threadIdx.x & 31, grp = threadIdx.x >> 5;
  float top = -kInf;
  for (int k = lane; k < p.count; k += 64) top = __builtin_fmaxf(top, a.part_ml[2 * (row0 + k * step + (k ? 0 : first))]);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, d, 64));
  const float ref = finite(top);
  f32x4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
  float total = 0.0f;
  for (int k0 = 0; k0 < p.count; k0 += 64) {
    // lane k: the factor of part k0 + k
    float f = 0.0f;
    if (k0 + lane < p.count) {
      const float* ml = a.part_ml + 2 * (row0 + (k0 + lane) * step + (k0 + lane ? 0 : first));
      f = __builtin_amdgcn_exp2f(ml[0] - ref);
      total += ml[1] * f;
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (128 * c >= a.head_dim) break;
      // lanes past the row read its end again and stay for the exchanges
      const int d = 4 * lane4 + 128 * c < a.head_dim ? 4 * lane4 + 128 * c : a.head_dim - 4;
      const auto load = [&](int i) {
        const int k = k0 + grp + G * i, at = k < p.count ? k : p.count - 1;
        return *reinterpret_cast<const f32x4*>(a.part_o + (row0 + at * step + (at ? 0 : first)) * a.head_dim + d);
      };
      const auto add = [&](int i, const f32x4& x) {
        const float y = __shfl(f, grp + G * i, 64);
        if (k0 + grp + G * i < p.count) acc[c] += x * y;
      };
      if (p.count <= G) {
        add(0, load(0));
      } else {
        f32x4 x[R];
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = load(i);
#pragma unroll
        for (int i = 0; i < R; ++i) add(i, x[i]);
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d, 64);
#pragma unroll
  for (int c = 0; c < 2; ++c) *reinterpret_cast<f32x4*>(&part[grp][4 * lane4 + 128 * c]) = acc[c];
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= a.head_dim) return;
  float y = 0.0f;
#pragma unroll
  for (int k = 0; k < G; ++k) y += part[k][d];
  y = total == 0.0f ? 0.0f : y * (1.0f / total);
  reinterpret_cast<uint16_t*>(a.out + p.b * a.ob + hh * a.oh)[d] = uint16_t(pack2<BF16>(y, 0.0f));
  if (d == 0) {
    if (a.lse) a.lse[p.b * a.lb + hh * a.lh] = (top + __builtin_amdgcn_logf(total)) * 0.6931471805599453f;
    if (a.final_ml) {
      float* ml = a.final_ml + 2 * (int64_t(p.b) * a.heads * a.group + hh);
      ml[0] = top;
      ml[1] = total;
    }
  }
}

// weights_out[i] = weights[i] + the sum over a cache head's query heads of exp2(logit - maximum) / sum.
// One lane a row, one workgroup 256 rows of one (sequence, cache head).  Bound: its launch, and the logits' bytes
// (28728 rows, 8 heads, groups of 4: 4.0 us; with 1024 rows a workgroup 8.4).
constexpr int kWeightRows = 256;
__global__ __launch_bounds__(kWeightRows) void paged_weights_kernel(AttentionArgs a, Div32 heads, Div32 chunks) {
  const uint32_t bh = udiv(blockIdx.x, chunks), chunk = blockIdx.x - bh * chunks.d;
  const int b = int(udiv(bh, heads)), h = int(bh - uint32_t(b) * heads.d);
  const int n = paged_len(a.lens, b, a.max_len);
  const int i = int(chunk) * kWeightRows + int(threadIdx.x);
  if (i >= n) return;
  const float before = a.weights[b * a.w.sb + h * a.w.sh + i * a.w.sc];
  const float* ml = a.final_ml + 2 * int64_t(bh) * a.group;
  const float* x = a.logits + int64_t(bh) * a.group * a.logit_row + i;
  float sum = 0.0f;
#pragma unroll 4
  for (int g = 0; g < a.group; ++g) {
    const float total = ml[2 * g + 1], inv = total == 0.0f ? 0.0f : 1.0f / total;
    sum += __builtin_amdgcn_exp2f(x[g * a.logit_row] - finite(ml[2 * g])) * inv;
  }
  a.weights_out[b * a.wo.sb + h * a.wo.sh + i * a.wo.sc] = before + sum;
}

template <bool BF16, bool E4M3, int DP, int HT, int PAGE, bool FULL>
void attend(const AttentionArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((paged_attention_kernel<BF16, E4M3, DP, HT, PAGE, FULL>), dim3(uint32_t(a.workgroups)),
                     dim3(kAttnThreads), 0, s, a);
}

// PAGE 16's lane offsets are 32-bit: 16 rows of either pool have to fit.
bool pages_of_16(const PagedPool& p) {
  const int64_t most = int64_t(1) << 27;
  return p.page_size % 16 == 0 && p.kr < most && p.vr < most;
}

template <bool BF16, bool E4M3, int DP, int HT>
void by_page(const AttentionArgs& a, hipStream_t s) {
  const bool full = a.head_dim == DP;
  if (pages_of_16(a.pool)) return full ? attend<BF16, E4M3, DP, HT, 16, true>(a, s) : attend<BF16, E4M3, DP, HT, 16, false>(a, s);
  if (a.pool.page_size % 4 == 0) return full ? attend<BF16, E4M3, DP, HT, 4, true>(a, s) : attend<BF16, E4M3, DP, HT, 4, false>(a, s);
  return attend<BF16, E4M3, DP, HT, 1, false>(a, s);
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

// As many runs as make up the workgroups that the card holds at once, to the nearest.  (Where the pairs do not divide those, some
// workgroups more wait for a second turn: 65536 rows of 256 under 8 heads take 93 us, as many bytes under 6 and 10 heads 138
// and 142.)
static int64_t runs_of(int64_t units, int64_t least, int64_t pairs, int64_t resident) {
  const int64_t fit = std::max<int64_t>(1, (resident * dev::kCus + pairs / 2) / pairs);
  return std::min((units + least - 1) / least, fit);
}

PagedCut paged_cut(int64_t batch, int64_t heads, int64_t group, int64_t head_dim, int64_t max_len, bool most) {
  PagedCut c{};
  // 32 heads at once for larger groups, where their outputs fit the registers
  c.tile_heads = group > 16 && head_dim <= 128 ? 32 : 16;
  c.head_tiles = (group + c.tile_heads - 1) / c.tile_heads;
  // a turn of the four waves (units of 64 or 32 rows: 64 sequences of mixed lengths 89 -> 90 or 93 us, others level);
  // at least two turns a run (one or two: level, four: 16 sequences under one head 22 -> 30 us)
  c.unit_rows = dev::kStep;
  c.least_units = 2;
  const int64_t pairs = heads * c.head_tiles;
  // short caches are not cut: four turns take less than the join's launch (16 sequences, 128 elements: 512 rows
  // in 9 us uncut, 513 in 12 us cut), and eight turns where every CU has a sequence and head anyway (8 heads of 128,
  // mixed lengths, uncut and cut: 16 sequences of up to 1000 rows 17 and 16 us, 32 18 and 23, 512 171 and 188; of up
  // to 2000 rows 32 sequences 31 and 30, 64 58 and 53)
  if (max_len <= 512 || (max_len <= 1024 && batch * pairs >= dev::kCus && !most)) {
    c.unit_rows = std::max<int64_t>(dev::kStep, (max_len + dev::kStep - 1) / dev::kStep * dev::kStep);
    c.least_units = 1;
  }
  c.units = batch * std::max<int64_t>(1, (max_len + c.unit_rows - 1) / c.unit_rows);
  c.cuts = c.units > batch;
  // uncut sequences get a run each, and workgroups that wait their turn hide each other's ends and beginnings (512 of 512
  // rows: 181 us, 206 in one run a CU)
  c.runs = !c.cuts ? batch
                   : runs_of(c.units, c.least_units, pairs,
                             dev::resident_workgroups(dev::padded_dim(int(head_dim)), true, int(c.tile_heads / 16), true));
  c.workgroups = c.runs * pairs;
  return c;
}

int launch_paged_attention(const AttentionArgs& in, int dtype, int cache_dtype, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  AttentionArgs a = in;
  const int64_t rows = int64_t(a.table.batch) * a.heads;
  const int64_t chunks = (int64_t(a.max_len) + dev::kWeightRows - 1) / dev::kWeightRows;
  if (a.weights_out && !launchable(rows * chunks, dev::kWeightRows)) return TC_E_RANGE;
  const int dp = dev::padded_dim(a.head_dim);
  const int64_t pairs = int64_t(a.heads) * a.head_tiles;
  if (a.parts)
    a.runs = int32_t(runs_of(a.units, a.least_units, pairs,
                             dev::resident_workgroups(dp, cache_dtype == TC_E4M3, a.tile_heads / 16,
                                                      dev::pages_of_16(a.pool) && a.head_dim == dp)));
  if (!launchable(a.runs * pairs, dev::kAttnThreads)) return TC_E_RANGE;
  a.workgroups = int32_t(a.runs * pairs);
  a.pairs_div = make_div32(uint32_t(pairs));
  a.heads_div = make_div32(uint32_t(a.heads));
  a.parts_of_sequences = a.table.batch <= a.runs;
  const bool bf16 = dtype == TC_BF16, e4m3 = cache_dtype == TC_E4M3;
  if (bf16)
    e4m3 ? dev::by_dim<true, true>(a, s) : dev::by_dim<true, false>(a, s);
  else
    e4m3 ? dev::by_dim<false, true>(a, s) : dev::by_dim<false, false>(a, s);
  if (a.parts) {
    const dim3 grid(uint32_t(std::min(a.table.batch, a.runs)), uint32_t(a.heads) * uint32_t(a.group));
    if (bf16)
      hipLaunchKernelGGL(dev::paged_join_kernel<true>, grid, dim3(dev::kJoinThreads), 0, s, a);
    else
      hipLaunchKernelGGL(dev::paged_join_kernel<false>, grid, dim3(dev::kJoinThreads), 0, s, a);
  }
  if (a.weights_out && chunks > 0)
    hipLaunchKernelGGL(dev::paged_weights_kernel, dim3(uint32_t(rows * chunks)), dim3(dev::kWeightRows), 0, s, a,
                       make_div32(uint32_t(a.heads)), make_div32(uint32_t(chunks)));
  return TC_OK;
}

}  // namespace tc
