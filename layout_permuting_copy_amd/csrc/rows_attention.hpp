// Attention of several query rows a sequence: of whole prompts over packed keys and values, and of each sequence's last
// tokens over its paged cache.  The kernels, which the .hip files beside this one instantiate.
#pragma once

#include <algorithm>

#include "paged_common.hpp"

namespace tc {
namespace dev {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr int kRowsThreads = 256;
// The exponents' reference follows a row's maximum only where that has grown by more than this (base 2), so the output is
// rescaled in few tiles.  Weights of bf16 values are held at 2^-8 of what they are, at most 1 then: sums of weights times values
// pass fp32's range where those of exp(x - max x) |v| do, and no earlier (bf16 holds such weights as exactly).  Not those of
// 8-bit rows, which are multiplied by their scales before they are rounded to bf16: at 2^-8 scales below 2^-114 would lose bits.
// A reference that does not lag has neither end's loss, and takes 6 to 10 % (16 trees of 12 tokens over 8192 rows: 127 -> 140 us).
constexpr int kSlackBits = 8;
constexpr float kSlack = kSlackBits;

// D = A B + C on 32 x 32 tiles with a contraction of 16.  Lane l (r = l % 32, h = l / 32) holds row r of A and column r of
// B at contraction indices 8 h .. 8 h + 7, and of C and D column r at rows 8 (i / 4) + 4 h + i % 4, i = 0 .. 15.
template <bool BF16>
__device__ __forceinline__ f32x16 mfma32(const u32x4& a, const u32x4& b, const f32x16& c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// 4 x 16 values of 16 bits, transposed on their way out of LDS: of 16 lanes, lane i reads columns 4 (i % 4) .. + 3 of row i / 4
// and receives column i.
typedef __attribute__((address_space(3))) s16x4* LdsQuad;
__device__ __forceinline__ u32x2 read_transposed(const unsigned char* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsQuad)(p)));
}

// The same of 8 x 16 values of 8 bits: lane i reads columns 8 (i % 2) .. + 7 of row i / 2.
typedef __attribute__((address_space(3))) i32x2* LdsPair;
__device__ __forceinline__ u32x2 read_transposed8(const unsigned char* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((LdsPair)(p)));
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}

// 16 bytes a lane from memory straight into LDS, at `lds` + 16 * lane, of the lanes that are on.  Nothing waits for them but
// loads_landed() (the compiler knows of no register that they write, and what it waits for on its own account is older).  Of a
// range: its scalar registers and offset may come from a vector instruction (read-lane) right before, and the compiler does not look
// inside: a load reads them five wait states later at least, which the move and the pause after it are.
// m0 is named because the compiler sets it too, for itself, and merges equal settings; that it is reserved is what it warns of.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void to_lds(const u32x4& rsrc, uint32_t offset, uint32_t more, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(__builtin_amdgcn_readfirstlane(int(lds))), "v"(offset), "s"(rsrc),
                  "s"(__builtin_amdgcn_readfirstlane(int(more))) : "memory", "m0");
}
__device__ __forceinline__ u32x4 range_of(const unsigned char* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  return u32x4{uint32_t(__builtin_amdgcn_readfirstlane(int(p))), uint32_t(__builtin_amdgcn_readfirstlane(int(p >> 32))) & 0xffffu,
               uint32_t(__builtin_amdgcn_readfirstlane(int(bytes))), uint32_t(kRsrcWord3)};
}
__device__ __forceinline__ void to_lds(const unsigned char* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" :: "s"(__builtin_amdgcn_readfirstlane(int(lds))), "v"(p) : "memory", "m0");
}
// (4 bytes a lane)
__device__ __forceinline__ void to_lds(const float* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" :: "s"(__builtin_amdgcn_readfirstlane(int(lds))), "v"(p) : "memory", "m0");
}
#pragma clang diagnostic pop
__device__ __forceinline__ void loads_landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ int64_t lane_of(int64_t x, int lane) {
  return int64_t(uint64_t(uint32_t(__builtin_amdgcn_readlane(int(x >> 32), lane))) << 32 |
                 uint32_t(__builtin_amdgcn_readlane(int(x), lane)));
}

// Whether any lane's is true, as a number that all have.
__device__ __forceinline__ uint32_t any_lane(bool x) {
  const uint64_t lanes = __ballot(x);
  return uint32_t(lanes) | uint32_t(lanes >> 32);
}

// x *= f where `need` (the same in all lanes).  A branch of the compiler's would have x in registers twice, before it and after;
// this one leaves it where it is.  x is the matrix unit's: its last write may still be on its way (18 cycles are enough), and its next read comes after ours.
__device__ __forceinline__ void scale_if(f32x16& x, float f, uint32_t need) {
  float x0 = x[0], x1 = x[1], x2 = x[2], x3 = x[3], x4 = x[4], x5 = x[5], x6 = x[6], x7 = x[7],
        x8 = x[8], x9 = x[9], x10 = x[10], x11 = x[11], x12 = x[12], x13 = x[13], x14 = x[14], x15 = x[15];
  asm("s_cmp_eq_u32 %17, 0\n\ts_cbranch_scc1 1f\n\ts_nop 15\n\ts_nop 7\n\t"
        "v_mul_f32 %0, %16, %0\n\tv_mul_f32 %1, %16, %1\n\tv_mul_f32 %2, %16, %2\n\tv_mul_f32 %3, %16, %3\n\t"
        "v_mul_f32 %4, %16, %4\n\tv_mul_f32 %5, %16, %5\n\tv_mul_f32 %6, %16, %6\n\tv_mul_f32 %7, %16, %7\n\t"
        "v_mul_f32 %8, %16, %8\n\tv_mul_f32 %9, %16, %9\n\tv_mul_f32 %10, %16, %10\n\tv_mul_f32 %11, %16, %11\n\t"
        "v_mul_f32 %12, %16, %12\n\tv_mul_f32 %13, %16, %13\n\tv_mul_f32 %14, %16, %14\n\tv_mul_f32 %15, %16, %15\n\t"
        "s_nop 7\n1:"
        : "+v"(x0), "+v"(x1), "+v"(x2), "+v"(x3), "+v"(x4), "+v"(x5), "+v"(x6), "+v"(x7),
          "+v"(x8), "+v"(x9), "+v"(x10), "+v"(x11), "+v"(x12), "+v"(x13), "+v"(x14), "+v"(x15)
        : "v"(f), "s"(need)
        : "scc");
  x = f32x16{x0, x1, x2, x3, x4, x5, x6, x7, x8, x9, x10, x11, x12, x13, x14, x15};
}

// Where a reference m c is this large or more, logits take the difference x - m before they take the factor: x c - (m c) leaves what
// rounding took of m c, half a step of it (2^-10 from here on; at 2^34 weights pass fp32's range, and m c itself may where m does not).
constexpr float kFar = 16384.0f;

// 2^-RAISE
template <int RAISE>
constexpr float unraise() {
  if constexpr (RAISE < 0) return float(1 << -RAISE);
  else return 1.0f / float(1 << RAISE);
}

// The log of a row's sum, by its maximum (of q k, before the scale) and its sum relative to that.
__device__ __forceinline__ float lse_of(float top, float sum, float scale) {
  return __builtin_fmaf(top, scale, __builtin_amdgcn_logf(sum) * 0.6931471805599453f);
}

// A sequence of the call: its query tokens [t0, t0 + n), its key rows (packed: from k0 on), m of them.
struct RowsSeq {
  int t0, n, k0, m;
};
__device__ __forceinline__ int within(int x, int lo, int hi) { return x < lo ? lo : x < hi ? x : hi; }
template <bool PAGED>
__device__ __forceinline__ RowsSeq rows_seq(const RowsArgs& a, int b) {
  RowsSeq s;
  s.t0 = within(a.starts[b], 0, a.tokens);
  s.n = within(a.starts[b + 1], s.t0, a.tokens) - s.t0;
  if constexpr (PAGED) {
    s.k0 = 0;
    s.m = paged_len(a.lens, b, a.max_len);
  } else {
    s.k0 = within(a.key_starts[b], 0, a.key_rows);
    s.m = within(a.key_starts[b + 1], s.k0, a.key_rows) - s.k0;
  }
  return s;
}

// The sum over all lanes, in all of them.
__device__ __forceinline__ uint32_t wave_sum(uint32_t x) { return uint32_t(__builtin_amdgcn_readlane(int(wave_scan(x)), 63)); }

// How the call is dealt out: a sequence's query rows (its tokens times the heads of a group, token by token) in tiles of
// BM, its key rows in units of KT.  Where the tiles alone would leave the card idle (a.slots), each tile is split over the
// units: a part takes as few as make all parts of all tiles and heads fit the workgroups that the card holds at once (or
// twice, thrice as many where the tiles alone are more), and the parts of a sequence are equally long.  Work item i of the
// walk is a part of a tile; a sequence's items are its tiles' first parts, their second ones, and so on.
template <bool PAGED, int BM, int KT>
struct RowsWalk {
  int per;       // sequences a lane looks after
  RowsSeq mine;  // where that is one
  uint32_t most; // units of a part
  __device__ __forceinline__ RowsSeq seq(const RowsArgs& a, int lane, int k) const {
    return per == 1 ? mine : rows_seq<PAGED>(a, lane * per + k);
  }
  __device__ __forceinline__ uint32_t tiles(const RowsArgs& a, const RowsSeq& s) const {
    return uint32_t(s.n * a.group + BM - 1) / BM;
  }
  __device__ __forceinline__ uint32_t units(const RowsSeq& s) const { return s.m > 0 ? uint32_t(s.m + KT - 1) / KT : 1u; }
  // ceil(x / y) of numbers below 2^25: the quotient in fp32 is off by one at most
  static __device__ __forceinline__ uint32_t quotient(uint32_t x, uint32_t y) {
    uint32_t q = uint32_t(float(x) * __builtin_amdgcn_rcpf(float(y)));
    if (q * y < x) ++q;
    if (q * y < x) ++q;
    return q && (q - 1) * y >= x ? q - 1 : q;
  }
  __device__ __forceinline__ uint32_t parts(const RowsArgs& a, const RowsSeq& s, uint32_t units_each) const {
    return a.slots ? quotient(units(s), units_each) : 1u;
  }
  __device__ __forceinline__ uint32_t parts(const RowsArgs& a, const RowsSeq& s) const { return parts(a, s, most); }
  // of this lane's sequences: items, where a part has that many units
  __device__ __forceinline__ uint32_t items(const RowsArgs& a, int lane, uint32_t units_each) const {
    uint32_t sum = 0;
    for (int k = 0; k < per && lane * per + k < a.batch; ++k) {
      const RowsSeq s = seq(a, lane, k);
      sum += tiles(a, s) * parts(a, s, units_each);
    }
    return sum;
  }
  // SEARCH: finds `most`, else it is what the workgroups of the attention found
  template <bool SEARCH>
  __device__ __forceinline__ void init(const RowsArgs& a) {
    const int lane = threadIdx.x & 63;
    per = (a.batch + 63) / 64;
    mine = RowsSeq{};
    if (per == 1 && lane < a.batch) mine = rows_seq<PAGED>(a, lane);
    most = 1;
    if (!a.slots) return;
    if constexpr (!SEARCH) {
      most = uint32_t(__builtin_amdgcn_readfirstlane(int(*a.part_units)));
      return;
    }
    uint32_t sum = 0, longest = 1;
    float work = 0.0f;
    for (int k = 0; k < per && lane * per + k < a.batch; ++k) {
      const RowsSeq s = seq(a, lane, k);
      sum += tiles(a, s);
      work += float(tiles(a, s)) * float(units(s));
      if (s.n > 0 && units(s) > longest) longest = units(s);
    }
    sum = wave_sum(sum) * uint32_t(a.heads);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      work += __shfl_xor(work, d, 64);
      const uint32_t other = uint32_t(__shfl_xor(int(longest), d, 64));
      longest = other > longest ? other : longest;
    }
    // places: a multiple of the slots; the least units a part that they allow lies between those that would fill them
    // evenly and the longest sequence's
    const uint32_t slots = uint32_t(a.slots), places = (sum + slots - 1) / slots * slots, fit = places / uint32_t(a.heads);
    uint32_t lo = uint32_t(work / float(fit)), hi = longest;
    if (lo < uint32_t(a.least)) lo = uint32_t(a.least);
    if (lo < 1) lo = 1;
    if (hi < lo) hi = lo;
    lo = uint32_t(__builtin_amdgcn_readfirstlane(int(lo))), hi = uint32_t(__builtin_amdgcn_readfirstlane(int(hi)));
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (wave_sum(items(a, lane, mid)) <= fit) hi = mid;
      else lo = mid + 1;
    }
    most = hi;
  }
  // Finds sequence and place of tile x of many sequences': those of sequence b are numbered from (its first row
  // over all sequences) / BM + b on.  Up to the next sequence's that leaves room for all of them, at most one number more, and
  // the numbers ascend with b: the 64 lanes look for x's sequence in log64 of their count steps.
  static __device__ __forceinline__ uint32_t place(const RowsArgs& a, int b) {
    return uint32_t(within(a.starts[b], 0, a.tokens) * a.group) / BM + uint32_t(b);
  }
  __device__ __forceinline__ bool find_among_many(const RowsArgs& a, uint32_t x, int* b, uint32_t* at, RowsSeq* s) const {
    const int lane = threadIdx.x & 63;
    int lo = 0, span = a.batch;
    while (span > 1) {
      const int step = (span + 63) / 64, probe = lane * step;
      const int k = __popcll(__ballot(probe < span && place(a, lo + probe) <= x)), skip = k > 1 ? (k - 1) * step : 0;
      lo += skip;
      span = step < span - skip ? step : span - skip;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    const RowsSeq q = rows_seq<PAGED>(a, lo);
    s->t0 = __builtin_amdgcn_readfirstlane(q.t0), s->n = __builtin_amdgcn_readfirstlane(q.n);
    s->k0 = __builtin_amdgcn_readfirstlane(q.k0), s->m = __builtin_amdgcn_readfirstlane(q.m);
    *b = lo;
    *at = x - uint32_t(__builtin_amdgcn_readfirstlane(int(place(a, lo))));
    return *at < tiles(a, *s);
  }
  // Finds sequence and place of item x (REVERSED: counted from the last; ITEMS: parts of tiles, else tiles); `first`: the
  // number of the sequence's first item of parts.
  template <bool REVERSED, bool ITEMS>
  __device__ __forceinline__ bool find(const RowsArgs& a, uint32_t x, int* b, uint32_t* at, uint32_t* first, RowsSeq* s) const {
    const int lane = threadIdx.x & 63;
    uint32_t sum = 0, all = 0;
    for (int k = 0; k < per && lane * per + k < a.batch; ++k) {
      const RowsSeq q = seq(a, lane, k);
      const uint32_t t = tiles(a, q), p = t * parts(a, q);
      sum += ITEMS ? p : t;
      all += p;
    }
    const uint32_t upto = wave_scan(sum), total = uint32_t(__builtin_amdgcn_readlane(int(upto), 63));
    const uint32_t before_all = ITEMS ? upto - sum : wave_scan(all) - all;
    if (x >= total) return false;
    if (REVERSED && !a.slots) x = total - 1 - x;
    // the lanes whose sequences all come before x
    const int l = __popcll(__ballot(upto <= x));
    uint32_t rest = x - uint32_t(__builtin_amdgcn_readlane(int(upto - sum), l));
    uint32_t items = uint32_t(__builtin_amdgcn_readlane(int(before_all), l));
    for (int k = 0;; ++k) {
      RowsSeq q = mine;
      if (per == 1) {
        q.t0 = __builtin_amdgcn_readlane(q.t0, l), q.n = __builtin_amdgcn_readlane(q.n, l);
        q.k0 = __builtin_amdgcn_readlane(q.k0, l), q.m = __builtin_amdgcn_readlane(q.m, l);
      } else {
        q = rows_seq<PAGED>(a, l * per + k);
        q.t0 = __builtin_amdgcn_readfirstlane(q.t0), q.n = __builtin_amdgcn_readfirstlane(q.n);
        q.k0 = __builtin_amdgcn_readfirstlane(q.k0), q.m = __builtin_amdgcn_readfirstlane(q.m);
      }
      const uint32_t t = tiles(a, q), p = t * parts(a, q), w = ITEMS ? p : t;
      if (rest < w || k + 1 >= per) {
        *b = l * per + k, *at = rest, *first = items, *s = q;
        return rest < w;
      }
      rest -= w;
      items += p;
    }
  }
};

// The `count` lowest bits (all below 1, none from 32 on: as a mask of 32 rows).
__device__ __forceinline__ uint32_t low_bits(int count) {
  return count <= 0 ? 0u : count >= 32 ? ~0u : (1u << count) - 1u;
}

// Where exponents are all ones (infinities, NaN) in a pair of 16-bit values: 0xffff in that half.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  const uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
  return ((w & e) == e ? 0xffffu : 0u) | ((w >> 16 & e) == e ? 0xffff0000u : 0u);
}

// The same of the NaN codes among four 8-bit values.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 32; i += 8) bad |= (w >> i & 0x7fu) == 0x7fu ? 0xffu << i : 0u;
  return bad;
}

// SRC: 0 packed rows, 1 a paged cache of 16-bit rows, 2 of 8-bit rows.  DP: head_dim rounded up.  WQ of the workgroup's waves
// take 32 query rows each, WAVES / WQ groups of waves share the key rows.  PARTS: 16-bit values that hold a weight.
template <bool BF16, int SRC, int DP, int WQ, int WAVES_, int PARTS>
struct Rows {
  static constexpr bool PAGED = SRC != 0, E4M3 = SRC == 2, VBF = BF16 || E4M3;
  static constexpr int WAVES = WAVES_, THREADS = 64 * WAVES;
  static constexpr int NG = WAVES / WQ;
  static constexpr int KT = 64;                      // key rows a turn
  static constexpr int NSUB = KT / 32 / NG;          // of them a wave's, 32 at a time
  static constexpr int NJ = DP > 128 || E4M3 ? 1 : NSUB;  // of these at once: what the registers hold
  static constexpr int BM = 32 * WQ;
  static constexpr int EB = E4M3 ? 1 : 2;
  static constexpr int PITCH = DP <= 64 ? 64 : DP <= 128 ? 128 : 256;  // elements a row has in LDS
  static constexpr int PB = PITCH * EB;
  static constexpr int KS = DP / 16, NF = DP / 32;
  static constexpr int CPR = PB / 16;             // lanes that load a row, 16 bytes each
  static constexpr int RPW = 64 / CPR;            // rows a wave loads at once
  static constexpr int RPP = WAVES * RPW;             // and a workgroup
  static constexpr int PASSES = KT / RPP;
  // weights are held 2^RAISE as large: fp16 ones above where its numbers grow coarse
  static constexpr int RAISE = E4M3 ? 0 : BF16 ? -kSlackBits : 7;
  static constexpr int TILE_BYTES = KT * PB, PASS_BYTES = 1024 * WAVES;
  static_assert(NSUB >= 1 && RPP % 16 == 0, "a wave has 32 key rows at least, a pass rows of the same exchange");
  // where the groups of waves meet: all but the first leave their outputs in LDS
  static constexpr int MEET_BYTES = (WAVES - WQ) * 32 * DP * 4;
  static constexpr int LDS_BYTES = 4 * TILE_BYTES > MEET_BYTES ? 4 * TILE_BYTES : MEET_BYTES;
  // Workgroups that a compute unit holds: eight waves, two a SIMD, that hide each other's waits.  (With one a SIMD and twice
  // the registers half of those are the matrix unit's own, and what has to be moved out of them and back costs more.)
  // Narrow heads of caches leave room for three (32 trees of 8 tokens, heads of 64: 68 -> 65 us).
  static constexpr int RESIDENT = WAVES == 8 ? 1 : PAGED && DP == 64 ? 3 : 2;
  static_assert(RESIDENT * LDS_BYTES <= 150 * 1024, "they share 160 KB of LDS");

  // Which 16-byte chunk of a row lies at place c of its row in LDS, and the other way round (an exchange): the rows that one
  // access reads at the same chunk, sixteen of keys (16 bytes a lane) and four or, of 8-bit values, eight (transposed, half a
  // chunk a lane), lie in different banks.
  static constexpr int KX = CPR < 16 ? CPR : 16;  // chunks that a key row's exchange covers: 16 rows at 16 places
  static __device__ __forceinline__ int key_chunk(int row, int c) { return c ^ (row / (PB < 256 ? 256 / PB : 1) & (KX - 1)); }
  static __device__ __forceinline__ int value_chunk(int row, int c) {
    if constexpr (E4M3) return c ^ (PB == 64 ? (row >> 3 & 1) << 1 : (row & 3) | (row >> 3 & 1) << 2);
    return c ^ (PB == 128 ? row >> 1 & 1 : row & 3) << 2;
  }
  // The element of a row that contraction index 8 hl + j of step k stands for (j = 0): 16 bytes of a key row serve one step, or
  // two of 8-bit elements.
  static __device__ __forceinline__ int q_element(int k, int hl) {
    return E4M3 ? (k >> 1) * 32 + hl * 16 + (k & 1) * 8 : k * 16 + hl * 8;
  }
};

// One pass over a tile's keys with the running maximum m and sum l of a softmax: x = q k, P = exp2(c (x - m)), O <- O f + P V,
// l <- l f + sum P, where f = exp2(c (m_old - m)).  A wave's lanes hold a query row each, twice: S^T = K Q^T leaves a lane
// half of its row's logits in the layout that O^T = V^T P^T takes its weights in, so maxima and sums need one exchange
// of halves and weights none.  Keys and values go to LDS without passing through registers, a unit of 64 rows ahead, and are read
// there without bank conflicts, values transposed on the way out.  All waves share the unit; where there are fewer tiles of
// 32 query rows than waves, groups of waves share out its rows and meet at the end.
// Bound: with prompts and chunks the matrix products and the softmax's vector instructions in turn (16384 causal tokens, 32
// heads of 128 over 8: 2080 us, 1057 TFLOP/s; the matrix units are busy 51 % of the time, vector instructions issue in 42 %,
// which leaves 7 % of waits; two waves a SIMD that take turns by barriers, one multiplying while the other softens, came to
// 2371 us, as a wave alone does not hide the reads of its operands); trees of few tokens by what a CU has in flight (32 trees of 8
// tokens over 4096 rows: 115 us, 4.7 TB/s); 8-bit caches by the conversions (16 trees of 12 tokens over 8192 rows: 127 us).
// MANY: of many sequences (RowsWalk::find_among_many), a kernel of its own, as the others' scalar registers do not suffice for
// both ways (32 trees of 26 tokens 62 us, in such a kernel 67).
template <bool BF16, int SRC, int DP, int WQ, int WAVES_, int PARTS, bool MANY>
__global__ __launch_bounds__(64 * WAVES_, (Rows<BF16, SRC, DP, WQ, WAVES_, PARTS>::RESIDENT * WAVES_ / 4))
void rows_attention_kernel(RowsArgs a) {
  typedef Rows<BF16, SRC, DP, WQ, WAVES_, PARTS> C;
  constexpr bool PAGED = C::PAGED, E4M3 = C::E4M3, VBF = C::VBF;
  constexpr int KT = C::KT, NSUB = C::NSUB, NJ = C::NJ, BM = C::BM, KS = C::KS, NF = C::NF, PB = C::PB, NG = C::NG, PASSES = C::PASSES;
  __shared__ __attribute__((aligned(16))) unsigned char lds[C::LDS_BYTES];
  __shared__ float scales[E4M3 ? 2 : 1][2][E4M3 ? KT : 1];
  __shared__ float meet_ml[NG == 1 ? 1 : C::WAVES - WQ][2][64];
  __shared__ int strange[C::WAVES];  // by wave: of a tile with rows that are not seen, some values are not finite

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, hl = lane >> 5;
  const uint32_t x = udiv(blockIdx.x, a.heads_div);
  const int h = int(blockIdx.x - x * a.heads_div.d);

  RowsWalk<PAGED, BM, KT> walk;
  int b;
  uint32_t at, first;
  RowsSeq seq;
  if constexpr (MANY) {
    if (!walk.find_among_many(a, PAGED ? x : uint32_t(a.tiles) - 1 - x, &b, &at, &seq)) return;
  } else {
    walk.template init<true>(a);
    if (a.slots && blockIdx.x == 0 && tid == 0) *a.part_units = walk.most;
    if (!walk.template find<!PAGED, true>(a, x, &b, &at, &first, &seq)) return;
  }
  const int tiles = int(walk.tiles(a, seq)), parts = MANY ? 1 : __builtin_amdgcn_readfirstlane(int(walk.parts(a, seq)));
  const int part = parts > 1 ? int(at / uint32_t(tiles)) : 0, tile = int(at) - part * tiles;
  const int rows = seq.n * a.group, row0 = tile * BM;
  const int off = seq.m - seq.n;  // token i's own row
  const int last_row = rows - 1 < row0 + BM - 1 ? rows - 1 : row0 + BM - 1;
  const int tok_lo = int(udiv(uint32_t(row0), a.group_div)), tok_hi = int(udiv(uint32_t(last_row), a.group_div));
  const bool chain = a.causal && !a.masks;
  // rows from `end` on are seen by no query of the tile, rows below `clear` by all of them
  const int end = chain ? within(off + tok_hi + 1, 0, seq.m) : seq.m;
  const int clear = a.causal ? (a.masks ? off : off + tok_lo + 1) : seq.m;
  const int units_all = (end + KT - 1) / KT;
  const int each = parts > 1 ? (int(walk.units(seq)) + parts - 1) / parts : units_all;
  const int u0 = part * each, u1 = u0 + each < units_all ? u0 + each : units_all;

  // this lane's query row (what was loaded is put right below, when the first keys and values are on their way)
  const int wq = wave % WQ, wg = wave / WQ;
  u32x4 q[KS];
  const auto load_queries = [&] {
    const int row = row0 + wq * 32 + r;
    const uint32_t rr = uint32_t(row < rows ? row : rows - 1);
    const int tok = int(udiv(rr, a.group_div)), g = int(rr) - tok * a.group;
    const unsigned char* at = a.q + int64_t(seq.t0 + tok) * a.qt + (int64_t(h) * a.group + g) * a.qh;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int e = C::q_element(k, hl);
      q[k] = *reinterpret_cast<const u32x4*>(at + (e < a.head_dim ? 2 * e : 0));
    }
  };
  const float c = a.scale_log2e;

  // two buffers of keys and values
  const auto keys_of = [](int buf) { return buf * 2 * C::TILE_BYTES; };
  const auto values_of = [](int buf) { return buf * 2 * C::TILE_BYTES + C::TILE_BYTES; };
  const uint32_t lds0 = lds_address(lds) + wave * 1024;
  if (DP < C::PITCH || a.head_dim < DP) {  // what lies past head_dim is zero for good
    for (int i = tid; i < 4 * C::TILE_BYTES / 16; i += C::THREADS) reinterpret_cast<u32x4*>(lds)[i] = u32x4{};
    __syncthreads();
  }

  int entry = 0;         // the table's for row `lane` of the next unit
  uint64_t missing = 0;  // rows of the unit requested that do not exist
  const auto load_entry = [&](int u) {
    if constexpr (PAGED) {
      int row = u * KT + lane;
      if (row >= seq.m) row = seq.m - 1;
      entry = a.table.p[int64_t(b) * a.table.sb + int64_t(udiv(uint32_t(row), a.pool.div)) * a.table.sc];
    }
  };
  // Where key row `key` lies, by its table entry (no page: page 0).
  struct Place {
    int page;
    int64_t in_page;
  };
  const auto place_of = [&](int key, int e) {
    return Place{uint32_t(e) < uint32_t(a.pool.pages) ? e : 0,
                 int64_t(uint32_t(key) - udiv(uint32_t(key), a.pool.div) * a.pool.div.d)};
  };
  // Requests unit u; of rows past the end: zeros (packed: outside the range, which counts the scalar offset) or the last one.  Rows go from memory into LDS as they are, a wave's lanes side by
  // side: what is exchanged is which chunk a lane loads.
  // (the rows that a wave loads at once lie on one page: its address is the wave's)
  const bool page_wise = PAGED && a.pool.page_size % C::RPW == 0 && a.pool.kr < 1 << 26 && a.pool.vr < 1 << 26;
  const auto request = [&](int u, int buf) {
    // this lane's row of a pass, its chunks of keys and of values (for wide heads found anew each time, for the registers' sake)
    const int ln = DP > 128 ? fresh(lane) : lane, up = ln / C::CPR, srow = wave * C::RPW + up;
    const int kc = C::key_chunk(srow, ln % C::CPR) * 16, vc = C::value_chunk(srow, ln % C::CPR) * 16;
    const bool k_in = kc < a.head_dim * C::EB, v_in = vc < a.head_dim * C::EB;
    const uint32_t lk = lds0 + keys_of(buf), lv = lds0 + values_of(buf);
    if constexpr (!PAGED) {
      const int left = seq.m - u * KT, rows_here = left < KT ? left : KT;
      const int64_t from = int64_t(seq.k0 + u * KT);
      const u32x4 rk = range_of(a.k + from * a.kt + int64_t(h) * a.kh, uint32_t((rows_here - 1) * a.kt) + a.head_dim * 2);
      const u32x4 rv = range_of(a.v + from * a.vt + int64_t(h) * a.vh, uint32_t((rows_here - 1) * a.vt) + a.head_dim * 2);
      const uint32_t kt = uint32_t(a.kt), vt = uint32_t(a.vt);
      if (k_in)
#pragma unroll
        for (int p = 0; p < PASSES; ++p) to_lds(rk, up * kt + kc, (p * C::RPP + wave * C::RPW) * kt, lk + p * C::PASS_BYTES);
      if (v_in)
#pragma unroll
        for (int p = 0; p < PASSES; ++p) to_lds(rv, up * vt + vc, (p * C::RPP + wave * C::RPW) * vt, lv + p * C::PASS_BYTES);
    } else {
      missing = __ballot(u * KT + lane >= seq.m || uint32_t(entry) >= uint32_t(a.pool.pages));
      const unsigned char* const hk = a.pool.k + int64_t(h) * a.pool.kh;
      const unsigned char* const hv = a.pool.v + int64_t(h) * a.pool.vh;
      if (page_wise) {
        // Lane i finds where row i lies (past the end: the last rows that a wave loads at once), the wave's rows are a lane's.
        const int key = u * KT + lane < seq.m ? u * KT + lane : (seq.m - 1) & ~(C::RPW - 1);
        const Place at = place_of(key, entry);
        const int64_t k_at = at.page * a.pool.kp + at.in_page * a.pool.kr, v_at = at.page * a.pool.vp + at.in_page * a.pool.vr;
        const uint32_t ko = up * uint32_t(a.pool.kr) + kc, vo = up * uint32_t(a.pool.vr) + vc;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          const int row = p * C::RPP + wave * C::RPW;
          const u32x4 rk = range_of(hk + lane_of(k_at, row), 0x7fffffffu), rv = range_of(hv + lane_of(v_at, row), 0x7fffffffu);
          if (k_in) to_lds(rk, ko, 0, lk + p * C::PASS_BYTES);
          if (v_in) to_lds(rv, vo, 0, lv + p * C::PASS_BYTES);
        }
      } else {
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          const int row = p * C::RPP + srow, key = u * KT + row < seq.m ? u * KT + row : seq.m - 1;
          const Place at = place_of(key, __shfl(entry, row, 64));
          if (k_in) to_lds(hk + at.page * a.pool.kp + at.in_page * a.pool.kr + kc, lk + p * C::PASS_BYTES);
          if (v_in) to_lds(hv + at.page * a.pool.vp + at.in_page * a.pool.vr + vc, lv + p * C::PASS_BYTES);
        }
      }
      if constexpr (E4M3) {
        if (wave == 0) {
          const Place at = place_of(u * KT + lane < seq.m ? u * KT + lane : seq.m - 1, entry);
          to_lds(a.pool.ks + (at.page * a.pool.ksp + at.in_page * a.pool.ksr + int64_t(h) * a.pool.ksh), lds_address(scales[buf][0]));
          to_lds(a.pool.vs + (at.page * a.pool.vsp + at.in_page * a.pool.vsr + int64_t(h) * a.pool.vsh), lds_address(scales[buf][1]));
        }
      }
    }
  };
  // Sees to it that what was requested is in LDS.
  const auto settle = [] {
    loads_landed();
    __syncthreads();
  };
  const auto edge_of = [&](int u) {
    return (u + 1) * KT > clear || (u + 1) * KT > seq.m || missing != 0;
  };

  // (hl, found anew where that saves its register)
  const auto half = [&] { return MANY && DP > 192 ? fresh(int(threadIdx.x)) >> 5 & 1 : hl; };
  f32x16 o[NF];
  float m = -kInf, l = 0.0f;
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[f][i] = 0.0f;

  // What a lane reads of LDS, from a tile's first row of 32 (keys) or 16 (values) on.  Keys: row r, the 16 bytes of step k (of
  // two steps of 8-bit elements).  Values: see read_transposed; the rows of a lane's element j are 4 hl + j (j < 4) and
  // 4 hl + 8 + j - 4, which is how S^T's rows lie in registers
  // (the exchanges stay among the chunks that the bases cover; the widest rows leave no registers for more than the first,
  // which is found anew for each product)
  constexpr int KB = C::KX / 2;
  constexpr bool EXCHANGE = DP > 192;
  // 8-bit tiles of 32 rows are in registers, as codes, before the first product: their conversions do not wait for LDS (16
  // trees of 12 tokens, 8 heads a group, over 8192 rows: 164 -> 133 us)
  constexpr bool EARLY = E4M3 && DP <= 128;
  struct Bases {
    int k[EXCHANGE ? 1 : KB], v[EXCHANGE ? 1 : 4];
  };
  const auto bases_of = [](int ln) {
    Bases x;
    const int hl = ln >> 5, i = ln & 15, g = ln >> 4 & 1;
#pragma unroll
    for (int j = 0; j < (EXCHANGE ? 1 : KB); ++j) x.k[j] = (ln & 31) * PB + C::key_chunk(ln & 31, 2 * j + hl) * 16;
#pragma unroll
    for (int j = 0; j < (EXCHANGE ? 1 : 4); ++j) {
      if constexpr (E4M3) {
        const int row = 4 * hl + (i >> 1 & 3) + (i >> 3) * 8;
        x.v[j] = row * PB + C::value_chunk(row, (2 * j + g) % C::CPR) * 16 + (i & 1) * 8;
      } else {
        const int row = 4 * hl + (i >> 2);
        x.v[j] = row * PB + C::value_chunk(row, (4 * j + 2 * g + (i >> 1 & 1)) % C::CPR) * 16 + (i & 1) * 8;
      }
    }
    return x;
  };
  Bases bases = bases_of(lane);
  const auto key_words = [&](const unsigned char* at, int j) {
    const int base = EXCHANGE ? bases.k[0] ^ j % KB * 32 : bases.k[EXCHANGE ? 0 : j % KB];
    return *reinterpret_cast<const u32x4*>(at + base + j / KB * 256);
  };
  const auto value_codes = [&](const unsigned char* at, int f) {
    return read_transposed8(at + (EXCHANGE ? bases.v[0] ^ (f & 3) * 32 : bases.v[EXCHANGE ? 0 : f & 3]) + (f >> 2) * 128);
  };
  const auto values_of_codes = [](const u32x2& w) {
    return u32x4{from_e4m3<true, false>(w[0]), from_e4m3<true, true>(w[0]), from_e4m3<true, false>(w[1]), from_e4m3<true, true>(w[1])};
  };
  const auto value_operand = [&](const unsigned char* at, int f) {
    if constexpr (E4M3) {
      return values_of_codes(value_codes(at, f));
    } else {
      const unsigned char* p = at + (EXCHANGE ? bases.v[0] ^ (f & 3) * 64 : bases.v[EXCHANGE ? 0 : f & 3]) + (f >> 2) * 256;
      const u32x2 lo = read_transposed(p), hi = read_transposed(p + 8 * PB);
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
  };

  bool edge = false;  // of the tile to be computed
  if (u0 < u1) {
    load_entry(u0);
    load_queries();
    request(u0, 0);
    edge = edge_of(u0);
    if (u0 + 1 < u1) load_entry(u0 + 1);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) q[k][i] = C::q_element(k, hl) < a.head_dim ? (q[k][i] & a.q_and) ^ a.q_xor : 0u;
    settle();
  }
#pragma unroll 1
  for (int u = u0; u < u1; ++u) {
    const int buf = (u - u0) & 1;
    const bool now_edge = edge, more = u + 1 < u1;
    const uint64_t now_missing = missing;
    if (more) {
      request(u + 1, buf ^ 1);
      edge = edge_of(u + 1);
      if (u + 2 < u1) load_entry(u + 2);
    }
    // which rows this lane's queries see: bit 8 (i / 4) + i % 4 for element i of S^T's 32 rows
    uint32_t seen[NSUB];
    if (now_edge) {
      // its last key row without masks, its mask (found anew in the few tiles that ask, for the registers' sake)
      const int mine_r = fresh(int(threadIdx.x)) & 31, my_row = row0 + wq * 32 + mine_r;
      const int my_tok = int(udiv(uint32_t(my_row < rows ? my_row : rows - 1), a.group_div));
      const int limit = chain && off + my_tok < seq.m ? off + my_tok : seq.m - 1;
      const uint64_t mask = PAGED && a.masks ? uint64_t(a.masks[seq.t0 + my_tok]) : 0;
#pragma unroll
      for (int n = 0; n < NSUB; ++n) {
        const int sub = wg * NSUB + n, key0 = u * KT + sub * 32;
        const uint32_t gone = PAGED ? uint32_t(now_missing >> sub * 32) : 0u;
        uint32_t w;
        if (PAGED && a.masks) {
          const int d = key0 - off;  // the first key's number among the drafted tokens
          w = d >= 64 ? 0u : d >= 0 ? uint32_t(mask >> d) : d <= -32 ? ~0u : uint32_t(mask << -d) | low_bits(-d);
          w &= low_bits(seq.m - key0);
        } else {
          w = low_bits(limit - key0 + 1);
        }
        seen[n] = (w & ~gone) >> 4 * half();
      }
      // A weight of 0 does not help against infinite or NaN values of rows that are not seen.  Where the tile has any,
      // each query's output first takes the infinities and NaN of the rows that it does see, as products of numbers that
      // overflow (both signs for a NaN); then they are zeros.
      u32x4* const mine = reinterpret_cast<u32x4*>(lds + values_of(buf)) + tid;
      uint32_t bad = 0;
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) bad |= E4M3 ? nan_codes(mine[p * C::THREADS][i]) : not_finite<BF16>(mine[p * C::THREADS][i]);
      const bool any = __ballot(bad != 0) != 0;
      if (lane == 0) strange[wave] = any;
      __syncthreads();
      int found = 0;
#pragma unroll
      for (int i = 0; i < C::WAVES; ++i) found |= strange[i];
      if (found) {
#pragma unroll 1
        for (int j = 0; j < 2 * NSUB; ++j) {
          const unsigned char* base = lds + values_of(buf) + (wg * NSUB * 2 + j) * 16 * PB;
          u32x4 big;  // 2^127 where a row is seen
          const uint32_t w = (NSUB > 1 && j >= 2 ? seen[NSUB - 1] : seen[0]) >> 16 * (j & 1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int bit = 8 * (i / 2) + 2 * i % 4;
            big[i] = (w >> bit & 1 ? 0x7f00u : 0u) | (w >> (bit + 1) & 1 ? 0x7f000000u : 0u);
          }
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            const u32x4 y = value_operand(base, f);
            u32x4 up, down;  // 2^127, -2^127 where the value is infinite, both where it is NaN
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t not_number = not_finite<VBF>(y[i]), frac = VBF ? 0x007fu : 0x03ffu;
              const uint32_t nan = ((y[i] & frac) ? 0xffffu : 0u) | ((y[i] >> 16 & frac) ? 0xffff0000u : 0u);
              const uint32_t minus = ((y[i] & 0x8000u) ? 0xffffu : 0u) | ((y[i] & 0x80000000u) ? 0xffff0000u : 0u);
              up[i] = 0x7f007f00u & not_number & (nan | ~minus);
              down[i] = 0xff00ff00u & not_number & (nan | minus);
            }
            o[f] = mfma32<true>(up, big, o[f]);
            o[f] = mfma32<true>(down, big, o[f]);
            __builtin_amdgcn_sched_barrier(0);  // one tile's registers at a time
          }
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          u32x4 w = mine[p * C::THREADS];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] &= ~(E4M3 ? nan_codes(w[i]) : not_finite<BF16>(w[i]));
          mine[p * C::THREADS] = w;
        }
        __syncthreads();
      }
    }

#pragma unroll 1
    for (int n0 = 0; n0 < NSUB; n0 += NJ) {
      const auto seen_of = [&](int n) { return NJ == NSUB ? seen[n] : n0 ? seen[NSUB - 1] : seen[0]; };
      if constexpr (EXCHANGE) bases = bases_of(fresh(int(threadIdx.x)) & 63);
      // S^T = K Q^T
      f32x16 s[NJ];
      u32x2 codes[EARLY ? 2 : 1][EARLY ? NF : 1];
#pragma unroll
      for (int n = 0; n < NJ; ++n) {
        const unsigned char* base = lds + keys_of(buf) + (wg * NSUB + n0 + n) * 32 * PB;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[n][i] = 0.0f;
        u32x4 early[EARLY ? KS / 2 : 1];
        if constexpr (EARLY) {
#pragma unroll
          for (int j = 0; j < KS / 2; ++j) early[j] = key_words(base, j);
          const unsigned char* values = lds + values_of(buf) + (wg * NSUB + n0 + n) * 32 * PB;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int f = 0; f < NF; ++f) codes[k][f] = value_codes(values + 16 * k * PB, f);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < (E4M3 ? KS / 2 : KS); ++j) {
          const u32x4 w = EARLY ? early[EARLY ? j : 0] : key_words(base, j);
#pragma unroll
          for (int half = 0; half < (E4M3 ? 2 : 1); ++half) {
            u32x4 y = w;
            if constexpr (E4M3) {
              const uint32_t lo = w[2 * half], hi = w[2 * half + 1];
              y = u32x4{from_e4m3<BF16, false>(lo), from_e4m3<BF16, true>(lo), from_e4m3<BF16, false>(hi), from_e4m3<BF16, true>(hi)};
            }
            s[n] = mfma32<BF16>(y, q[E4M3 ? 2 * j + half : j], s[n]);
          }
        }
      }

      // scales of the 8-bit rows, masks
      if constexpr (E4M3) {
#pragma unroll
        for (int n = 0; n < NJ; ++n)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(&scales[buf][0][(wg * NSUB + n0 + n) * 32 + 2 * i + 4 * half()]);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[n][i + j] *= x[j];
          }
      }
      if (now_edge) {
#pragma unroll
        for (int n = 0; n < NJ; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[n][i] = seen_of(n) >> (8 * (i / 4) + i % 4) & 1 ? s[n][i] : -kInf;
      }

      // the running softmax; P^T in B's layout as 16-bit parts
      u32x4 p[NJ][2][PARTS];
      float top = -kInf;
#pragma unroll
      for (int n = 0; n < NJ; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[n][i]);
      float other;
      partners<32>(top, &top, &other);
      top = __builtin_fmaxf(top, other);
      const uint32_t need = any_lane((top - m) * c > kSlack);
      const float to = need ? __builtin_fmaxf(top, m) : m;
      // (no row seen so far: there is nothing to shrink but infinities of values)
      const float shrink = !need || m == -kInf ? 1.0f : __builtin_amdgcn_exp2f((m - finite(to)) * c);
      l *= shrink;
      m = to;
      if constexpr (DP > 64) {
#pragma unroll
        for (int f = 0; f < NF; ++f) scale_if(o[f], shrink, need);
      } else if (need) {
#pragma unroll
        for (int f = 0; f < NF; ++f) o[f] *= shrink;
      }
      // far from zero (keys of the type's lowest value) the difference comes first
      float ref = m * c;
      if (any_lane(__builtin_fabsf(ref) >= kFar && __builtin_fabsf(m) < kInf)) {
#pragma unroll
        for (int n = 0; n < NJ; ++n) s[n] -= finite(m);
        ref = 0.0f;
      }
      ref = finite(ref);
      if constexpr (C::RAISE < 0) ref -= C::RAISE;  // (a reference like another: sums of weights are relative to it as well)
      constexpr int CHAINS = DP > 128 ? 1 : 4;  // of additions
      float sum[CHAINS] = {l};
      const auto weight = [&](int n, int i) {
        float e = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][i], c, -ref));
        if constexpr (C::RAISE > 0) e *= float(1 << C::RAISE);
        sum[i % CHAINS] += e;
        return e;
      };
      if constexpr (E4M3) {
#pragma unroll
        for (int n = 0; n < NJ; ++n) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(&scales[buf][1][(wg * NSUB + n0 + n) * 32 + 2 * i + 4 * half()]);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[n][i + j] = weight(n, i + j) * x[j];
          }
          if (now_edge) {  // (0 times a scale that is no number)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[n][i] = seen_of(n) >> (8 * (i / 4) + i % 4) & 1 ? s[n][i] : 0.0f;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NJ; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = E4M3 ? s[n][8 * k + i] : weight(n, 8 * k + i);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = e[2 * i], y = e[2 * i + 1];
#pragma unroll
            for (int z = 0; z < PARTS; ++z) {
              const uint32_t w = p[n][k][z][i] = pack2<VBF>(x, y);
              x -= low_half<VBF>(w);
              y -= high_half<VBF>(w);
            }
          }
          if constexpr (DP > 192 && PARTS > 1) __builtin_amdgcn_sched_barrier(0);
        }

      if constexpr (DP > 192) __builtin_amdgcn_sched_barrier(0);  // (one product's registers at a time)
      l = CHAINS == 1 ? sum[0] : (sum[0] + sum[1 % CHAINS]) + (sum[2 % CHAINS] + sum[3 % CHAINS]);

      if constexpr (EXCHANGE) bases = bases_of(fresh(int(threadIdx.x)) & 63);
      // O^T += V^T P^T
#pragma unroll
      for (int n = 0; n < NJ; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const unsigned char* base = lds + values_of(buf) + ((wg * NSUB + n0 + n) * 32 + 16 * k) * PB;
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            const u32x4 y = EARLY ? values_of_codes(codes[EARLY ? k : 0][EARLY ? f : 0]) : value_operand(base, f);
#pragma unroll
            for (int z = 0; z < PARTS; ++z) o[f] = mfma32<VBF>(y, p[n][k][z], o[f]);
          }
        }
    }

    if (more) settle();
  }

  // a lane's sums are of half its rows' keys
  {
    float y, z;
    partners<32>(l, &y, &z);
    l = y + z;
  }
  // (a lane's place as if it were new: what follows from it is not kept in registers through the loop)
  const int end_tid = fresh(int(threadIdx.x)), end_lane = end_tid & 63, end_r = end_tid & 31, end_hl = end_tid >> 5 & 1;
  if constexpr (NG > 1) {
    // the groups of waves meet: equal lanes hold the same query row and elements
    float* const meet = reinterpret_cast<float*>(lds);
    __syncthreads();  // the last tile has been read
    if (wg > 0) {
      const int at = wave - WQ;
      meet_ml[at][0][end_lane] = m, meet_ml[at][1][end_lane] = l;
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<f32x4*>(meet + ((at * NF + f) * 4 + i / 4) * 256 + end_lane * 4) = f32x4{o[f][i], o[f][i + 1], o[f][i + 2], o[f][i + 3]};
    }
    __syncthreads();
    if (wg > 0) return;
    float top = m;
#pragma unroll
    for (int k = 1; k < NG; ++k) top = __builtin_fmaxf(top, meet_ml[(k - 1) * WQ + wq][0][end_lane]);
    const float ref = finite(top), own = __builtin_amdgcn_exp2f((m - ref) * c);
    l *= own;
#pragma unroll
    for (int f = 0; f < NF; ++f) o[f] *= own;
#pragma unroll
    for (int k = 1; k < NG; ++k) {
      const int at = (k - 1) * WQ + wq;
      const float theirs = __builtin_amdgcn_exp2f((meet_ml[at][0][end_lane] - ref) * c);
      l += meet_ml[at][1][end_lane] * theirs;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const f32x4 x = *reinterpret_cast<const f32x4*>(meet + ((at * NF + f) * 4 + i / 4) * 256 + end_lane * 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float y = o[f][i + j] + x[j] * theirs;
            if constexpr (MANY && DP > 192) asm volatile("" : "+v"(y));  // (now, not behind the stores before it: x's registers)
            o[f][i + j] = y;
          }
        }
      }
    }
    m = top;
  }
  const int local = wq * 32 + end_r, row = row0 + local;
  const bool real = row < rows;
  if (parts > 1) {
    const int64_t slot = int64_t(blockIdx.x) * BM + local;
    if (end_hl == 0) a.part_ml[2 * slot] = m, a.part_ml[2 * slot + 1] = l;
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 32 * f + 8 * i + 4 * end_hl;
        f32x4 y;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = o[f][4 * i + j];
        if (real && d < a.head_dim) *reinterpret_cast<f32x4*>(a.part_o + slot * a.head_dim + d) = y;
      }
    return;
  }
  const int tok = int(udiv(uint32_t(real ? row : rows - 1), a.group_div)), g = (real ? row : rows - 1) - tok * a.group;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  unsigned char* out = a.out + int64_t(seq.t0 + tok) * a.ot + (int64_t(h) * a.group + g) * a.oh;
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // elements 32 f + 16 i + 8 y + 4 hl + j, y = 0, 1: the halves exchange so that each lane has eight neighbours
      u32x2 w[2];
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int j = 0; j < 2; ++j) w[y][j] = pack2<BF16>(o[f][8 * i + 4 * y + 2 * j] * inv, o[f][8 * i + 4 * y + 2 * j + 1] * inv);
      const auto e0 = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
      const auto e1 = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
      const int d = 32 * f + 16 * i + 8 * end_hl;
      if (real && d < a.head_dim) *reinterpret_cast<u32x4*>(out + 2 * d) = u32x4{e0[0], e1[0], e0[1], e1[1]};
    }
  if (a.lse && real && end_hl == 0)
    a.lse[int64_t(seq.t0 + tok) * a.lt + (int64_t(h) * a.group + g) * a.lh] = lse_of(m, l * unraise<C::RAISE>(), a.scale);
}

// The parts of a tile's query rows joined, a few lanes a row (32, or 64 above 128 elements): the parts' maxima give their
// factors, sums and outputs are added in the parts' order.  Grid: tiles, heads, a tile's rows 16 at a time; tiles in one part
// end at once.  Bound: its launch and three trips to memory one after another (lengths; the parts' sums and first outputs
// together; the rest); 34 MB of parts of 32 trees 9.7 us, 14.3 where every row's sums were waited for before its outputs.
constexpr int kJoinRows = 16;
template <bool BF16, bool PAGED, int DP, int BM, int KT, int RAISE>
__global__ __launch_bounds__(kRowsThreads) void rows_join_kernel(RowsArgs a) {
  constexpr int LPR = DP <= 128 ? 32 : 64, AT_ONCE = kRowsThreads / LPR, CHUNKS = BM / kJoinRows, MINE = kJoinRows / AT_ONCE;
  const int lane = threadIdx.x % LPR;
  RowsWalk<PAGED, BM, KT> walk;
  walk.template init<false>(a);
  const uint32_t chunk = blockIdx.x % CHUNKS, y = blockIdx.x / CHUNKS, x = udiv(y, a.heads_div);
  const int h = int(y - x * a.heads_div.d);
  int b;
  uint32_t tile, first;
  RowsSeq seq;
  if (!walk.template find<false, false>(a, x, &b, &tile, &first, &seq)) return;
  const int parts = int(walk.parts(a, seq)), tiles = int(walk.tiles(a, seq)), rows = seq.n * a.group;
  const int row0 = int(tile) * BM + int(chunk) * kJoinRows;
  if (parts == 1 || row0 >= rows) return;
  // (starts that do not ascend can ask for more parts than there were workgroups)
  if ((int64_t(first + tile) + int64_t(parts - 1) * tiles) * a.heads + h >= a.workgroups) return;
  // part k's rows are those of workgroup (first + k * tiles + tile) * heads + h
  const int64_t step = int64_t(tiles) * a.heads * BM, slot0 = (int64_t(first + tile) * a.heads + h) * BM + chunk * kJoinRows;
  const int d0 = 4 * lane < a.head_dim ? 4 * lane : 0;
  // a lane's MINE rows side by side; past the last row, that one again
  const float* ml[MINE];
  const float* from[MINE];
  f32x4 all[MINE];
  float top[MINE], total[MINE], m[MINE], l[MINE];
  constexpr int AHEAD = 4;  // parts requested at once
  f32x4 v[MINE][AHEAD];
#pragma unroll
  for (int z = 0; z < MINE; ++z) {
    const int i = int(threadIdx.x) / LPR + z * AT_ONCE;
    const int64_t slot = slot0 + (row0 + i < rows ? i : rows - 1 - row0);
    ml[z] = a.part_ml + 2 * slot;
    from[z] = a.part_o + slot * a.head_dim + d0;
    const float* at = ml[z] + 2 * (lane < parts ? lane : 0) * step;
    m[z] = at[0], l[z] = at[1];
  }
  const auto request = [&](int k0) {
#pragma unroll
    for (int z = 0; z < MINE; ++z)
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        v[z][j] = *reinterpret_cast<const f32x4*>(from[z] + (k0 + j < parts ? k0 + j : parts - 1) * step * a.head_dim);
  };
  request(0);
#pragma unroll
  for (int z = 0; z < MINE; ++z) {
    if (lane >= parts) m[z] = -kInf;
    top[z] = m[z];
    for (int k = lane + LPR; k < parts; k += LPR) top[z] = __builtin_fmaxf(top[z], ml[z][2 * k * step]);
#pragma unroll
    for (int d = 1; d < LPR; d *= 2) top[z] = __builtin_fmaxf(top[z], __shfl_xor(top[z], d, LPR));
    all[z] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    total[z] = 0.0f;
  }
  for (int k0 = 0; k0 < parts; k0 += LPR) {
    float f[MINE];  // of part k0 + lane
#pragma unroll
    for (int z = 0; z < MINE; ++z) {
      if (k0) {
        const float* at = ml[z] + 2 * (k0 + lane < parts ? k0 + lane : 0) * step;
        m[z] = k0 + lane < parts ? at[0] : -kInf, l[z] = at[1];
      }
      f[z] = k0 + lane < parts ? __builtin_amdgcn_exp2f((m[z] - finite(top[z])) * a.scale_log2e) : 0.0f;
      if (k0 + lane < parts) total[z] += l[z] * f[z];
    }
    for (int k = k0; k < parts && k < k0 + LPR; k += AHEAD) {
      if (k) request(k);
#pragma unroll
      for (int z = 0; z < MINE; ++z)
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
          const float g = __shfl(f[z], k - k0 + j, LPR);
          if (k + j < parts) all[z] += v[z][j] * g;
        }
    }
  }
#pragma unroll
  for (int z = 0; z < MINE; ++z) {
#pragma unroll
    for (int d = 1; d < LPR; d *= 2) total[z] += __shfl_xor(total[z], d, LPR);
    const int row = row0 + int(threadIdx.x) / LPR + z * AT_ONCE;
    if (row >= rows) continue;
    const int tok = int(udiv(uint32_t(row), a.group_div)), g = row - tok * a.group;
    const float inv = total[z] == 0.0f ? 0.0f : 1.0f / total[z];
    if (4 * lane < a.head_dim) {
      unsigned char* out = a.out + int64_t(seq.t0 + tok) * a.ot + (int64_t(h) * a.group + g) * a.oh;
      *reinterpret_cast<u32x2*>(out + 8 * lane) = u32x2{pack2<BF16>(all[z][0] * inv, all[z][1] * inv), pack2<BF16>(all[z][2] * inv, all[z][3] * inv)};
    }
    if (a.lse && lane == 0)
      a.lse[int64_t(seq.t0 + tok) * a.lt + (int64_t(h) * a.group + g) * a.lh] = lse_of(top[z], total[z] * unraise<RAISE>(), a.scale);
  }
}

}  // namespace dev
}  // namespace tc
