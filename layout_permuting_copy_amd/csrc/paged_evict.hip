// Eviction from a paged cache by accumulated attention weight: which rows stay, and their copy.
#include "paged_common.hpp"

namespace tc {
namespace dev {

constexpr int kBins = 2048;  // histogram bins: 11 bits of a key

// An unsigned integer that orders weights as numbers: equal zeros, any NaN above all.  The lowest, -infinity's, is
// 0x007fffff.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.0f);  // -0 + 0 = 0
  return w != w ? 0xffffffffu : u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}

// How many lanes below this one a ballot holds.
__device__ __forceinline__ uint32_t lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi(uint32_t(m >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(m), 0));
}

// The sum of x[0 .. wave - 1] (WAVES <= 16 values in LDS, one a lane).
template <int WAVES>
__device__ __forceinline__ uint32_t sum_below(const uint32_t* x, int wave, int lane) {
  const uint32_t upto = wave_scan(lane < WAVES ? x[lane] : 0u);
  return wave ? uint32_t(__builtin_amdgcn_readlane(int(upto), wave - 1)) : 0u;
}

// One workgroup a (sequence, head): the kept rows of a sequence over its budget.  The budget -
// recent heaviest of the first n - recent rows are those with key > T and the first `left` with
// key == T; T is found by a radix selection of 11 + 11 + 10 bits from the top, each pass a
// histogram in LDS of the keys that share the digits found so far, ended as soon as every key with
// those digits stays.  Every wave owns a stretch of the rows, so a walk in order needs only the waves' counts to
// place what it keeps.
//
// KEYS: weights a lane holds in registers, with their keys (one read of the weights; THREADS * KEYS rows at most), or
// 0: every pass reads them again, from the caches.  HISTS: copies of the histogram, one for every HISTS-th wave, so that
// fewer lanes add to one bin.  Bound: trips to memory, barriers, LDS atomics and, with many rows, the vector
// instructions of one workgroup's walks (8 heads of 2049 rows 6.5 us, 128 of up to 16384 rows 15.4 us; with the keys made
// again by every walk 20 us, with the weights read again by every pass 33 us).
template <int THREADS, int KEYS, int HISTS>
__global__ __launch_bounds__(THREADS) void paged_select_kernel(EvictArgs a, Div32 heads) {
  constexpr int WAVES = THREADS / 64, BPT = kBins / THREADS;  // bins a thread sums
  const int b = int(udiv(blockIdx.x, heads)), h = int(blockIdx.x - uint32_t(b) * heads.d);
  const int n = paged_len(a.lens, b, a.max_len);
  const int kept_n = n < a.budget ? n : a.budget;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int32_t* kept = a.kept + b * a.kr.sb + h * a.kr.sh;
  const float* w = a.weights + b * a.w.sb + h * a.w.sh;
  float* wo = a.weights_out ? a.weights_out + b * a.wo.sb + h * a.wo.sh : nullptr;
  if (h == 0 && tid == 0) a.lens_out[b] = kept_n;
  for (int64_t j = kept_n + tid; j < a.kr.cols; j += THREADS) kept[j * a.kr.sc] = -1;
  if (n <= a.budget) {
    for (int j = tid; j < n; j += THREADS) {
      kept[j * a.kr.sc] = j;
      if (wo) wo[j * a.wo.sc] = w[j * a.w.sc];
    }
    return;
  }
  const int cand = n - a.recent, want = a.budget - a.recent;  // cand > want >= 0
  const int seg = ((cand + WAVES - 1) / WAVES + 63) / 64 * 64;  // at most 64 * KEYS, if those are held
  const int lo = wave * seg, hi = lo + seg < cand ? lo + seg : cand;
  float held[KEYS ? KEYS : 1];
  uint32_t key_held[KEYS ? KEYS : 1];
#pragma unroll
  for (int k = 0; k < KEYS; ++k) held[k] = lo + 64 * k + lane < hi ? w[(lo + 64 * k + lane) * a.w.sc] : 0.0f;
  for (int j = tid; j < a.recent; j += THREADS) {
    kept[(want + j) * a.kr.sc] = cand + j;
    if (wo) wo[(want + j) * a.wo.sc] = w[(cand + j) * a.w.sc];
  }
  if (want == 0) return;
#pragma unroll
  for (int k = 0; k < KEYS; ++k) key_held[k] = lo + 64 * k + lane < hi ? weight_key(held[k]) : 0u;
  // f(row, weight, key) over the wave's rows, 64 at a time, in order; lanes past them have key 0, which no weight has
  const auto each = [&](auto f) {
    if constexpr (KEYS > 0) {
#pragma unroll
      for (int k = 0; k < KEYS; ++k)
        if (lo + 64 * k < hi) f(lo + 64 * k + lane, held[k], key_held[k]);
    } else {
      for (int i = lo + lane; i - lane < hi; i += 64) {
        const float x = i < hi ? w[i * a.w.sc] : 0.0f;
        f(i, x, i < hi ? weight_key(x) : 0u);
      }
    }
  };

  __shared__ uint32_t hist[HISTS][kBins];
  __shared__ uint32_t wave_sum[WAVES], wave_eq[WAVES];
  __shared__ uint32_t found_digit, found_above, found_count;
  uint32_t prefix = 0, mask = 0;
  bool all = false;
  uint32_t left = uint32_t(want);  // keys still to be found among those that match the prefix
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bins = pass == 2 ? 1024 : 2048;
    for (int i = tid; i < HISTS * kBins / 4; i += THREADS) reinterpret_cast<u32x4*>(&hist[0][0])[i] = u32x4{};
    __syncthreads();
    each([&](int, float, uint32_t key) {
      if (pass ? (key & mask) == prefix : key != 0) atomicAdd(&hist[wave % HISTS][(key >> shift) & (bins - 1)], 1u);
    });
    __syncthreads();
    // thread t sums the BPT bins below kBins - BPT * t; the wanted bin is where the count from the top first
    // reaches `left`
    const int top = kBins - 1 - BPT * tid;
    uint32_t c[BPT], sum = 0;
#pragma unroll
    for (int k = 0; k < BPT; ++k) {
      c[k] = 0;
#pragma unroll
      for (int i = 0; i < HISTS; ++i) c[k] += hist[i][top - k];
      sum += c[k];
    }
    const uint32_t upto = wave_scan(sum);
    if (lane == 63) wave_sum[wave] = upto;
    __syncthreads();
    uint32_t before = upto - sum + sum_below<WAVES>(wave_sum, wave, lane);
    if (before < left && before + sum >= left) {
#pragma unroll
      for (int k = 0; k < BPT; ++k) {
        if (before < left && before + c[k] >= left) {
          found_digit = uint32_t(top - k);
          found_above = before;
          found_count = c[k];
        }
        before += c[k];
      }
    }
    __syncthreads();
    prefix |= found_digit << shift;
    mask |= (bins - 1) << shift;
    left -= found_above;
    all = found_count == left;
    if (all) break;
    __syncthreads();  // found_*, wave_sum and hist are written again
  }
  __syncthreads();

  // (64-bit products a row would take as long as the rest of the walk)
  const bool dense = a.kr.sc == 1 && (!wo || a.wo.sc == 1);
  const auto keep = [&](int i, float x, uint32_t j) {
    if (dense) {
      kept[j] = i;
      if (wo) wo[j] = x;
    } else {
      kept[j * a.kr.sc] = i;
      if (wo) wo[j * a.wo.sc] = x;
    }
  };
  if (all) {
    // every key with the prefix or above stays
    uint32_t count = 0;
    each([&](int, float, uint32_t key) { count += __popcll(__ballot(key >= prefix)); });
    if (lane == 0) wave_sum[wave] = count;
    __syncthreads();
    uint32_t before = sum_below<WAVES>(wave_sum, wave, lane);
    each([&](int i, float x, uint32_t key) {
      const uint64_t m = __ballot(key >= prefix);
      if (m >> lane & 1) keep(i, x, before + lanes_below(m));
      before += __popcll(m);
    });
    return;
  }
  // keys above T stay, and `left` of those equal to it, the lowest rows first
  uint32_t gt = 0, eq = 0;
  each([&](int, float, uint32_t key) {
    gt += __popcll(__ballot(key > prefix));
    eq += __popcll(__ballot(key == prefix));
  });
  if (lane == 0) {
    wave_sum[wave] = gt;
    wave_eq[wave] = eq;
  }
  __syncthreads();
  uint32_t gt_before = sum_below<WAVES>(wave_sum, wave, lane), eq_before = sum_below<WAVES>(wave_eq, wave, lane);
  each([&](int i, float x, uint32_t key) {
    const uint64_t g = __ballot(key > prefix), e = __ballot(key == prefix);
    const uint32_t eq_rank = eq_before + lanes_below(e);
    const uint32_t ties = eq_rank < left ? eq_rank : left;  // kept ties below this row
    if ((g >> lane & 1) || ((e >> lane & 1) && eq_rank < left)) keep(i, x, gt_before + lanes_below(g) + ties);
    gt_before += __popcll(g);
    eq_before += __popcll(e);
  });
}

template <int THREADS, int KEYS, int HISTS>
void select(const EvictArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((paged_select_kernel<THREADS, KEYS, HISTS>), dim3(uint32_t(a.table.batch * a.heads)), dim3(THREADS), 0, s, a,
                     make_div32(uint32_t(a.heads)));
}

constexpr int kCopyThreads = 256;

// The kept rows of keys and values into their new pages: LPR lanes a row, 16 bytes a lane (two or four
// rows a lane: level).  Grid: (sequence, rows, head), the heads fastest: those of the same new rows are neighbours
// where a pool keeps a row's heads together.  Bound: HBM, by rows of 256 bytes read here and there (16 sequences to
// 4096 rows: 408 MB in 84 us, 4.9 TB/s).
template <bool E4M3, int LPR>
__global__ __launch_bounds__(kCopyThreads) void paged_move_kernel(EvictArgs a, Div32 heads, Div32 chunks) {
  constexpr int ROWS = kCopyThreads / LPR;
  const uint32_t bc = udiv(blockIdx.x, heads), bb = udiv(bc, chunks), chunk = bc - bb * chunks.d;
  const int b = int(bb), h = int(blockIdx.x - bc * heads.d);
  const int n = paged_len(a.lens, b, a.max_len);
  const int kept_n = n < a.budget ? n : a.budget;
  const int j = int(chunk) * ROWS + int(threadIdx.x) / LPR, c = threadIdx.x % LPR;
  if (int(chunk) * ROWS >= kept_n) return;
  const int32_t* kept = a.kept + b * a.kr.sb + h * a.kr.sh;
  const int from = kept[(j < kept_n ? j : 0) * a.kr.sc];
  const int dp = j < kept_n ? paged_page(a.dst_table, a.dst, b, udiv(uint32_t(j), a.dst.div)) : -1;
  const int sp = paged_page(a.table, a.src, b, udiv(uint32_t(from), a.src.div));
  const bool moves = sp >= 0 && dp >= 0 && 16 * c < a.row_bytes;
  const uint32_t src_row = uint32_t(from) - udiv(uint32_t(from), a.src.div) * a.src.div.d;
  const uint32_t dst_row = uint32_t(j) - udiv(uint32_t(j), a.dst.div) * a.dst.div.d;
  u32x4 k, v;
  float ks, vs;
  if (moves) {
    gload<16, 1>(a.src.k + sp * a.src.kp + src_row * a.src.kr + h * a.src.kh + 16 * c, reinterpret_cast<uint32_t*>(&k));
    gload<16, 1>(a.src.v + sp * a.src.vp + src_row * a.src.vr + h * a.src.vh + 16 * c, reinterpret_cast<uint32_t*>(&v));
    if (E4M3 && c == 0) {
      ks = a.src.ks[sp * a.src.ksp + src_row * a.src.ksr + h * a.src.ksh];
      vs = a.src.vs[sp * a.src.vsp + src_row * a.src.vsr + h * a.src.vsh];
    }
  }
  if (!moves) return;
  gstore<16, 2>(a.dst.k + dp * a.dst.kp + dst_row * a.dst.kr + h * a.dst.kh + 16 * c, reinterpret_cast<uint32_t*>(&k));
  gstore<16, 2>(a.dst.v + dp * a.dst.vp + dst_row * a.dst.vr + h * a.dst.vh + 16 * c, reinterpret_cast<uint32_t*>(&v));
  if (E4M3 && c == 0) {
    a.dst.ks[dp * a.dst.ksp + dst_row * a.dst.ksr + h * a.dst.ksh] = ks;
    a.dst.vs[dp * a.dst.vsp + dst_row * a.dst.vsr + h * a.dst.vsh] = vs;
  }
}

// Lanes a row of so many bytes takes, 16 bytes each, and the workgroups that the rows of one (sequence, head) take.
constexpr int move_lanes(int row_bytes) {
  int lanes = 1;
  while (16 * lanes < row_bytes) lanes *= 2;
  return lanes;
}
constexpr int64_t move_chunks(int most, int lanes) {
  const int per = kCopyThreads / lanes;
  return (int64_t(most) + per - 1) / per;
}

template <bool E4M3, int LPR>
void move(const EvictArgs& a, int most, hipStream_t s) {
  const int64_t chunks = move_chunks(most, LPR), wgs = chunks * a.table.batch * a.heads;
  hipLaunchKernelGGL((paged_move_kernel<E4M3, LPR>), dim3(uint32_t(wgs)), dim3(kCopyThreads), 0, s, a,
                     make_div32(uint32_t(a.heads)), make_div32(uint32_t(chunks)));
}

template <bool E4M3>
void move_rows(const EvictArgs& a, int most, hipStream_t s) {
  const int lanes = move_lanes(a.row_bytes);
  if constexpr (E4M3) {
    if (lanes == 1) return move<E4M3, 1>(a, most, s);
  } else {
    if (lanes == 32) return move<E4M3, 32>(a, most, s);
  }
  if (lanes == 2) return move<E4M3, 2>(a, most, s);
  if (lanes == 4) return move<E4M3, 4>(a, most, s);
  if (lanes == 8) return move<E4M3, 8>(a, most, s);
  return move<E4M3, 16>(a, most, s);
}

}  // namespace dev

int launch_paged_evict(const EvictArgs& a, int cache_dtype, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int most = a.budget < a.max_len ? a.budget : a.max_len;
  // both grids have to fit before anything is launched
  const int64_t rows = int64_t(a.table.batch) * a.heads, chunks = dev::move_chunks(most, dev::move_lanes(a.row_bytes));
  if (!launchable(rows, 1024) || !launchable(chunks * rows, dev::kCopyThreads)) return TC_E_RANGE;
  if (a.max_len <= 1024)
    dev::select<256, 4, 1>(a, s);
  else if (a.max_len <= 4096)
    dev::select<1024, 4, 2>(a, s);
  else if (a.max_len <= 16384)
    dev::select<1024, 16, 4>(a, s);
  else if (a.max_len <= 32768)
    dev::select<1024, 32, 4>(a, s);
  else
    dev::select<1024, 0, 4>(a, s);
  if (most == 0) return TC_OK;
  if (cache_dtype == TC_E4M3)
    dev::move_rows<true>(a, most, s);
  else
    dev::move_rows<false>(a, most, s);
  return TC_OK;
}

}  // namespace tc
