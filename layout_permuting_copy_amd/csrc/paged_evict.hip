// Eviction from a paged cache by accumulated attention weight: which rows stay, and their copy.
#include "paged_common.hpp"

namespace tc {
namespace dev {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / 64;
constexpr int kBins = 2048;  // histogram bins: 11 bits of a key
constexpr int kHists = 4;    // copies of the histogram, one for every fourth wave

// An unsigned integer that orders weights as numbers: equal zeros, any NaN above all.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __builtin_bit_cast(uint32_t, w);
  if (w != w) return 0xffffffffu;
  if ((u << 1) == 0) return 0x80000000u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One workgroup a (sequence, head): the kept rows of a sequence over its budget.  The budget -
// recent heaviest of the first n - recent rows are those with key > T and the first `need` with
// key == T; T is found by a radix selection of 11 + 11 + 10 bits from the top, each pass a
// histogram in LDS of the keys that share the digits found so far.  Every wave owns a stretch of
// the rows, so a walk in order needs only the waves' counts to place what it keeps.
// Bound: the passes over the weights, which after the first come from the caches.
__global__ __launch_bounds__(kSelectThreads) void paged_select_kernel(EvictArgs a, Div32 heads) {
  const int b = int(udiv(blockIdx.x, heads)), h = int(blockIdx.x - uint32_t(b) * heads.d);
  const int n = paged_len(a.lens, b, a.max_len);
  const int kept_n = n < a.budget ? n : a.budget;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int32_t* kept = a.kept + b * a.kr.sb + h * a.kr.sh;
  const float* w = a.weights + b * a.w.sb + h * a.w.sh;
  float* wo = a.weights_out ? a.weights_out + b * a.wo.sb + h * a.wo.sh : nullptr;
  if (h == 0 && tid == 0) a.lens_out[b] = kept_n;
  for (int64_t j = kept_n + tid; j < a.kr.cols; j += kSelectThreads) kept[j * a.kr.sc] = -1;
  if (n <= a.budget) {
    for (int j = tid; j < n; j += kSelectThreads) {
      kept[j * a.kr.sc] = j;
      if (wo) wo[j * a.wo.sc] = w[j * a.w.sc];
    }
    return;
  }
  const int cand = n - a.recent, want = a.budget - a.recent;  // cand > want >= 0
  for (int j = tid; j < a.recent; j += kSelectThreads) {
    kept[(want + j) * a.kr.sc] = cand + j;
    if (wo) wo[(want + j) * a.wo.sc] = w[(cand + j) * a.w.sc];
  }
  if (want == 0) return;

  __shared__ uint32_t hist[kHists][kBins];
  __shared__ uint32_t wave_sum[kSelectWaves], wave_eq[kSelectWaves];
  __shared__ uint32_t found_digit, found_above;
  const int seg = ((cand + kSelectWaves - 1) / kSelectWaves + 63) / 64 * 64;
  const int lo = wave * seg, hi = lo + seg < cand ? lo + seg : cand;

  uint32_t prefix = 0, mask = 0;
  int left = want;  // keys still to be found among those that match the prefix
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bins = pass == 2 ? 1024 : 2048;
    for (int i = tid; i < kHists * kBins; i += kSelectThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    for (int i = lo + lane; i < hi; i += 64) {
      const uint32_t key = weight_key(w[i * a.w.sc]);
      if ((key & mask) == prefix) atomicAdd(&hist[wave % kHists][(key >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // bins from the top: thread t holds bins 2047 - 2 t and 2046 - 2 t; the wanted bin is where
    // the running count from the top first reaches `left`
    const int top = kBins - 1 - 2 * tid;
    uint32_t c0 = 0, c1 = 0;
#pragma unroll
    for (int k = 0; k < kHists; ++k) {
      c0 += hist[k][top];
      c1 += hist[k][top - 1];
    }
    uint32_t sum = c0 + c1;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t o = __shfl_up(sum, d, 64);
      if (lane >= d) sum += o;
    }
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    uint32_t before = sum - c0 - c1;
    for (int k = 0; k < wave; ++k) before += wave_sum[k];
    if (before < uint32_t(left) && before + c0 + c1 >= uint32_t(left)) {
      const bool first = before + c0 >= uint32_t(left);
      found_digit = uint32_t(first ? top : top - 1);
      found_above = first ? before : before + c0;
    }
    __syncthreads();
    prefix |= found_digit << shift;
    mask |= (bins - 1) << shift;
    left -= int(found_above);
    __syncthreads();  // found_*, wave_sum and hist are written again
  }

  // T = prefix; `left` of the keys equal to it stay, the lowest rows first
  uint32_t gt = 0, eq = 0;
  for (int i = lo + lane; i - lane < hi; i += 64) {
    const uint32_t key = i < hi ? weight_key(w[i * a.w.sc]) : 0;
    gt += __popcll(__ballot(i < hi && key > prefix));
    eq += __popcll(__ballot(i < hi && key == prefix));
  }
  if (lane == 0) {
    wave_sum[wave] = gt;
    wave_eq[wave] = eq;
  }
  __syncthreads();
  uint32_t gt_before = 0, eq_before = 0;
  for (int k = 0; k < wave; ++k) {
    gt_before += wave_sum[k];
    eq_before += wave_eq[k];
  }
  const uint64_t below = (uint64_t(1) << lane) - 1;
  for (int i = lo + lane; i - lane < hi; i += 64) {
    const float x = i < hi ? w[i * a.w.sc] : 0.0f;
    const uint32_t key = weight_key(x);
    const uint64_t g = __ballot(i < hi && key > prefix), e = __ballot(i < hi && key == prefix);
    const uint32_t eq_rank = eq_before + __popcll(e & below);
    const uint32_t ties = eq_rank < uint32_t(left) ? eq_rank : uint32_t(left);  // kept ties below this row
    const bool keep = (g >> lane & 1) || ((e >> lane & 1) && eq_rank < uint32_t(left));
    if (keep) {
      const int64_t j = gt_before + __popcll(g & below) + ties;
      kept[j * a.kr.sc] = i;
      if (wo) wo[j * a.wo.sc] = x;
    }
    gt_before += __popcll(g);
    eq_before += __popcll(e);
  }
}

constexpr int kCopyThreads = 256;

// The kept rows of keys and values into their new pages: LPR lanes a row, 16 bytes a lane.
// Grid: (sequence, head) times `chunks` workgroups over the rows.  Bound: HBM.
template <bool E4M3, int LPR>
__global__ __launch_bounds__(kCopyThreads) void paged_move_kernel(EvictArgs a, Div32 heads, Div32 chunks) {
  constexpr int RPW = kCopyThreads / LPR;
  const uint32_t bh = udiv(blockIdx.x, chunks), chunk = blockIdx.x - bh * chunks.d;
  const int b = int(udiv(bh, heads)), h = int(bh - uint32_t(b) * heads.d);
  const int n = paged_len(a.lens, b, a.max_len);
  const int kept_n = n < a.budget ? n : a.budget;
  const int j = int(chunk) * RPW + int(threadIdx.x) / LPR, c = threadIdx.x % LPR;
  if (j >= kept_n || 16 * c >= a.row_bytes) return;
  const int i = a.kept[b * a.kr.sb + h * a.kr.sh + j * a.kr.sc];
  const uint32_t sc = udiv(uint32_t(i), a.src.div), dc = udiv(uint32_t(j), a.dst.div);
  const uint32_t sr = uint32_t(i) - sc * a.src.div.d, dr = uint32_t(j) - dc * a.dst.div.d;
  const int sp = paged_page(a.table, a.src, b, sc), dp = paged_page(a.dst_table, a.dst, b, dc);
  if (sp < 0 || dp < 0) return;
  const u32x4 k = *reinterpret_cast<const u32x4*>(a.src.k + sp * a.src.kp + sr * a.src.kr + h * a.src.kh + 16 * c);
  const u32x4 v = *reinterpret_cast<const u32x4*>(a.src.v + sp * a.src.vp + sr * a.src.vr + h * a.src.vh + 16 * c);
  *reinterpret_cast<u32x4*>(a.dst.k + dp * a.dst.kp + dr * a.dst.kr + h * a.dst.kh + 16 * c) = k;
  *reinterpret_cast<u32x4*>(a.dst.v + dp * a.dst.vp + dr * a.dst.vr + h * a.dst.vh + 16 * c) = v;
  if (E4M3 && c == 0) {
    a.dst.ks[dp * a.dst.ksp + dr * a.dst.ksr + h * a.dst.ksh] = a.src.ks[sp * a.src.ksp + sr * a.src.ksr + h * a.src.ksh];
    a.dst.vs[dp * a.dst.vsp + dr * a.dst.vsr + h * a.dst.vsh] = a.src.vs[sp * a.src.vsp + sr * a.src.vsr + h * a.src.vsh];
  }
}

template <bool E4M3, int LPR>
int move(const EvictArgs& a, int most, hipStream_t s) {
  constexpr int per = kCopyThreads / LPR;
  const int64_t chunks = (int64_t(most) + per - 1) / per, wgs = chunks * a.table.batch * a.heads;
  if (wgs >= int64_t(1) << 31) return TC_E_RANGE;
  hipLaunchKernelGGL((paged_move_kernel<E4M3, LPR>), dim3(uint32_t(wgs)), dim3(kCopyThreads), 0, s, a,
                     make_div32(uint32_t(a.heads)), make_div32(uint32_t(chunks)));
  return TC_OK;
}

template <bool E4M3>
int move_rows(const EvictArgs& a, int most, hipStream_t s) {
  const int lanes = a.row_bytes / 16;
  if (lanes <= 1) return move<E4M3, 1>(a, most, s);
  if (lanes <= 2) return move<E4M3, 2>(a, most, s);
  if (lanes <= 4) return move<E4M3, 4>(a, most, s);
  if (lanes <= 8) return move<E4M3, 8>(a, most, s);
  if (lanes <= 16) return move<E4M3, 16>(a, most, s);
  return move<E4M3, 32>(a, most, s);
}

}  // namespace dev

int launch_paged_evict(const EvictArgs& a, int cache_dtype, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int most = a.budget < a.max_len ? a.budget : a.max_len;
  // the move's grid has to fit before anything is launched (8 rows a workgroup at the widest rows)
  if ((int64_t(most) / 8 + 1) * a.table.batch * a.heads >= int64_t(1) << 31) return TC_E_RANGE;
  hipLaunchKernelGGL(dev::paged_select_kernel, dim3(uint32_t(a.table.batch * a.heads)), dim3(dev::kSelectThreads), 0, s, a,
                     make_div32(uint32_t(a.heads)));
  if (most == 0) return TC_OK;
  return cache_dtype == TC_E4M3 ? dev::move_rows<true>(a, most, s) : dev::move_rows<false>(a, most, s);
}

}  // namespace tc
