// Block tables that grow and shrink with their sequences: pages onto and off a stack of free ones, and the places of the
// new rows.
#include "paged_common.hpp"

namespace tc {
namespace dev {

constexpr int kResizeThreads = 1024;
constexpr int kResizeWaves = kResizeThreads / 64;
constexpr int kMostRows = 0x7fffffff;
constexpr int kPlaceThreads = 256;
constexpr int kPlaceTokens = 4;      // a lane
constexpr int kPlaceStarts = 4096;   // sequences whose starts fit LDS

__device__ __forceinline__ int resized(int n, int change) {
  const int64_t x = int64_t(n) + change;
  return x < 0 ? 0 : x < kMostRows ? int(x) : kMostRows;
}
// Pages of n rows that the table has columns for.
__device__ __forceinline__ int columns_of(int n, const Div32& page, int cols) {
  const uint32_t q = udiv(uint32_t(n), page), c = q + (q * page.d != uint32_t(n));
  return c < uint32_t(cols) ? int(c) : cols;
}
// Sums stop at kMostRows (also in any order).
__device__ __forceinline__ uint32_t sum_to_most(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < uint32_t(kMostRows) ? s : uint32_t(kMostRows);
}

// The sums of x over the lanes before this one of the workgroup; *total: of all.
__device__ __forceinline__ uint32_t sums_before(uint32_t x, uint32_t* shared, uint32_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t upto = x;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t y = __shfl_up(upto, d, 64);
    if (lane >= d) upto = sum_to_most(upto, y);
  }
  __syncthreads();  // the last sums have been read
  if (lane == 63) shared[wave] = upto;
  __syncthreads();
  uint32_t before = __shfl_up(upto, 1, 64);
  if (lane == 0) before = 0;
  uint32_t all = 0;
#pragma unroll
  for (int w = 0; w < kResizeWaves; ++w) {
    if (w == wave) before = sum_to_most(before, all);
    all = sum_to_most(all, shared[w]);
  }
  *total = all;
  return before;
}

// The last i < count with starts[i] <= t (starts ascending, starts[0] <= t).
__device__ __forceinline__ int find_start(const uint32_t* starts, int count, uint32_t t) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void place(const ResizeArgs& a, int b, int row, int64_t t) {
  const uint32_t col = udiv(uint32_t(row), a.page);
  if (a.slots) {
    const int page = col < uint32_t(a.table.cols) ? a.table.p[int64_t(b) * a.table.sb + int64_t(col) * a.table.sc] : -1;
    a.slots[t] = page < 0 ? -1 : int64_t(page) * a.page.d + (uint32_t(row) - col * a.page.d);
  }
  if (a.positions) a.positions[t] = row;
}

// One workgroup: sequences 1024 at a time, a lane each, their pages and tokens numbered by running sums; then a lane a page or
// token, its sequence found among the sums in LDS.  Pages that come back go onto the stack first, as far as they are pages and
// it has room; then those needed come off it.  PLACES: the new rows' places too; else only those of the one sequence whose
// rows the starts no longer count, as they stop at kMostRows (paged_places_kernel finds a row from where its sequence ends).
// Bound: its launch and a few dependent trips to memory, which is why one workgroup does it all.
template <bool PLACES>
__global__ __launch_bounds__(kResizeThreads) void paged_resize_kernel(ResizeArgs a) {
  __shared__ uint32_t shared[kResizeWaves];
  __shared__ uint32_t sums[kResizeThreads], token_sums[PLACES ? kResizeThreads : 1];
  __shared__ int from[kResizeThreads], row_from[PLACES ? kResizeThreads : 1];
  __shared__ int past, past_row;  // the sequence that passes kMostRows, its first new row
  const int tid = threadIdx.x, batch = a.table.batch, cols = a.table.cols;
  const auto length = [&](int b) { return a.lens[b] > 0 ? a.lens[b] : 0; };
  const int held = a.free_count[0];
  int top = held < 0 ? 0 : held < a.capacity ? held : a.capacity;

  for (int b0 = 0; b0 < batch; b0 += kResizeThreads) {
    const int b = b0 + tid, count = batch - b0 < kResizeThreads ? batch - b0 : kResizeThreads;
    uint32_t back = 0;
    if (b < batch) {
      const int n = length(b), first = columns_of(resized(n, a.change[b]), a.page, cols);
      const int last = columns_of(n, a.page, cols);
      back = last > first ? uint32_t(last - first) : 0u;
      from[tid] = first;
    }
    uint32_t total;
    sums[tid] = sums_before(back, shared, &total);
    __syncthreads();
    for (uint32_t t0 = 0; t0 < total; t0 += kResizeThreads) {
      const uint32_t t = t0 + tid;
      int page = -1;
      if (t < total) {
        const int i = find_start(sums, count, t);
        page = a.table.p[int64_t(b0 + i) * a.table.sb + int64_t(from[i] + int(t - sums[i])) * a.table.sc];
      }
      uint32_t pages;
      const uint32_t at = sums_before(page >= 0, shared, &pages);
      const int left = a.capacity - top;
      if (page >= 0 && at < uint32_t(left)) a.free_pages[top + int(at)] = page;
      top += pages < uint32_t(left) ? int(pages) : left;
    }
    __syncthreads();  // sums and from are written anew
  }

  uint32_t taken = 0, tokens = 0;
  for (int b0 = 0; b0 < batch; b0 += kResizeThreads) {
    const int b = b0 + tid, count = batch - b0 < kResizeThreads ? batch - b0 : kResizeThreads;
    uint32_t take = 0, grow = 0;
    int from_row = 0;
    if (b < batch) {
      const int n = length(b), now = resized(n, a.change[b]);
      const int first = columns_of(n, a.page, cols), last = columns_of(now, a.page, cols);
      take = last > first ? uint32_t(last - first) : 0u;
      grow = now > n ? uint32_t(now - n) : 0u;
      from[tid] = first;
      from_row = n;
      if (PLACES) row_from[tid] = n;
      a.lens_out[b] = now;
    }
    uint32_t total, all = 0;
    sums[tid] = sums_before(take, shared, &total);
    if (a.starts) {
      const uint32_t before = sums_before(grow, shared, &all);
      if (PLACES) token_sums[tid] = before;
      const uint32_t start = sum_to_most(tokens, before);
      if (b < batch) a.starts[b] = int32_t(start);
      if (!PLACES && grow && start < uint32_t(kMostRows) && sum_to_most(start, grow) == uint32_t(kMostRows)) past = b, past_row = from_row;
    }
    __syncthreads();
    for (uint32_t t = tid; t < total; t += kResizeThreads) {
      const int i = find_start(sums, count, t);
      const int64_t at = int64_t(top) - 1 - taken - t;
      a.table_out[int64_t(b0 + i) * a.table.sb + int64_t(from[i] + int(t - sums[i])) * a.table.sc] = at >= 0 ? a.free_pages[at] : -1;
    }
    taken += total;
    if constexpr (PLACES) {
      __syncthreads();  // the table holds the pages
      for (uint32_t t = tid; t < all; t += kResizeThreads) {
        const uint32_t to = sum_to_most(tokens, t);
        if (to >= uint32_t(a.tokens)) break;
        const int i = find_start(token_sums, count, t);
        place(a, b0 + i, row_from[i] + int(t - token_sums[i]), to);
      }
    } else if (tokens < uint32_t(kMostRows) && sum_to_most(tokens, all) == uint32_t(kMostRows)) {
      __syncthreads();
      const int start = a.starts[past];
      for (int64_t t = int64_t(start) + tid; t < a.tokens; t += kResizeThreads) place(a, past, past_row + int(t - start), t);
    }
    tokens = sum_to_most(tokens, all);
    __syncthreads();
  }
  if (tid == 0) {
    if (a.starts) a.starts[batch] = int32_t(tokens);
    a.count_out[0] = taken < uint32_t(top) ? top - int(taken) : 0;
    if (a.missing) a.missing[0] = taken < uint32_t(top) ? 0 : int(taken - uint32_t(top));
  }
  if constexpr (PLACES)
    for (int64_t t = int64_t(tokens) + tid; t < a.tokens; t += kResizeThreads) {
      if (a.slots) a.slots[t] = -1;
      if (a.positions) a.positions[t] = -1;
    }
}

// The places of many new rows, four a lane, once the pages are in the table.  A row counts back from its sequence's end, since
// lens_out may have taken the place of the old lengths; where that end is kMostRows the sums stopped, and the first kernel
// has placed the rows.
__global__ __launch_bounds__(kPlaceThreads) void paged_places_kernel(ResizeArgs a) {
  __shared__ uint32_t held[kPlaceStarts];
  const int batch = a.table.batch;
  const uint32_t* starts = reinterpret_cast<const uint32_t*>(a.starts);
  if (batch <= kPlaceStarts) {
    for (int i = threadIdx.x; i < batch; i += kPlaceThreads) held[i] = starts[i];
    __syncthreads();
  }
  const int total = a.starts[batch];
  const int64_t t0 = (int64_t(blockIdx.x) * kPlaceThreads + threadIdx.x) * kPlaceTokens;
  if (t0 >= a.tokens) return;
  int b = 0, row = 0, end = 0;
  if (t0 < total) {
    b = batch <= kPlaceStarts ? find_start(held, batch, uint32_t(t0)) : find_start(starts, batch, uint32_t(t0));
    end = a.starts[b + 1];
    row = a.lens_out[b] - (end - int(t0));
  }
#pragma unroll 1
  for (int k = 0; k < kPlaceTokens; ++k, ++row) {
    const int64_t t = t0 + k;
    if (t >= a.tokens) return;
    if (t >= total) {
      if (a.slots) a.slots[t] = -1;
      if (a.positions) a.positions[t] = -1;
      continue;
    }
    if (t >= end) {
      do end = a.starts[++b + 1];
      while (t >= end);
      row = a.lens_out[b] - (end - int(t));
    }
    if (end == kMostRows) return;
    place(a, b, row, t);
  }
}

}  // namespace dev

int launch_paged_resize(const ResizeArgs& a, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  // one workgroup places as many rows while a second launch would cost more
  const bool here = a.tokens <= 8 * dev::kResizeThreads;
  const int64_t lanes = (int64_t(a.tokens) + dev::kPlaceTokens - 1) / dev::kPlaceTokens;
  const int64_t groups = (lanes + dev::kPlaceThreads - 1) / dev::kPlaceThreads;
  if (!launchable(groups, dev::kPlaceThreads)) return TC_E_RANGE;
  if (here && a.tokens)
    hipLaunchKernelGGL(dev::paged_resize_kernel<true>, dim3(1), dim3(dev::kResizeThreads), 0, s, a);
  else
    hipLaunchKernelGGL(dev::paged_resize_kernel<false>, dim3(1), dim3(dev::kResizeThreads), 0, s, a);
  if (!here) hipLaunchKernelGGL(dev::paged_places_kernel, dim3(uint32_t(groups)), dim3(dev::kPlaceThreads), 0, s, a);
  return TC_OK;
}

}  // namespace tc
