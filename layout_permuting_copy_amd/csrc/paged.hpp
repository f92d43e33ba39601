// The paged key-value cache operators: argument blocks the kernels take, launchers, and the device
// side they share (finding a cache row through a block table).
#pragma once

#include <cstdint>
#include <string>

#include "plan.hpp"

namespace tc {

constexpr int kPagedMaxHeadDim = 256;

// A pool of pages: base pointers and byte strides of pages, rows and heads (scales: in floats).
struct PagedPool {
  unsigned char* k;
  unsigned char* v;
  float* ks;
  float* vs;
  int64_t kp, kr, kh, vp, vr, vh;
  int64_t ksp, ksr, ksh, vsp, vsr, vsh;
  int32_t pages, page_size;
  Div32 div;  // by page_size
};

// A block table: int32, (batch, cols), strides in elements.
struct PagedTable {
  const int32_t* p;
  int64_t sb, sc;
  int32_t batch, cols;
};

// fp32 or int32 of (batch, heads, columns), strides in elements.
struct PagedRows {
  int64_t sb, sh, sc;
  int64_t cols;
};

struct AppendArgs {
  PagedPool pool;
  PagedTable table;
  const unsigned char* k;  // new rows; byte strides
  const unsigned char* v;
  int64_t kt, kh, vt, vh;
  const int32_t* lens;
  const int32_t* starts;  // or NULL: one token a sequence
  float* weights;         // or NULL
  PagedRows w;
  int64_t tokens;
  int32_t heads, head_dim;
};

// The parts of a sequence that several runs share: `count` of them (0: nothing is shared), the first in slot
// `slot` of the workgroups of run `run`, the others in slots 0 of the next runs'.
struct PagedParts {
  int32_t b, run, count, slot;
};

struct AttentionArgs {
  PagedPool pool;
  PagedTable table;
  const unsigned char* q;
  unsigned char* out;
  int64_t qb, qh, ob, oh;  // byte strides
  const int32_t* lens;
  float* lse;  // or NULL
  int64_t lb, lh;
  const float* weights;
  float* weights_out;  // or NULL
  PagedRows w, wo;
  float* part_o;    // [workgroups][2][tile_heads][head_dim]: a part's sum of p v, relative to its maximum
  float* part_ml;   // [workgroups][2][tile_heads][2]: its maximum (base 2) and sum
  PagedParts* parts;  // by sequence, or by run where there are fewer of those; NULL where nothing can be cut
  float* final_ml;  // [batch * q_heads][2]: the same of whole rows, where weights are wanted
  float* logits;    // [batch * q_heads][logit_row]: scale * q . k * log2 e, where weights are wanted
  int64_t logit_row;
  int32_t heads, group, head_dim;
  int32_t max_len, workgroups, runs, least_units, tile_heads, head_tiles, parts_of_sequences;
  int64_t units;    // at most
  Div32 unit;       // by the rows of a unit
  Div32 pairs_div;  // by heads * head_tiles
  Div32 heads_div;  // by heads
  float scale_log2e;
};

struct EvictArgs {
  PagedPool src, dst;
  PagedTable table, dst_table;
  const int32_t* lens;
  const float* weights;
  PagedRows w;
  int32_t* lens_out;
  int32_t* kept;
  PagedRows kr;
  float* weights_out;  // or NULL
  PagedRows wo;
  int32_t heads, row_bytes;
  int32_t max_len, budget, recent;
};

// How an attention call is cut over the cache's length: units of `unit_rows` rows (at most `units` in all), `runs` runs
// of at least least_units of them, query heads in tiles of tile_heads, at most `workgroups` workgroups; whether a
// sequence's rows can fall to more than one run.  `most`: as a call of a smaller batch may be cut where this one is not, so
// that sizes that follow from it grow with batch and max_len.
struct PagedCut {
  int64_t unit_rows, units, least_units, runs, workgroups, tile_heads, head_tiles;
  bool cuts;
};
PagedCut paged_cut(int64_t batch, int64_t heads, int64_t group, int64_t head_dim, int64_t max_len, bool most);
// Columns a row of the logits workspace holds: max_len rounded up to whole tiles.
int64_t paged_logit_row(int64_t max_len);

// A launch counts its lanes in 32 bits.
constexpr bool launchable(int64_t workgroups, int64_t threads) { return workgroups * threads < int64_t(1) << 32; }

// Launchers: TC_OK, or TC_E_RANGE, and nothing launched, where a grid would be too large.  `dtype` is that of the new rows or of
// q, `cache_dtype` the pool's; `wide`: new rows take 16-byte loads.
int launch_paged_append(const AppendArgs& a, int dtype, int cache_dtype, bool wide, void* stream);
int launch_paged_attention(const AttentionArgs& a, int dtype, int cache_dtype, void* stream);
int launch_paged_evict(const EvictArgs& a, int cache_dtype, void* stream);

}  // namespace tc
