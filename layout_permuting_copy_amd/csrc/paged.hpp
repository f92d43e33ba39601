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

// Attention of several query rows a sequence, over packed keys and values (k, v; key_starts) or a paged cache (pool, table,
// lens).  Byte strides of tokens and heads.
struct RowsArgs {
  PagedPool pool;
  PagedTable table;
  const int32_t* lens;
  const unsigned char* k;
  const unsigned char* v;
  int64_t kt, kh, vt, vh;
  const int32_t* key_starts;
  const unsigned char* q;
  unsigned char* out;
  int64_t qt, qh, ot, oh;
  float* lse;  // or NULL
  int64_t lt, lh;
  const int32_t* starts;
  const int64_t* masks;  // or NULL: a token sees the rows up to its own, where causal
  float* part_o;         // [workgroups][tile rows][head_dim]: a part's sum of p v, relative to its maximum
  float* part_ml;        // [workgroups][tile rows][2]: its maximum (of q k) and sum
  uint32_t* part_units;  // units that a part has at most, before all of these
  int32_t batch, tokens, key_rows, heads, group, head_dim, max_len, causal;
  int32_t slots, least;  // workgroups that the parts of tiles should fill (0: tiles are whole), units a part has at least
  int64_t tiles, workgroups;  // at most: tiles of all sequences, workgroups of the call
  Div32 group_div, heads_div;
  float scale, scale_log2e;  // of |scale|: its sign is q's (q_xor), a scale of 0 is a q of 0 (q_and)
  uint32_t q_and, q_xor;
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

struct ResizeArgs {
  PagedTable table;
  int32_t* table_out;  // its entries
  const int32_t* lens;
  const int32_t* change;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* lens_out;
  int32_t* count_out;
  int32_t* missing;    // or NULL
  int32_t* starts;     // or NULL, as slots and positions
  int64_t* slots;
  int32_t* positions;
  int32_t capacity, tokens;
  Div32 page;
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

// How a call of attention of several rows is dealt out: query rows in tiles of tile_rows, key rows in units of unit_rows, the
// card filled by parts of tiles (slots, least as in RowsArgs) where tiles are few.
struct RowsShape {
  int64_t tile_rows, unit_rows, tiles, slots, least, workgroups, bytes;
  bool many;  // tiles are numbered as those of many sequences
};
// Lanes of a workgroup: eight waves for wide heads and the largest tiles, else four, as for many sequences' 8-bit rows.
constexpr int64_t rows_threads(bool codes, int64_t head_dim, int64_t tile_rows, bool many) {
  return (head_dim > 128 && !(many && codes)) || tile_rows == 256 ? 512 : 256;
}
constexpr int64_t kRowsWorkspaceHead = 256;  // bytes: a number, and the parts on lines of their own
RowsShape rows_shape(bool paged, bool codes, int64_t batch, int64_t tokens, int64_t heads, int64_t group, int64_t head_dim, int64_t max_len);
// Bytes that suffice for the parts of tiles at these sizes and at any smaller batch, tokens and max_len.
int64_t rows_workspace(int64_t batch, int64_t tokens, int64_t heads, int64_t group, int64_t head_dim, int64_t max_len);

// A launch counts its lanes in 32 bits.
constexpr bool launchable(int64_t workgroups, int64_t threads) { return workgroups * threads < int64_t(1) << 32; }

// Launchers: TC_OK, or TC_E_RANGE, and nothing launched, where a grid would be too large.  `dtype` is that of the new rows or of
// q, `cache_dtype` the pool's; `wide`: new rows take 16-byte loads.
int launch_paged_append(const AppendArgs& a, int dtype, int cache_dtype, bool wide, void* stream);
int launch_paged_attention(const AttentionArgs& a, int dtype, int cache_dtype, void* stream);
int launch_paged_evict(const EvictArgs& a, int cache_dtype, void* stream);
int launch_prompt_attention(const RowsArgs& a, const RowsShape& shape, int dtype, void* stream);
int launch_tree_attention(const RowsArgs& a, const RowsShape& shape, int dtype, int cache_dtype, void* stream);
int launch_paged_resize(const ResizeArgs& a, void* stream);

}  // namespace tc
