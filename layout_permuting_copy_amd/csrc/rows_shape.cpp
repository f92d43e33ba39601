// How attention of several query rows a sequence is dealt out to workgroups, and its workspace.
#include <algorithm>

#include "paged.hpp"

namespace tc {

namespace {

constexpr int64_t kCards = 256;  // compute units
// Workgroups that a compute unit holds: by the LDS that their two tiles of keys and values take.
int64_t resident(int64_t tile, int64_t head_dim) { return head_dim > 128 || (tile == 32 && head_dim > 64) ? 1 : 2; }
int64_t least_tile(int64_t head_dim) { return head_dim > 128 ? 64 : 32; }
int64_t tiles_of(int64_t rows, int64_t batch, int64_t tile) { return std::min(rows, rows / tile + batch); }

}  // namespace

RowsShape rows_shape(bool paged, int64_t batch, int64_t tokens, int64_t heads, int64_t group, int64_t head_dim, int64_t max_len) {
  RowsShape c{};
  const int64_t rows = tokens * group;
  if (paged) {
    // a cache's rows are read once a tile: tiles that hold a sequence's query rows
    c.tile_rows = least_tile(head_dim);
    while (c.tile_rows < 128 && c.tile_rows * batch < rows) c.tile_rows *= 2;
  } else {
    // tiles of 64 rows until larger ones would be four a compute unit: how evenly the last of them end counts for more than
    // that their keys and values are loaded half as often (a prompt of 1024 tokens, 32 heads of 128 over 8: 27 us, in tiles
    // of 128 rows 42; of 4096: 174 and 164).  Heads above 128 elements want eight waves, two a SIMD with 256 registers each
    // (8192 tokens of 256: 1046 us; four waves with 512 each, 1757)
    const int64_t most = head_dim > 128 ? 256 : 128;
    c.tile_rows = tiles_of(rows, batch, most) * heads >= 4 * kCards ? most : 64;
  }
  c.unit_rows = c.tile_rows == 32 ? 128 : 64;
  c.tiles = tiles_of(rows, batch, c.tile_rows);
  c.workgroups = c.tiles * heads;
  const int64_t fill = kCards * resident(c.tile_rows, head_dim);
  if (paged && c.workgroups < 2 * fill && max_len > 512) {
    c.slots = fill;
    c.least = 256 / c.unit_rows;
    c.workgroups += fill + heads;
  }
  return c;
}

int64_t rows_workspace(int64_t batch, int64_t tokens, int64_t heads, int64_t group, int64_t head_dim, int64_t max_len) {
  if (max_len <= 512) return 0;
  int64_t most = 0;
  // (tiles grow as long as their halves do not hold a sequence's rows)
  for (int64_t tile = least_tile(head_dim); tile <= 128 && (tile == least_tile(head_dim) || tile / 2 < tokens * group); tile *= 2) {
    const int64_t fill = kCards * resident(tile, head_dim);
    const int64_t workgroups = std::min(tiles_of(tokens * group, batch, tile) * heads, 2 * fill) + fill + heads;
    most = std::max(most, workgroups * tile * (head_dim + 2) * 4);
  }
  return tokens * group == 0 || batch == 0 ? 0 : most;
}

}  // namespace tc
