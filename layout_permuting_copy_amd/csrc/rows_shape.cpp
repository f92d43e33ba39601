// How attention of several query rows a sequence is dealt out to workgroups, and its workspace.
#include <algorithm>

#include "paged.hpp"

namespace tc {

namespace {

constexpr int64_t kCus = 256;
// Workgroups that a compute unit holds: one of eight waves (heads above 128 elements, tiles of 256 rows), else two of four, or three.
int64_t resident(bool paged, int64_t head_dim, int64_t tile) { return head_dim > 128 || tile == 256 ? 1 : head_dim > 64 || !paged ? 2 : 3; }
int64_t least_tile(int64_t head_dim) { return head_dim > 128 ? 128 : 64; }
int64_t tiles_of(int64_t rows, int64_t batch, int64_t tile) { return std::min(rows, rows / tile + batch); }

}  // namespace

RowsShape rows_shape(bool paged, bool codes, int64_t batch, int64_t tokens, int64_t heads, int64_t group, int64_t head_dim, int64_t max_len) {
  RowsShape c{};
  const int64_t rows = tokens * group;
  if (paged) {
    // A cache's rows are read once a tile: tiles that hold a sequence's query rows, of 128 from half that many on (32 trees of
    // 26 tokens, 4 heads a group: 69 us, in tiles of 64 rows, whose bf16 weights keep more bits, 84).  Half empty ones cost more
    // than the rows read twice save from there down (16 trees of 64 rows over 8-bit caches: 112 us, in tiles of 128 rows 160).
    c.tile_rows = least_tile(head_dim);
    while (c.tile_rows < 128 && c.tile_rows * batch < 2 * rows) c.tile_rows *= 2;
    // ... and of 256, by eight waves, once they are full (trees of 64 tokens, 8 heads a group, over 65536 rows: 356 -> 312 us;
    // chunks of 1024 tokens over 16384: 636 -> 566; of 300, heads of 256: 355 -> 284).  Not of narrow heads, as of
    // prompts, nor of wide 8-bit ones, for which the registers do not suffice.
    if (head_dim > 64 && !(codes && head_dim > 128) && rows >= 256 * batch) c.tile_rows = 256;
  } else {
    // Larger tiles load their keys and values less often, smaller ones end more evenly: tiles of 128 rows once they are four a
    // compute unit (1024 tokens, 32 heads of 128 over 8: 42 us, in tiles of 64 rows 27; 4096 tokens 164 and 174), of 256 once
    // they are two and a sequence's rows fill eight of them (16384 tokens: 2155 us, in tiles of 128 rows 2255), but for
    // narrow heads, which wait for their exponentials (of 64 elements: 1595 and 1497 us).
    c.tile_rows = least_tile(head_dim);
    if (tiles_of(rows, batch, 128) * heads >= 4 * kCus) c.tile_rows = 128;
    if (head_dim > 64 && tiles_of(rows, batch, 256) * heads >= 2 * kCus && rows >= 2048 * batch) c.tile_rows = 256;
  }
  // Tiles that leave half of the card idle are split over their keys: a cache's always, unless they are short (trees of 8 tokens, 32
  // heads over 8, whole and split, us: one over 256 rows 13.4 and 16.2, over 512 19.6 and 16.5, over 1024 31.8 and 17.6; 8 over 256
  // 13.6 and 17.3, over 512 19.9 and 18.7, over 1024 33.0 and 22.7; 32 over 512 22.0 and 28.2, over 1024 34.6 and 37.4), a prompt's where
  // its keys (`max_len` is their mean) are long enough for the joining to pay (64 tokens of 32 heads over 8, 8064 keys: 145 us,
  // split 33; 512 of 8 over 1, 4608 keys: 85 and 35; 1024 causal tokens of 8 over 8: 24 and 27).  Prompts whose tiles come to
  // more are faster whole (2048 tokens of 16 heads of 256 over 4: 86 us, split 92).
  bool split = max_len > 512;
  if (!paged) split = max_len > 1536 && 2 * tiles_of(rows, batch, c.tile_rows) * heads <= kCus * resident(paged, head_dim, c.tile_rows);
  c.unit_rows = 64;
  c.tiles = tiles_of(rows, batch, c.tile_rows);
  c.workgroups = c.tiles * heads;
  const int64_t fill = kCus * resident(paged, head_dim, c.tile_rows);
  if (split && c.workgroups < 2 * fill) {
    c.slots = fill;
    c.least = 2;  // (one tree of 8 tokens over 523 rows: 16.7 us, at least 4 units a part 18.6, one 17.1)
    // all parts fit the least multiple of `fill` that the tiles do
    c.workgroups = (c.workgroups + fill - 1) / fill * fill;
    c.bytes = kRowsWorkspaceHead + c.workgroups * c.tile_rows * (head_dim + 2) * 4;
  } else if (batch > 12288 || (c.tile_rows < 256 && batch > std::max<int64_t>(1024, 8 * max_len))) {
    // Adding up the tiles before its own costs a workgroup time in proportion to the sequences; finding them by numbers, a few
    // steps, with a number for nobody a sequence where tiles are full, and the least tiles, which read long keys more often.
    // (Added up and numbered, us: 2049 prompts of 8 tokens, 8 heads, 657 and 182, 1025 of 32, 32 heads over 8, 320 and 239; 1025
    // trees of 8 tokens, 8 heads over 1, over 128 rows 46 and 51, 1400 64 and 63; with sequences that fill tiles of 256 rows, chunks
    // of 64 tokens, 8 heads over 1: 2049 over 340 rows 614 and 672, 6145 over 2000 6079 and 7173; 32768 prompts of one token, 8
    // heads, 142000 and 2700.)
    c.many = true;
    c.tile_rows = least_tile(head_dim);
    c.tiles = rows / c.tile_rows + batch;  // as RowsWalk::place numbers them
    c.workgroups = c.tiles * heads;
  }
  return c;
}

int64_t rows_workspace(int64_t batch, int64_t tokens, int64_t heads, int64_t group, int64_t head_dim, int64_t max_len) {
  if (max_len <= 512) return 0;
  int64_t most = 0;
  for (int64_t tile = least_tile(head_dim); tile <= 256; tile *= 2) {
    const int64_t fill = kCus * resident(true, head_dim, tile);
    const int64_t workgroups = (std::min(tiles_of(tokens * group, batch, tile) * heads, 2 * fill) + fill - 1) / fill * fill;
    most = std::max(most, kRowsWorkspaceHead + workgroups * tile * (head_dim + 2) * 4);
  }
  return tokens * group == 0 || batch == 0 ? 0 : most;
}

}  // namespace tc
