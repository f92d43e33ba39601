// Attention of each sequence's last tokens over its paged cache: the instances of one pair of types.
#pragma once

#include "rows_launch.hpp"

namespace tc {
namespace dev {

// 8-bit rows' weights are bf16 values, as their scales may pass fp16's range: for fp16 queries the sum of two in every tile (one
// holds 8 bits, fewer than out; 16 trees of 12 tokens over 8192 rows 153 us, with one 133).  bf16 queries' are the sum of two in
// tiles of 64 rows of heads of up to 128 elements, whose matrix units wait for memory anyway, else one (32 trees of 26 tokens:
// rms error against 64 bits 0.0022, in tiles of 64 rows 0.0017, which is out's own rounding; over 8-bit rows 0.0023 and 0.0017).
template <bool BF16, int SRC, int DP, int PARTS>
void tree_by_tile(const RowsArgs& a, const RowsShape& shape, hipStream_t s) {
  constexpr int LARGE = SRC == 2 && !BF16 ? 2 : 1;
  // (of many sequences' wide 8-bit rows: eight waves would need scratch memory there)
  if (shape.many) return attend_rows<BF16, SRC, DP, (DP > 128 ? 4 : 2), (DP > 128 && SRC != 2 ? 8 : 4), (DP > 128 ? LARGE : PARTS), true>(a, s);
  if constexpr (DP > 64 && !(SRC == 2 && DP > 128))
    if (shape.tile_rows == 256) return attend_rows<BF16, SRC, DP, 8, 8, LARGE>(a, s);
  if constexpr (DP > 128) return attend_rows<BF16, SRC, DP, 4, 8, LARGE>(a, s);
  else if (shape.tile_rows == 64) return attend_rows<BF16, SRC, DP, 2, 4, PARTS>(a, s);
  else return attend_rows<BF16, SRC, DP, 4, 4, LARGE>(a, s);
}

template <bool BF16, int SRC>
void tree_by_dim(const RowsArgs& a, const RowsShape& shape, hipStream_t s) {
  constexpr int PARTS = BF16 || SRC == 2 ? 2 : 1;
  if (a.head_dim <= 64) return tree_by_tile<BF16, SRC, 64, PARTS>(a, shape, s);
  if (a.head_dim <= 128) return tree_by_tile<BF16, SRC, 128, PARTS>(a, shape, s);
  return tree_by_tile<BF16, SRC, 256, PARTS>(a, shape, s);
}

}  // namespace dev
}  // namespace tc
