// Attention of whole prompts: packed sequences, keys and values as the projection left them.
#include "rows_launch.hpp"

namespace tc {
namespace dev {

template <bool BF16, int DP>
void prompt_by_tile(const RowsArgs& a, const RowsShape& shape, hipStream_t s) {
  if (shape.many) return attend_rows<BF16, 0, DP, (DP > 128 ? 4 : 2), (DP > 128 ? 8 : 4), 1, true>(a, s);
  if constexpr (DP > 64)
    if (shape.tile_rows == 256) return attend_rows<BF16, 0, DP, 8, 8, 1>(a, s);
  if constexpr (DP > 128) return attend_rows<BF16, 0, DP, 4, 8, 1>(a, s);
  else if (shape.tile_rows == 128) return attend_rows<BF16, 0, DP, 4, 4, 1>(a, s);
  else return attend_rows<BF16, 0, DP, 2, 4, 1>(a, s);
}

template <bool BF16>
void prompt_by_dim(const RowsArgs& a, const RowsShape& shape, hipStream_t s) {
  if (a.head_dim <= 64) return prompt_by_tile<BF16, 64>(a, shape, s);
  if (a.head_dim <= 96) return prompt_by_tile<BF16, 96>(a, shape, s);
  if (a.head_dim <= 128) return prompt_by_tile<BF16, 128>(a, shape, s);
  if (a.head_dim <= 192) return prompt_by_tile<BF16, 192>(a, shape, s);
  return prompt_by_tile<BF16, 256>(a, shape, s);
}

}  // namespace dev

int launch_prompt_attention(const RowsArgs& a, const RowsShape& shape, int dtype, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (!launchable(a.workgroups, rows_threads(false, a.head_dim, shape.tile_rows, shape.many))) return TC_E_RANGE;
  if (dtype == TC_BF16)
    dev::prompt_by_dim<true>(a, shape, s);
  else
    dev::prompt_by_dim<false>(a, shape, s);
  return TC_OK;
}

}  // namespace tc
