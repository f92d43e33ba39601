// Attention of each sequence's last tokens over its paged cache: the launch.
#include <hip/hip_runtime.h>

#include "paged.hpp"

namespace tc {

void tree_attention_f16(const RowsArgs& a, const RowsShape& shape, hipStream_t s);
void tree_attention_bf16(const RowsArgs& a, const RowsShape& shape, hipStream_t s);
void tree_attention_e4m3_f16(const RowsArgs& a, const RowsShape& shape, hipStream_t s);
void tree_attention_e4m3_bf16(const RowsArgs& a, const RowsShape& shape, hipStream_t s);

int launch_tree_attention(const RowsArgs& a, const RowsShape& shape, int dtype, int cache_dtype, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (!launchable(a.workgroups, rows_threads(cache_dtype == TC_E4M3, a.head_dim, shape.tile_rows, shape.many))) return TC_E_RANGE;
  const bool bf16 = dtype == TC_BF16;
  if (cache_dtype == TC_E4M3)
    bf16 ? tree_attention_e4m3_bf16(a, shape, s) : tree_attention_e4m3_f16(a, shape, s);
  else
    bf16 ? tree_attention_bf16(a, shape, s) : tree_attention_f16(a, shape, s);
  return TC_OK;
}

}  // namespace tc
