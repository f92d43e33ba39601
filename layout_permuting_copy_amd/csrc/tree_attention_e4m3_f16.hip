#include "tree_attention.hpp"

namespace tc {
void tree_attention_e4m3_f16(const RowsArgs& a, const RowsShape& shape, hipStream_t s) { dev::tree_by_dim<false, 2>(a, shape, s); }
}  // namespace tc
