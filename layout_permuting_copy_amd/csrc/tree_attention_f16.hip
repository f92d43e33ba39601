#include "tree_attention.hpp"

namespace tc {
void tree_attention_f16(const RowsArgs& a, const RowsShape& shape, hipStream_t s) { dev::tree_by_dim<false, 1>(a, shape, s); }
}  // namespace tc
