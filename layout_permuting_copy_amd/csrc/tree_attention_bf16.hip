#include "tree_attention.hpp"

namespace tc {
void tree_attention_bf16(const RowsArgs& a, const RowsShape& shape, hipStream_t s) { dev::tree_by_dim<true, 1>(a, shape, s); }
}  // namespace tc
