// Choice of the instance of rows_attention_kernel, shared by the files that instantiate it.
#pragma once

#include "rows_attention.hpp"

namespace tc {
namespace dev {

template <bool BF16, int SRC, int DP, int WQ, int WAVES, int PARTS, bool MANY = false>
void attend_rows(const RowsArgs& a, hipStream_t s) {
  typedef Rows<BF16, SRC, DP, WQ, WAVES, PARTS> C;
  static_assert(C::THREADS == rows_threads(SRC == 2, DP, C::BM, MANY), "what the launch is checked for");
  hipLaunchKernelGGL((rows_attention_kernel<BF16, SRC, DP, WQ, WAVES, PARTS, MANY>), dim3(uint32_t(a.workgroups)), dim3(C::THREADS), 0, s, a);
  if constexpr (!MANY && (C::PAGED || C::BM <= 128))  // (prompts in tiles of 256 rows are whole)
    if (a.slots)  // (fewer tiles than two turns of the card's workgroups: no launch is too large for them)
      hipLaunchKernelGGL((rows_join_kernel<BF16, C::PAGED, DP, C::BM, C::KT, C::RAISE>), dim3(uint32_t(a.tiles * a.heads * (C::BM / kJoinRows))),
                         dim3(kRowsThreads), 0, s, a);
}

}  // namespace dev
}  // namespace tc
