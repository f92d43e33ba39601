// Choice of the instance of rows_attention_kernel, shared by the files that instantiate it.
#pragma once

#include "rows_attention.hpp"

namespace tc {
namespace dev {

template <bool BF16, int SRC, int DP, int QT, int WQ, int PARTS>
void attend_rows(const RowsArgs& a, hipStream_t s) {
  typedef Rows<BF16, SRC, DP, QT, WQ, PARTS> C;
  hipLaunchKernelGGL((rows_attention_kernel<BF16, SRC, DP, QT, WQ, PARTS>), dim3(uint32_t(a.workgroups)), dim3(C::THREADS), 0, s, a);
  if (a.slots)
    hipLaunchKernelGGL((rows_join_kernel<BF16, C::PAGED, C::BM, C::KT>), dim3(uint32_t(a.tiles * a.heads * (C::BM / 4))),
                       dim3(kRowsThreads), 0, s, a);
}

}  // namespace dev
}  // namespace tc
