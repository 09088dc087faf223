// Tensor-core attention over bf16 caches: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_bf16(int head_dim, int tiles) {
  if (head_dim == 64) return tiles == 1 ? tc_kernel<false, 64, 1>() : tc_kernel<false, 64, 2>();
  return tiles == 1 ? tc_kernel<false, 128, 1>() : tc_kernel<false, 128, 2>();
}

}  // namespace sv
