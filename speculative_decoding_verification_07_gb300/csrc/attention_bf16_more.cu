// Tensor-core attention over bf16 caches with forms of the scores or
// shared prefixes: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_bf16_more(int head_dim, int tiles) {
  if (head_dim == 64) return tiles == 1 ? tc_kernel<false, 64, 1, true>() : tc_kernel<false, 64, 2, true>();
  return tiles == 1 ? tc_kernel<false, 128, 1, true>() : tc_kernel<false, 128, 2, true>();
}

}  // namespace sv
