// Tensor-core attention over 8-bit caches with forms of the scores or
// shared prefixes: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_e4m3_more(int head_dim, int tiles) {
  if (head_dim == 64) return tiles == 1 ? tc_kernel<true, 64, 1, true>() : tc_kernel<true, 64, 2, true>();
  return tiles == 1 ? tc_kernel<true, 128, 1, true>() : tc_kernel<true, 128, 2, true>();
}

}  // namespace sv
