// Tensor-core attention over 8-bit caches: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_e4m3(int head_dim, int tiles) {
  if (head_dim == 64) return tiles == 1 ? tc_kernel<true, 64, 1>() : tc_kernel<true, 64, 2>();
  return tiles == 1 ? tc_kernel<true, 128, 1>() : tc_kernel<true, 128, 2>();
}

}  // namespace sv
