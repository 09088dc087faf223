// Tensor-core attention over 8-bit caches: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_e4m3(int head_dim, int tiles) { return tc_kernel<true, 0>(head_dim, tiles); }

}  // namespace sv
