// Tensor-core attention over 8-bit caches and shared prefixes: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_e4m3_shared(int head_dim, int tiles) { return tc_kernel<true, kShare>(head_dim, tiles); }

}  // namespace sv
