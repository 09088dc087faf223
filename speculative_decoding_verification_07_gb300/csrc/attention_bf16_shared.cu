// Tensor-core attention over bf16 caches and shared prefixes: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_bf16_shared(int head_dim, int tiles) { return tc_kernel<false, kShare>(head_dim, tiles); }

}  // namespace sv
