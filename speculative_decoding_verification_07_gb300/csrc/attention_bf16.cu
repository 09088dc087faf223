// Tensor-core attention over bf16 caches: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_bf16(int head_dim, int tiles) { return tc_kernel<false, 0>(head_dim, tiles); }

}  // namespace sv
