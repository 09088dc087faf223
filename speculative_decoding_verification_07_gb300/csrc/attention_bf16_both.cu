// Tensor-core attention over bf16 caches and shared prefixes with forms of the scores: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_bf16_both(int head_dim, int tiles) { return tc_kernel<false, kForms | kShare>(head_dim, tiles); }

}  // namespace sv
