// Tensor-core attention over bf16 caches with forms of the scores: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_bf16_forms(int head_dim, int tiles) { return tc_kernel<false, kForms>(head_dim, tiles); }

}  // namespace sv
