// Tensor-core attention over 8-bit caches and shared prefixes with forms of the scores: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_e4m3_both(int head_dim, int tiles) { return tc_kernel<true, kForms | kShare>(head_dim, tiles); }

}  // namespace sv
