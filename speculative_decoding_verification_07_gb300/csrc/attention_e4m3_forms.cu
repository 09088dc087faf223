// Tensor-core attention over 8-bit caches with forms of the scores: instantiations.
#include "attention_tc.cuh"

namespace sv {

TcKernel tc_kernel_e4m3_forms(int head_dim, int tiles) { return tc_kernel<true, kForms>(head_dim, tiles); }

}  // namespace sv
