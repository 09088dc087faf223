// Ancestor bits and depths of token trees, made once per step for the
// attention, the rotary positions and the logit rules of every layer.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace sv {

// anc(0) = {0}, anc(i) = anc(parent i) + {i}.  One CTA per request keeps the
// parents in shared memory; a warp takes a row, walks its path (every lane
// together, one shared-memory read a step) and each lane keeps the words it
// owns, so a row is written once, coalesced.  The launch is latency: bytes are
// 4 (N + 1) (W + 1) per request.  One tree of 14 nodes 1.4 us, 256 of up to 127 5.2.
// Each row's whole path is walked, and again for every 1024 nodes: nodes x depth
// bound deep trees (chains of 127, 1023 and 4095 nodes 18 us, 0.9 ms, 58 ms).
__global__ void __launch_bounds__(1024) tree_mask_kernel(int N, const int32_t* __restrict__ parent,
                                                         const int32_t* __restrict__ n_nodes,
                                                         uint32_t* __restrict__ mask, int64_t mask_ld,
                                                         int32_t* __restrict__ depth, int* err) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int16_t s_par[];
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < N; i += blockDim.x) {
    int p = parent[(size_t)b * N + i];
    if (p < 0 || p > i) {
      if (!n_nodes || i < n_nodes[b]) report(err, SV_ERR_STATE);
      p = 0;
    }
    s_par[i] = (int16_t)p;
  }
  int n = n_nodes ? n_nodes[b] : N;
  if (n > N) {
    if (threadIdx.x == 0) report(err, SV_ERR_STATE);
    n = N;
  }
  __syncthreads();
  for (int i = warp; i <= N; i += blockDim.x >> 5) {
    uint32_t* row = mask + ((size_t)b * (N + 1) + i) * mask_ld;
    int d = 0;
    for (int64_t w0 = 0; w0 < mask_ld; w0 += 32) {  // one pass for trees of up to 1024 nodes
      uint32_t word = 0;
      d = 0;
      if (i <= n) {
        int j = i;
        while (true) {
          if ((j >> 5) == (int)w0 + lane) word |= 1u << (j & 31);
          if (j == 0) break;
          j = s_par[j - 1];
          ++d;
        }
      }
      if (w0 + lane < mask_ld) row[w0 + lane] = word;
    }
    if (lane == 0) depth[(size_t)b * (N + 1) + i] = d;
  }
}

}  // namespace sv

using namespace sv;

extern "C" sv_status sv_tree_mask(sv_handle* h, int32_t B, int32_t N, const int32_t* parent,
                                  const int32_t* n_nodes, uint32_t* mask, int64_t mask_ld,
                                  int32_t* depth, sv_stream_t stream) {
  if (!h || B < 0 || N < 0 || N > SV_TREE_MAX_NODES || mask_ld < (N + 32) / 32) return SV_ERR_INVALID;
  if (B == 0) return SV_OK;
  if (!mask || !depth || (N > 0 && !parent)) return SV_ERR_INVALID;
  const int threads = N + 1 < 32 ? (N + 1) * 32 : 1024;
  if (sv_launch_pdl(tree_mask_kernel, dim3((unsigned)B), dim3((unsigned)threads), (size_t)N * 2 + 2,
                    (cudaStream_t)stream, (int)N, parent, n_nodes, mask, mask_ld, depth,
                    h->d_err) != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return SV_OK;
}
