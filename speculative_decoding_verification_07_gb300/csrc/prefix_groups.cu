// Which neighbouring requests hold the same leading blocks.
#include "common.cuh"

namespace sv {

constexpr int kPrefixThreads = 256, kGroupThreads = 1024;
constexpr int kClusterCtas = 8, kClusterRequests = kClusterCtas * kGroupThreads / 32;  // a warp each

// How many leading blocks request b has in common with its left neighbour, by one
// CTA each: the first entry at which the two table rows differ, 1024 entries at a
// time.  A row's loads are one trip to memory, which is all that it costs.  shared_len gets
// the positions of these blocks, 0 where the request starts a group.
__global__ void __launch_bounds__(kPrefixThreads) common_blocks_kernel(const int32_t* __restrict__ seq_len,
                                                                       const int32_t* __restrict__ table, int max_blocks,
                                                                       int block_size, int least, int32_t* shared_len, int* err) {
  pdl_wait();
  pdl_trigger();
  constexpr int kEach = 4;
  const int b = blockIdx.x;
  const int64_t room = (int64_t)max_blocks * block_size;
  const int S = seq_len[b], left = b > 0 ? seq_len[b - 1] : 0;
  const bool bad = S < 0 || S > room;
  int most = bad || b == 0 || left < 0 || left > room ? 0 : min(S, left) / block_size;
  const int32_t* row = table + (int64_t)b * max_blocks;
  for (int j0 = 0; j0 < most; j0 += kEach * kPrefixThreads) {
    int x[kEach], y[kEach], differs = INT32_MAX;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int j = j0 + e * kPrefixThreads + threadIdx.x;
      x[e] = y[e] = 0;
      if (j < most) x[e] = row[j], y[e] = row[j - max_blocks];
    }
#pragma unroll
    for (int e = kEach - 1; e >= 0; --e)
      if (x[e] != y[e] || x[e] < 0) differs = j0 + e * kPrefixThreads + (int)threadIdx.x;
    __shared__ int s_first;
    if (threadIdx.x == 0) s_first = most;
    __syncthreads();
    const int first = __reduce_min_sync(0xFFFFFFFFu, differs);
    if (threadIdx.x % 32 == 0 && first < most) atomicMin(&s_first, first);
    __syncthreads();
    const int found = s_first;
    __syncthreads();
    if (found < most) {
      most = found;
      break;
    }
  }
  if (threadIdx.x == 0) {
    if (bad) report(err, SV_ERR_STATE);
    const int n = most * block_size;  // at most S
    shared_len[b] = n > 0 && n >= least ? n : 0;
  }
}

// Groups from the neighbours' common positions: a warp finds the end and the least
// of each group that starts at one of its requests, 32 members at a time.  What
// other warps still read is written after all have read: the first sweep leaves a
// group's size and least in its first two members' words, which every group of two
// has.  One CTA, since a batch is a few hundred requests: latency bounds it.
__global__ void __launch_bounds__(kGroupThreads) groups_kernel(int B, int32_t* shared_len, int32_t* members) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kGroupThreads / 32;
  for (int b = warp; b < B; b += warps) {
    if (shared_len[b] != 0) continue;
    int least = INT32_MAX, e = b + 1;
    while (true) {
      const int x = e + lane < B ? shared_len[e + lane] : 0;
      const uint32_t ends = __ballot_sync(0xFFFFFFFFu, x == 0);
      const int n = ends ? __ffs(ends) - 1 : 32;
      if (lane < n) least = min(least, x);
      e += n;
      if (n < 32) break;
    }
    least = __reduce_min_sync(0xFFFFFFFFu, least);
    for (int j = b + lane; j < e; j += 32)
      members[j] = e - b < 2 ? 0 : j == b ? e - b : j == b + 1 ? least : 0;
  }
  __syncthreads();
  for (int b = warp; b < B; b += warps) {
    if (shared_len[b] != 0) continue;
    const int n = members[b];
    if (n == 0) continue;
    const int least = members[b + 1];
    __syncwarp();
    for (int j = b + lane; j < b + n; j += 32) shared_len[j] = least;
    if (lane == 0) members[b + 1] = 0;
  }
}

// Both steps in one launch of one cluster, for up to 256 requests, a warp each: 256 entries
// of its row and its left neighbour's at a time; then the first CTA makes the groups from
// shared memory.  One launch less on the host, which bounds small calls: 4 requests 8.4 us with
// two launches, 256 of 512 blocks 8.4.  More requests would wait for one another's warps.
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kGroupThreads)
    prefix_groups_kernel(int B, const int32_t* __restrict__ seq_len, const int32_t* __restrict__ table, int max_blocks, int block_size,
                         int least, int32_t* shared_len, int32_t* members, int* err) {
  pdl_wait();
  pdl_trigger();
  constexpr int kEach = 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x + kClusterCtas * warp;
  if (b < B) {
    const int64_t room = (int64_t)max_blocks * block_size;
    const int S = seq_len[b], left = b > 0 ? seq_len[b - 1] : 0;
    const bool bad = S < 0 || S > room;
    int most = bad || b == 0 || left < 0 || left > room ? 0 : min(S, left) / block_size;
    const int32_t* row = table + (int64_t)b * max_blocks;
    for (int j0 = 0; j0 < most; j0 += kEach * 32) {
      int x[kEach], y[kEach], differs = INT32_MAX;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int j = j0 + e * 32 + lane;
        x[e] = y[e] = 0;
        if (j < most) x[e] = row[j], y[e] = row[j - max_blocks];
      }
#pragma unroll
      for (int e = kEach - 1; e >= 0; --e)
        if (x[e] != y[e] || x[e] < 0) differs = j0 + e * 32 + lane;
      differs = __reduce_min_sync(0xFFFFFFFFu, differs);
      if (differs < most) {
        most = differs;
        break;
      }
    }
    if (lane == 0) {
      if (bad) report(err, SV_ERR_STATE);
      const int n = most * block_size;  // at most S
      __stcg(shared_len + b, n > 0 && n >= least ? n : 0);
    }
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (blockIdx.x != 0) return;
  __shared__ int s_common[kClusterRequests];
  for (int i = threadIdx.x; i < B; i += kGroupThreads) s_common[i] = __ldcg(shared_len + i);
  __syncthreads();
  for (int i = warp; i < B; i += kGroupThreads / 32) {
    if (s_common[i] != 0) continue;
    int fewest = INT32_MAX, e = i + 1;
    while (true) {
      const int x = e + lane < B ? s_common[e + lane] : 0;
      const uint32_t ends = __ballot_sync(0xFFFFFFFFu, x == 0);
      const int n = ends ? __ffs(ends) - 1 : 32;
      if (lane < n) fewest = min(fewest, x);
      e += n;
      if (n < 32) break;
    }
    fewest = __reduce_min_sync(0xFFFFFFFFu, fewest);
    for (int j = i + lane; j < e; j += 32) shared_len[j] = e - i < 2 ? 0 : fewest, members[j] = j == i && e - i > 1 ? e - i : 0;
  }
}

static bool overlap(const void* p, size_t n, const void* q, size_t m) {
  return (uintptr_t)p < (uintptr_t)q + m && (uintptr_t)q < (uintptr_t)p + n;
}

}  // namespace sv

using namespace sv;

extern "C" sv_status sv_prefix_groups(sv_handle* h, int32_t B, const int32_t* seq_len, const int32_t* table,
                                      int32_t max_blocks, int32_t block_size, int32_t least, int32_t* shared_len,
                                      int32_t* members, sv_stream_t stream) {
  if (!h || B < 0 || max_blocks < 0 || block_size < 1) return SV_ERR_INVALID;
  if (B == 0) return SV_OK;
  if (!seq_len || (!table && max_blocks) || !shared_len || !members) return SV_ERR_INVALID;
  const size_t row = (size_t)B * 4;  // what one CTA writes others still read
  for (const int32_t* out : {shared_len, members})
    if (overlap(out, row, seq_len, row) || overlap(out, row, table, row * (size_t)max_blocks) || (out == members && overlap(out, row, shared_len, row)))
      return SV_ERR_INVALID;
  if (B <= kClusterRequests) {
    if (sv_launch_pdl(prefix_groups_kernel, dim3(kClusterCtas), dim3(kGroupThreads), 0, (cudaStream_t)stream, B, seq_len, table, max_blocks,
                      block_size, least, shared_len, members, h->d_err) != cudaSuccess) {
      (void)cudaGetLastError();
      return SV_ERR_CUDA;
    }
    return SV_OK;
  }
  if (sv_launch_pdl(common_blocks_kernel, dim3((unsigned)B), dim3(kPrefixThreads), 0, (cudaStream_t)stream, seq_len, table,
                    max_blocks, block_size, least, shared_len, h->d_err) != cudaSuccess ||
      sv_launch_pdl(groups_kernel, dim3(1), dim3(kGroupThreads), 0, (cudaStream_t)stream, B, shared_len, members) != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return SV_OK;
}
