// What the attention kernels share: parameters, a request's extent, mask bits,
// and the joining of partial results.
#pragma once

#include "entries.cuh"

namespace sv {

struct AttnParams {
  sv_attention_args a;
  float* part;      // partial results of split rows
  uint32_t* ticket; // arrivals per shared item, zero between calls
  int* err;
  int splits;
};

// A request's extent: S cached positions, then n + 1 entries (n = -1: none).
// What does not fit its table or its rows is reported and left without rows.
struct Extent {
  int S, n;
};

__device__ __forceinline__ Extent extent_of(const sv_attention_args& a, int b, int* err) {
  Extent x = {a.seq_len[b], a.n_nodes ? a.n_nodes[b] : a.R - 1};
  const int64_t last = (int64_t)x.S + (a.stage.data ? 0 : x.n + 1);
  if (x.n < 0) x.n = -1;
  if (x.S < 0 || x.n >= a.R || last > (int64_t)a.cache.max_blocks * a.cache.block_size) {
    report(err, SV_ERR_STATE);
    x.n = -1;
  }
  return x;
}

// Bits u .. u + 31 of what row i sees, u counted from entry 0: everything below
// it (the cached positions), the mask's bits for entries 0 .. n, nothing after.
__device__ __forceinline__ uint32_t seen_bits(const sv_attention_args& a, int b, int i, int n, int u) {
  if (u + 32 <= 0) return 0xFFFFFFFFu;
  if (u > n) return 0;
  const int lo = u < 0 ? 0 : u;
  uint32_t w;
  if (a.mask) {
    const uint32_t* row = a.mask + ((int64_t)b * a.R + i) * a.mask_ld;
    const int k = lo >> 5;
    const uint32_t w0 = row[k], w1 = (k + 1) * 32 <= n ? row[k + 1] : 0u;
    w = __funnelshift_r(w0, w1, lo & 31);
  } else {
    w = i - lo >= 31 ? 0xFFFFFFFFu : i < lo ? 0u : (2u << (i - lo)) - 1u;
  }
  if (n - lo < 31) w &= (2u << (n - lo)) - 1u;
  return u < 0 ? w << -u | ((1u << -u) - 1u) : w;
}

// Position of entry i past S_b, for distances.
__device__ __forceinline__ int depth_of(const sv_attention_args& a, int b, int i) {
  return a.depth ? min(max(__ldg(a.depth + (int64_t)b * a.R + i), 0), a.R - 1) : i;
}

// The first cached position that any row of request b may see: no row sits before S.
__device__ __forceinline__ int first_seen(const sv_attention_args& a, int S) { return a.window > 0 ? max(0, S - a.window + 1) : 0; }

// The positions that request b shares with its group, whole blocks.
__device__ __forceinline__ int shared_of(const sv_attention_args& a, int b) {
  const int n = a.shared_len[b], S = a.seq_len[b];
  return n <= 0 || n > S || S > (int64_t)a.cache.max_blocks * a.cache.block_size ? 0 : n / a.cache.block_size * a.cache.block_size;
}

}  // namespace sv
