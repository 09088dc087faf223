// The list of items of attention calls with forms of the scores or shared prefixes.
//
// With every CTA counting for itself, as the plain calls do, a call of 256 requests in
// groups spent 15 us before its first tile (each group's members are looked up), and the
// places of items 5000 to 10000 cycles each on the way; so one CTA makes a list, in
// a few microseconds that are latency alone, and the attention's CTAs find their place in it.
#include "attention_plan.cuh"

namespace sv {

constexpr int kPlanThreads = 1024, kRangeThreads = 256;

// Inclusive sums or maxima over the block's threads; w: 32 words of scratch each.
__device__ __forceinline__ int block_max(int x, int* w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x = max(x, y);
  }
  if (lane == 31) w[warp] = x;
  __syncthreads();
  int before = lane < warp ? w[lane] : INT32_MIN;
  before = __reduce_max_sync(0xFFFFFFFFu, before);
  __syncthreads();
  return max(x, before);
}
__device__ __forceinline__ int block_sum(int x, int* w, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) w[warp] = x;
  __syncthreads();
  const int y = w[lane];
  const int before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? y : 0);
  *all = __reduce_add_sync(0xFFFFFFFFu, y);
  __syncthreads();
  return x + before;
}

// Lots of requests in their order, 1024 requests at a time.  A group is cut into equal
// lots whose rows fill an item at most; its first request has the lot.  (A lot ends where
// groups overlap or disagree, so that every request is in one lot at most, whatever
// the arrays hold; such groups are reported.)
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ TcPlanning p) {
  pdl_wait();
  pdl_trigger();
  const sv_attention_args& a = p.a;
  __shared__ int s_boxes[kPlanThreads + kMembers], s_shared[kPlanThreads + kMembers], s_starts[kPlanThreads + kMembers],
      s_rows[kPlanThreads + kMembers], s_w[32], s_first;
  const int tid = threadIdx.x, rows = a.R * p.group;
  const int widest = p.which & 2 ? 2 * kTile : kTile;
  int units[2] = {0, 0}, lots[2] = {0, 0};
  int first0 = -1;  // the nearest request before these that starts a group
  for (int base = 0; base < a.B; base += kPlanThreads) {
    for (int x = tid; x < kPlanThreads + kMembers; x += kPlanThreads) {
      const int b = base + x;
      int boxes = 0, shared = 0, starts = 0, have = 0;
      if (b < a.B && p.sharing) {
        const Extent E = extent_of(a, b, x < kPlanThreads ? p.err : nullptr);
        shared = shared_of(a, b), starts = a.shared_members[b];
        boxes = own_boxes(a, p.box, p.shift, shared, E), have = E.n + 1;
      }
      s_boxes[x] = boxes, s_shared[x] = shared, s_starts[x] = starts, s_rows[x] = have;
    }
    __syncthreads();
    const int b = base + tid;
    TcLot lot = {};
    int to = p.which == 2;
    bool grouped = false;
    if (p.sharing) {
      const int first = max(first0, block_max(s_starts[tid] > 0 ? b : -1, s_w));
      if (tid == kPlanThreads - 1) s_first = first;
      const int before = max(first0, block_max(tid > 0 && s_starts[tid - 1] > 0 ? b - 1 : -1, s_w));
      if (b < a.B) {
        const int size = first < 0 ? 0 : min(a.shared_members[first], a.B - first), at = b - first;
        bool bad = s_starts[tid] < 0 || s_starts[tid] > a.B - b;
        grouped = size > 1 && at < size && s_shared[tid] > 0;
        if (first >= 0 && at < size) bad |= s_shared[tid] != shared_of(a, first);
        if (s_shared[tid] > 0 && at >= size) bad = true;  // in no group
        if (s_starts[tid] > 0 && before >= 0) bad |= a.shared_members[before] > b - before;  // or starts one inside another
        if (bad) report(p.err, SV_ERR_STATE);
        if (grouped) {
          const int most = min(kMembers, max(1, widest / rows)), n = (size + most - 1) / most, each = (size + n - 1) / n;
          if (at % each == 0) {
            int boxes = 0, m = 0, live = 0;
            for (int j = 0; j < min(each, size - at); ++j) {
              if (s_shared[tid + j] != s_shared[tid] || (j > 0 && s_starts[tid + j] > 0)) break;
              boxes += s_boxes[tid + j], live += s_rows[tid + j], m = j + 1;
            }
            if (p.which == 3) to = m * rows > kTile;
            const int q = to ? 2 * kTile : kTile, tp = (s_shared[tid] + kTile - 1) / kTile;
            lot = {b, m, boxes, s_shared[tid], m * a.R - 1, 0, kLead + tp + ((boxes << p.shift) + kTile - 1) / kTile, tp,
                   (m * rows + q - 1) / q, 0, 0, 0};
            if (live > 0) lot.units = lot.T * a.cache.heads * lot.blocks;
          }
        }
      }
    }
    if (b < a.B && !grouped) {
      const Extent E = extent_of(a, b, p.err);
      const int q = to ? 2 * kTile : kTile, begin = first_seen(a, E.S) & -p.box;  // a TMA box starts at a multiple of its rows
      const int tp = (E.S - begin + (a.stage.data ? 0 : E.n + 1) + kTile - 1) / kTile;
      lot = {b, 0, 0, E.S, E.n, begin, kLead + tp + (a.stage.data ? (E.n + kTile) / kTile : 0), tp, ((E.n + 1) * p.group + q - 1) / q, 0, 0, 0};
      if (p.ranges && lot.blocks > 1) {  // units before each row block; they hold each one's own
        int* cum = p.ranges + (int64_t)b * p.words;
        int sum = 0;
        cum[0] = 0;
        for (int r = 1; r <= lot.blocks; ++r) cum[r] = sum += cum[r];
        lot.T = sum, lot.units = sum * a.cache.heads;
      } else if (E.n >= 0) {
        lot.units = lot.T * a.cache.heads * lot.blocks;
      }
    }
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      if (!(p.which >> l & 1)) continue;
      const bool mine = lot.units > 0 && to == l;
      int n, u;
      const int at = block_sum(mine, s_w, &n), cum = block_sum(mine ? lot.units : 0, s_w, &u);
      if (mine) {
        lot.cum = units[l] + cum - lot.units;
        p.lots[l][lots[l] + at - 1] = lot;
      }
      lots[l] += n, units[l] += u;
    }
    __syncthreads();
    if (p.sharing) first0 = s_first;
  }
  if (tid < 2) p.head[2 * tid] = units[tid], p.head[2 * tid + 1] = lots[tid];
}

// Which tiles a row block of a request sees: from the first to the last with a key that
// the mask and the window leave any of its rows, by a CTA each.  Without it a prompt's
// row blocks go through all tiles: the mask hides half of them, a window nearly all.
// Writes the block's units (kLead and its tiles) and its first tile.
__global__ void __launch_bounds__(kRangeThreads) ranges_kernel(const __grid_constant__ TcPlanning p) {
  pdl_wait();
  pdl_trigger();
  const sv_attention_args& a = p.a;
  const int rb = blockIdx.x, b = blockIdx.y, q = p.which == 2 ? 2 * kTile : kTile, G = p.group;
  const Extent E = extent_of(a, b, nullptr);
  const int blocks = ((E.n + 1) * G + q - 1) / q;
  if (rb >= blocks || blocks < 2) return;
  const int i0 = (int)((int64_t)rb * q / G), i1 = min(E.n, (int)(((int64_t)(rb + 1) * q - 1) / G));
  __shared__ int s_least, s_most, s_from, s_to;
  __shared__ uint32_t s_seen[32];
  if (threadIdx.x == 0) s_least = INT32_MAX, s_most = -1, s_from = INT32_MAX, s_to = -1;
  __syncthreads();
  for (int i = i0 + threadIdx.x; i <= i1; i += kRangeThreads) {
    const int d = depth_of(a, b, i);
    atomicMin(&s_least, d), atomicMax(&s_most, d);
  }
  __syncthreads();
  const int least = s_least, most = s_most, lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  // entries: 32 words of the mask's rows at a time
  for (int w0 = 0; w0 * 32 <= E.n; w0 += 32) {
    if (threadIdx.x < 32) s_seen[threadIdx.x] = 0;
    __syncthreads();
    uint32_t bits = 0;
    if ((w0 + lane) * 32 <= E.n)
#pragma unroll 8
      for (int i = i0 + part; i <= i1; i += kRangeThreads / 32) bits |= seen_bits(a, b, i, E.n, (w0 + lane) * 32);
    if (bits) atomicOr(&s_seen[lane], bits);
    __syncthreads();
    if (part == 0) {
      bits = s_seen[lane];
      if (a.window > 0)
        for (uint32_t left = bits; left; left &= left - 1) {
          const int d = depth_of(a, b, (w0 + lane) * 32 + __ffs(left) - 1);
          if (d <= least - a.window || d - a.window >= most) bits &= ~(left & -left);
        }
      if (bits) atomicMin(&s_from, (w0 + lane) * 32 + __ffs(bits) - 1), atomicMax(&s_to, (w0 + lane) * 32 + 31 - __clz(bits));
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const int begin = first_seen(a, E.S) & -p.box, jmin = s_from, jmax = s_to;
    const bool cached = E.S > 0 && (a.window == 0 || least + 1 < a.window);
    const int x0 = (a.window == 0 ? 0 : max(0, E.S + least - a.window + 1)) - begin;  // the first cached position seen
    const int staged = (E.S - begin + kTile - 1) / kTile;  // tiles before the staged entries'
    int lo = 0, hi = 1;
    if (a.stage.data) {
      if (cached || jmax >= 0) lo = cached ? x0 / kTile : staged + jmin / kTile, hi = jmax >= 0 ? staged + jmax / kTile + 1 : staged;
    } else if (cached || jmax >= 0) {
      lo = (cached ? x0 : E.S - begin + jmin) / kTile, hi = (jmax >= 0 ? E.S - begin + jmax : E.S - begin - 1) / kTile + 1;
    }
    int* mine = p.ranges + (int64_t)b * p.words;
    mine[rb + 1] = kLead + max(1, hi - lo);
    mine[(p.words + 1) / 2 + rb] = lo;
  }
}

sv_status plan_launch(const TcPlanning& p, cudaStream_t stream) {
  if (p.ranges && sv_launch_pdl(ranges_kernel, dim3((unsigned)(p.words / 2), (unsigned)p.a.B), dim3(kRangeThreads), 0, stream, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  if (sv_launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return SV_OK;
}

}  // namespace sv
