// The list of items of attention calls with forms of the scores or shared prefixes.
//
// With every CTA counting for itself, as the plain calls do, a call of 256 requests in
// groups spent 15 us before its first tile (each group's members are looked up), and the
// places of items 5000 to 10000 cycles each on the way; so one CTA makes a list, in
// a few microseconds that are latency alone (4 to 7 us after other work, in part under the
// attention's own start), and the attention's CTAs find their place in it.
#include "attention_plan.cuh"

namespace sv {

constexpr int kPlanThreads = 1024, kRangeThreads = 256;

// Inclusive over the block's threads: the sums of x and y and the maxima of m; w: scratch of as
// many words as warps for each.
struct Scan {
  int x, y, m;
};
__device__ __forceinline__ Scan block_scan(Scan s, int (&w)[3][32], int* all_x, int* all_y) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, s.x, o), y = __shfl_up_sync(0xFFFFFFFFu, s.y, o), m = __shfl_up_sync(0xFFFFFFFFu, s.m, o);
    if (lane >= o) s.x += x, s.y += y, s.m = max(s.m, m);
  }
  if (lane == 31) w[0][warp] = s.x, w[1][warp] = s.y, w[2][warp] = s.m;
  __syncthreads();
  const bool is = lane < (int)blockDim.x / 32, before = lane < warp;
  const int x = is ? w[0][lane] : 0, y = is ? w[1][lane] : 0, m = before ? w[2][lane] : INT32_MIN;
  *all_x = __reduce_add_sync(0xFFFFFFFFu, x), *all_y = __reduce_add_sync(0xFFFFFFFFu, y);
  s.x += __reduce_add_sync(0xFFFFFFFFu, before ? x : 0), s.y += __reduce_add_sync(0xFFFFFFFFu, before ? y : 0);
  s.m = max(s.m, __reduce_max_sync(0xFFFFFFFFu, m));
  __syncthreads();
  return s;
}

// How many requests of a group share an item.  More of them read the prefix less often,
// but their rows fill the tile: 32 rows are weighed by all warps together, and a tile of own
// keys is weighed by the warps of one request alone.  In hundreds of cycles a tile and
// CTA, from the attention's own clocks (two streams): prefixes, which come from L2,
// 10, 12 and 18 for up to 32, 64 and 128 rows (15, 19, 27 in 8 bits), own keys 28, 28
// and 36 (19, 25, 40), an item's start and end 80.
__device__ __forceinline__ int lot_size(const TcPlanning& p, int size, int shared, int boxes) {
  const int rows = p.a.R * p.group;
  if (rows > p.rows / 2) return 1;  // prompts
  const bool f8 = p.a.cache.format == SV_KV_E4M3;
  const float tiles = (float)((shared + kTile - 1) / kTile), own = (float)boxes * (float)(1 << p.shift) / kTile;
  int best = 1;
  float least = __int_as_float(0x7F800000);
  for (int c = 0; c < 3; ++c) {
    const int most = min(kMembers, max(1, (32 << c) / rows)), n = (size + most - 1) / most, filled = (size + n - 1) / n * rows;
    const float pre = filled <= 32 ? (f8 ? 15 : 10) : filled <= 64 ? (f8 ? 19 : 12) : f8 ? 27 : 18;
    const float one = filled <= 32 ? (f8 ? 19 : 28) : filled <= 64 ? (f8 ? 25 : 28) : f8 ? 40 : 36;
    const float cost = n * (80.0f + tiles * pre) + (own + 0.5f * n) * one;
    if (cost < least) least = cost, best = most;
  }
  return best;
}

// Lots of requests in their order, blockDim.x requests at a time.  A group is cut into equal
// lots; a lot's first request has it.  (A lot ends where groups overlap or disagree, so
// that every request is in one lot at most, whatever the arrays hold; such groups are
// reported.)  Then the CTAs' shares are equal numbers of units, and each gets the lot in
// which its share starts.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ TcPlanning p) {
  pdl_wait();
  pdl_trigger();
  const sv_attention_args& a = p.a;
  __shared__ int s_boxes[kPlanThreads + kMembers], s_shared[kPlanThreads + kMembers], s_starts[kPlanThreads + kMembers],
      s_rows[kPlanThreads + kMembers], s_sum[kPlanThreads], s_first[kPlanThreads], s_cum[kPlanThreads], s_w[3][32], s_items;
  if (threadIdx.x == 0) s_items = 0;
  const int tid = threadIdx.x, threads = blockDim.x, rows = a.R * p.group;
  int units = 0, lots = 0;
  int first0 = -1;  // the nearest request before these that starts a group
  for (int base = 0; base < a.B; base += threads) {
    const int b = base + tid;
    bool grouped = false;
    TcLot lot = {};
    if (p.sharing) {
      for (int x = tid; x < threads + kMembers; x += threads) {
        int boxes = 0, shared = 0, starts = 0, have = 0;
        if (base + x < a.B) {
          const Extent E = extent_of(a, base + x, x < threads ? p.err : nullptr);
          shared = shared_of(a, base + x), starts = a.shared_members[base + x];
          boxes = own_boxes(a, p.box, p.shift, shared, E), have = E.n + 1;
        }
        s_boxes[x] = boxes, s_shared[x] = shared, s_starts[x] = starts, s_rows[x] = have;
      }
      __syncthreads();
      int all, none;
      const Scan so_far = block_scan({s_boxes[tid], 0, s_starts[tid] > 0 ? b : first0}, s_w, &all, &none);
      const int first = so_far.m;
      s_sum[tid] = so_far.x, s_first[tid] = first;
      __syncthreads();
      const int before = tid > 0 ? s_first[tid - 1] : first0;
      if (b < a.B) {
        const int size = first < 0 ? 0 : min(a.shared_members[first], a.B - first), at = b - first;
        bool bad = s_starts[tid] < 0 || s_starts[tid] > a.B - b;
        grouped = size > 1 && at < size && s_shared[tid] > 0;
        if (first >= 0 && at < size) bad |= s_shared[tid] != shared_of(a, first);
        if (s_shared[tid] > 0 && at >= size) bad = true;  // in no group
        if (s_starts[tid] > 0 && before >= 0) bad |= a.shared_members[before] > b - before;  // or starts one inside another
        if (bad) report(p.err, SV_ERR_STATE);
        if (grouped) {
          int most = max(1, p.rows / rows);
          if (first >= base && first + size <= base + threads) {  // all here
            const int own = s_sum[first + size - 1 - base] - (first > base ? s_sum[first - 1 - base] : 0);
            most = lot_size(p, size, s_shared[first - base], own);
          }
          most = min(most, kMembers);
          const int n = (size + most - 1) / most, each = (size + n - 1) / n;
          if (at % each == 0) {
            int boxes = 0, m = 0, live = 0;
            for (int j = 0; j < min(each, size - at); ++j) {
              if (s_shared[tid + j] != s_shared[tid] || (j > 0 && s_starts[tid + j] > 0)) break;
              boxes += s_boxes[tid + j], live += s_rows[tid + j], m = j + 1;
            }
            const int tp = (s_shared[tid] + kTile - 1) / kTile;
            lot = {b, m, boxes, s_shared[tid], m * a.R - 1, 0, p.lead + tp + ((boxes + (kTile >> p.shift) - 1) >> (7 - p.shift)), tp,
                   (m * rows + p.rows - 1) / p.rows, 0, 0, 0};
            if (live > 0) lot.units = lot.T * a.cache.heads * lot.blocks;
          }
        }
      }
    }
    if (b < a.B && !grouped) {
      const Extent E = extent_of(a, b, p.err);
      const int begin = first_seen(a, E.S) & -p.box;  // a TMA box starts at a multiple of its rows
      const int tp = (E.S - begin + (a.stage.data ? 0 : E.n + 1) + kTile - 1) / kTile;
      lot = {b, 0, 0, E.S, E.n, begin, p.lead + tp + (a.stage.data ? (E.n + kTile) / kTile : 0), tp, ((E.n + 1) * p.group + p.rows - 1) / p.rows, 0, 0, 0};
      if (p.ranges && lot.blocks > 1) {  // units before each row block; they hold each one's own
        int* cum = p.ranges + (int64_t)b * p.words;
        int sum = 0;
        cum[0] = 0;
        for (int r0 = 1; r0 <= lot.blocks; r0 += 16) {
          int t[16];
#pragma unroll
          for (int r = 0; r < 16; ++r) t[r] = r0 + r <= lot.blocks ? cum[r0 + r] : 0;
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (r0 + r <= lot.blocks) cum[r0 + r] = sum += t[r];
        }
        lot.T = sum, lot.units = sum * a.cache.heads;
      } else if (E.n >= 0) {
        lot.units = lot.T * a.cache.heads * lot.blocks;
      }
    }
    int n, u;
    const Scan so_far = block_scan({lot.units > 0, lot.units, 0}, s_w, &n, &u);
    if (lot.units > 0) {
      const int at = lots + so_far.x - 1;
      lot.cum = units + so_far.y - lot.units;
      p.lots[at] = lot;
      if (at < kPlanThreads) s_cum[at] = lot.cum;
      atomicAdd(&s_items, a.cache.heads * lot.blocks);
    }
    lots += n, units += u;
    if (p.sharing) first0 = s_first[threads - 1];
    __syncthreads();
  }
  // short items stay whole, but where there are few of them
  if (tid == 0) p.head[0] = units, p.head[1] = lots, p.head[2] = p.lead + (s_items <= p.ctas / 4 ? kWholeOne : kWhole);
  // the lot that holds the first unit of each CTA's share: the last that starts at or before it
  const int ctas = units > 0 ? sharing_ctas(a, p.group, p.ctas, units) : 0;
  const bool here = lots <= kPlanThreads;
  for (int c = tid; c < p.ctas; c += threads) {
    int lo = 0, hi = lots;
    if (c < ctas) {
      const int w = (int)((uint64_t)(uint32_t)units * (uint32_t)c / (uint32_t)ctas);
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if ((here ? s_cum[mid] : p.lots[mid].cum) <= w) lo = mid; else hi = mid;
      }
    }
    p.first[c] = lo;
  }
}

// Which tiles a row block of a request sees: from the first to the last with a key that
// the mask and the window leave any of its rows, by a CTA each.  Without it a prompt's
// row blocks go through all tiles: the mask hides half of them, a window nearly all.
// Writes the block's units (p.lead and its tiles) and its first tile.  Four prompts of up to
// 2041 entries under a window of 1024: 14 us here, and 1971 -> 392 us for the attention with it (and
// with scores shaped in registers).  Latency of the mask's rows bounds it.
__global__ void __launch_bounds__(kRangeThreads) ranges_kernel(const __grid_constant__ TcPlanning p) {
  pdl_wait();
  pdl_trigger();
  const sv_attention_args& a = p.a;
  const int most_blocks = p.words / 2, b = blockIdx.x / most_blocks, rb = blockIdx.x - b * most_blocks, q = p.rows, G = p.group;
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
#pragma unroll 4
    for (int w = part; w < 32; w += kRangeThreads / 32) {  // a lane an entry
      const int j = (w0 + w) * 32 + lane;
      bool on = s_seen[w] >> lane & 1;
      if (a.window > 0 && on) {
        const int d = depth_of(a, b, j);
        on = d > least - a.window && d - a.window < most;
      }
      const uint32_t left = __ballot_sync(0xFFFFFFFFu, on);
      if (left && lane == 0) atomicMin(&s_from, (w0 + w) * 32 + __ffs(left) - 1), atomicMax(&s_to, (w0 + w) * 32 + 31 - __clz(left));
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
    mine[rb + 1] = p.lead + max(1, hi - lo);
    mine[(p.words + 1) / 2 + rb] = lo;
  }
}

sv_status plan_launch(const TcPlanning& p, cudaStream_t stream) {
  if (p.ranges && sv_launch_pdl(ranges_kernel, dim3((unsigned)(p.words / 2 * p.a.B)), dim3(kRangeThreads), 0, stream, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  const int threads = p.a.B <= 128 ? 128 : p.a.B <= 512 ? 512 : kPlanThreads;
  if (sv_launch_pdl(plan_kernel, dim3(1), dim3((unsigned)threads), 0, stream, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return SV_OK;
}

}  // namespace sv
