// Attention of a verify pass on the tensor cores: scores and outputs by
// tcgen05.mma with accumulators in tensor memory, K and V by TMA, for bf16 and
// 8-bit caches with heads of 64 or 128.
#pragma once

#include <cuda_fp16.h>

#include "attention.cuh"
#include "attention_plan.cuh"
#include "tcgen05.cuh"

namespace sv {

constexpr int kScaleRing = 4;     // tiles whose scales are held
constexpr int kSegments = 4;      // items whose places are held (calls with forms or shared prefixes)

struct TcParams {
  AttnParams p;
  CUtensorMap pages, stage;  // {column, slot or entry, (layer, K or V, head), block or request}
  CUtensorMap page_tails, stage_tails;  // of 8-bit entries' last 16 bytes, K's and V's in one box
  int box;          // cached positions per TMA box: the largest power of two up to 128 (16 where
                    // requests share prefixes) that divides block_size
  int stage_box;    // staged entries per TMA box: kStageBox, or box where requests share prefixes
  int block_shift;  // log2 of block_size, -1 if it is no power of two
  int group;        // G: query heads of a KV head
  uint32_t group_magic;  // ceil(2^32 / G), 0 for G = 1: a row's entry without a division
  // of calls with forms or shared prefixes
  uint32_t entries_magic;  // the same for R
  int box_shift;           // log2 of box
  bool down;               // items' tiles from the last to the first
  TcList list;             // what plan_kernel made
};

// The instruction cache is shared by roles that run different code at the same
// time: with every wait, walk and division inlined the kernel was 138 KB and
// warps waited for instructions more than for anything else.  Hence the calls
// and the rolled loops below.
__device__ __forceinline__ int block_of(const TcParams& P, int x) {
  return P.block_shift >= 0 ? x >> P.block_shift : x / P.p.a.cache.block_size;
}
__device__ __forceinline__ int entry_of(const TcParams& P, int row) {  // row / G, exact below 2^32 / G rows
  return P.group_magic ? (int)__umulhi((uint32_t)row, P.group_magic) : row;
}

// lo: the item's first tile; rev: t0 + t1 - 1 where tiles go down, else -1.  m > 0: the
// rows of m requests from b on share their first X.S positions, X.n + 1 = m R entries, and
// have nb boxes of their own.
struct TcSegment {
  int b, h, rb, t0, t1, T, tp, item0;  // T: units of the item, item0: where it starts in the list
  Extent X;
  int begin, m, nb, lo, rev;
};

// Requests that share a prefix have their rows in one item, whose tiles are the
// prefix's and then their own keys': boxes of `box` rows, the cached positions past the
// prefix and the staged entries of one request after the other, packed so that a few
// own keys of each do not cost a tile of each.  A row sees the boxes of its own request.
struct TcMembers {
  int start[kMembers + 1];  // the request's first box
  int S[kMembers], n[kMembers];
};
struct TcPlace {
  TcSegment seg;  // T = 0: the end
  int found;      // its tiles of V had non-finite values, now cleared
  uint32_t spoiled[8];  // which of them: a bit for a tile, or for 2^k where they are more than 256
  TcMembers mem;
};
__device__ __forceinline__ int spoiled_bit(const TcSegment& s, int t) { return (t - s.t0) >> max(0, 24 - __clz(s.t1 - s.t0 - 1)); }

// F8: an 8-bit cache.  D: head_dim.  QM: row tiles of 128 per CTA.
//   QM = 1: up to 128 rows; the two streams (score, weight and output regions
//           of tensor memory, each with its softmax group of four warps) take
//           the even and the odd key tiles and are merged at the end.  Up to 64
//           (32) rows fill the tile's 128 twice (four times), and each copy
//           weighs a half (a quarter) of a tile's keys: all warps share the
//           exponentials of a few rows, and a product of 128 rows costs the same.
//   QM = 2: more rows; the streams are two row tiles that share every key tile.
//   kMode: 0, or kForms and kShare: scores have a form, requests share prefixes; items then
//           come from a list made by a kernel before (see attention_plan.cuh).
template <bool F8, int D, int QM, int kMode>
struct TcShape {
  // two softmax groups of four warps; K loads; products; V loads; one for scales
  // and dead rows
  static constexpr int kThreads = 384;
  static constexpr int kRow = F8 ? D : 2 * D;                // bytes of a row without its tail
  static constexpr int kSw = kRow < 128 ? kRow : 128;        // swizzle = bytes of a row per half
  static constexpr int kHalves = kRow / kSw;
  static constexpr int kHalfBytes = kTile * kSw;
  static constexpr int kTileBytes = kTile * kRow;
  static constexpr int kQBytes = kTile * 2 * D;              // bf16 rows, or two 8-bit parts
  static constexpr int kStep = F8 ? 32 : 16;                 // keys of one product of weights and V
  static constexpr int kRows = kTile * QM;
  static constexpr int kQAll = QM * kQBytes > 32768 ? QM * kQBytes : 32768;  // also holds 128 x 64 outputs, 32 of each half
  static constexpr int kMisc = 3072 + 4 * kRows + (F8 ? kScaleRing * 2 * kTile * 4 + 2 * kTile * 4 + (kMode ? 128 : 0) : 0) +
                               (kMode ? kSegments * (int)sizeof(TcPlace) : 0) + (kMode & kForms ? 4 * kTile * 4 : 0);
  // tiles held; a slot of K has its keys' tails and V's
  static constexpr int kTails = F8 ? 2 * kTile * kTail : 0, kKBytes = kTileBytes + kTails;
  static constexpr int kRoom = 232448 - 1024 - kMisc - kQAll, kPairs = kRoom / (kTileBytes + kKBytes);
  static constexpr int kV = kPairs < 6 ? kPairs : 6;
  static constexpr int kK = kPairs < 6 && kRoom - kPairs * (kTileBytes + kKBytes) >= kKBytes ? kV + 1 : kV;
  static constexpr int kSmem = 1024 + kMisc + kQAll + kK * kKBytes + kV * kTileBytes;
  static constexpr int kPart = kRows * (D + 2);              // floats of a partial result
};

// One copy of the division's code for all of the walk (a small call waits for
// instructions to arrive more than for anything else).
static __device__ __noinline__ uint32_t quotient(uint32_t a, uint32_t b) { return a / b; }

struct TcWalk {
  int qrows, w, w1, b, base, T, items, tp, blocks;
  Extent X;
  __device__ __forceinline__ int count() const { return T * items; }
};

// The units of a request of extent X.
static __device__ __noinline__ void plan(const TcParams& P, TcWalk& k, int b, Extent X) {
  const sv_attention_args& a = P.p.a;
  k.b = b, k.X = X;
  k.T = 0, k.items = 0, k.tp = 0, k.blocks = 1;
  if (X.n < 0) return;
  k.blocks = ((X.n + 1) * P.group + k.qrows - 1) >> (k.qrows == kTile ? 7 : 8);
  k.items = a.cache.heads * k.blocks;
  k.tp = (X.S + (a.stage.data ? 0 : X.n + 1) + kTile - 1) / kTile;
  k.T = kLead + (a.stage.data ? k.tp + (X.n + kTile) / kTile : k.tp);
}
static __device__ __forceinline__ void walk_to(const TcParams& P, TcWalk& k, int b) {
  plan(P, k, b, extent_of(P.p.a, b, P.p.err));
}

// floor(x * m / d); small products without a 64-bit division, whose code alone
// takes a cold instruction cache a microsecond.
static __device__ __noinline__ int mul_div(int x, int m, int d) {
  const uint64_t p = (uint64_t)(uint32_t)x * (uint32_t)m;
  if (p >> 32 == 0) return (int)quotient((uint32_t)p, (uint32_t)d);
  return (int)(p / (uint32_t)d);
}

// The next segment (one item's consecutive tiles); false at the end.  A share's
// bounds inside a short item move to the item's nearer end, the same for both
// neighbours: joining its parts would take longer than its tiles.
static __device__ __noinline__ bool next_segment(const TcParams& P, TcWalk& k, TcSegment& s) {
  while (k.w < k.w1) {
    while (k.w >= k.base + k.count()) {
      k.base += k.count();
      walk_to(P, k, k.b + 1);
    }
    const int at = k.w - k.base, item = (int)quotient(at, k.T), item0 = k.base + item * k.T;
    int from = k.w - item0, to = min(k.T, k.w1 - item0);
    if (k.T <= kLead + (P.p.a.B == 1 ? kWholeOne : kWhole)) {
      const bool mine = 2 * from < k.T;  // from > 0 only at the share's start
      from = 0, to = mine && 2 * to >= k.T ? k.T : 0;
    }
    k.w = min(k.w1, item0 + k.T);
    if (to <= kLead) continue;  // none of the item's tiles
    s.b = k.b, s.h = k.blocks == 1 ? item : (int)quotient(item, k.blocks), s.rb = item - s.h * k.blocks;
    s.T = k.T, s.tp = k.tp, s.X = k.X;
    s.t0 = max(0, from - kLead);
    s.t1 = to - kLead;
    s.item0 = item0;
    return true;
  }
  return false;
}

// The CTA whose share holds unit x of the list: the last whose start,
// floor(total c / ctas), is not past x.
static __device__ __noinline__ int share_of(int x, int total, int ctas) {
  int c = min(ctas - 1, (int)__fdividef((float)x * (float)ctas, (float)total));
  while (c + 1 < ctas && mul_div(total, c + 1, ctas) <= x) ++c;
  while (c > 0 && mul_div(total, c, ctas) > x) --c;
  return c;
}

// A CTA's place in the list of lots.
struct TcWalker {
  int w, w1, at, count, whole;
  TcLot lot;
};

__device__ __forceinline__ TcLot load_lot(const TcLot* l) {
  const int4* p = reinterpret_cast<const int4*>(l);
  const int4 x = __ldcg(p), y = __ldcg(p + 1), z = __ldcg(p + 2);
  return TcLot{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
}

// next_segment over the list, by a whole warp, into shared memory.
template <int kMode>
static __device__ __noinline__ bool next_place(const TcParams& P, TcWalker& k, TcPlace* to) {
  const int lane = threadIdx.x & 31;
  TcSegment s = {};
  while (k.w < k.w1) {
    while (k.w >= k.lot.cum + k.lot.units) {
      if (k.at + 1 >= k.count) {
        k.w = k.w1;
        break;
      }
      k.lot = load_lot(P.list.lots + ++k.at);
    }
    if (k.w >= k.w1) break;
    const int at = k.w - k.lot.cum;
    int item = (int)quotient(at, k.lot.T), item0 = k.lot.cum + item * k.lot.T, T = k.lot.T, lo = 0;
    if ((kMode & kForms) && P.list.ranges && k.lot.blocks > 1) {  // the row block within the head
      const int* cum = P.list.ranges + (int64_t)k.lot.b * P.list.words;
      const int in = at - item * T;
      int rb = 0;
      for (int r0 = 0; r0 < k.lot.blocks; r0 += 32)
        rb += __popc(__ballot_sync(0xFFFFFFFFu, r0 + lane < k.lot.blocks && __ldcg(cum + min(r0 + lane, k.lot.blocks)) <= in));
      --rb;
      item0 += cum[rb], T = cum[rb + 1] - cum[rb], item = item * k.lot.blocks + rb;
      lo = cum[(P.list.words + 1) / 2 + rb];
    }
    int from = k.w - item0, upto = min(T, k.w1 - item0);
    if (T <= k.whole) {
      const bool mine = 2 * from < T;  // from > 0 only at the share's start
      from = 0, upto = mine && 2 * upto >= T ? T : 0;
    }
    k.w = min(k.w1, item0 + T);
    if (upto <= P.list.lead) continue;  // none of the item's tiles
    s.b = k.lot.b, s.h = k.lot.blocks == 1 ? item : (int)quotient(item, k.lot.blocks), s.rb = item - s.h * k.lot.blocks;
    s.T = T, s.tp = k.lot.tp, s.X = {k.lot.S, k.lot.n};
    s.t0 = max(0, from - P.list.lead), s.t1 = upto - P.list.lead, s.item0 = item0;
    s.begin = k.lot.begin, s.m = k.lot.m, s.nb = k.lot.nb, s.lo = lo, s.rev = P.down ? s.t0 + s.t1 - 1 : -1;
    break;
  }
  if (lane == 0) to->seg = s, to->found = 0;
  if (lane < 8) to->spoiled[lane] = 0;
  if ((kMode & kShare) && s.m > 0) {
    Extent E = {0, -1};
    if (lane < s.m) E = extent_of(P.p.a, s.b + lane, nullptr);
    const int mine = own_boxes(P.p.a, P.box, P.box_shift, s.X.S, E);
    int x = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    to->mem.start[lane] = x - mine, to->mem.S[lane] = E.S, to->mem.n[lane] = E.n;
    if (lane == 31) to->mem.start[kMembers] = x;
  }
  return s.T > 0;
}

// What a tile holds: `valid` keys, and u0, the entry number of its first key
// (negative: cached positions before entry 0).  prefix: cached positions only,
// all of them seen (but for a window).  own: boxes of the requests of a group, x0
// the first of them.
struct TcTile {
  bool staged, prefix, own;
  int x0, valid, u0;
};

// The tile that a segment's t-th one is.
template <int kMode>
__device__ __forceinline__ int place_of(const TcSegment& s, int t) {
  return kMode & kForms ? (s.rev >= 0 ? s.rev - t : t) + s.lo : t;
}
template <int kMode>
__device__ __forceinline__ TcTile tile_of(const TcParams& P, const TcSegment& s, int t) {
  const sv_attention_args& a = P.p.a;
  TcTile k;
  t = place_of<kMode>(s, t);
  k.own = (kMode & kShare) && s.m > 0 && t >= s.tp;
  if ((kMode & kShare) && s.m > 0) {
    k.staged = false, k.prefix = !k.own;
    k.x0 = k.own ? (t - s.tp) << (7 - P.box_shift) : t * kTile;
    k.valid = k.own ? min(kTile >> P.box_shift, s.nb - k.x0) << P.box_shift : min(kTile, s.X.S - k.x0);
    k.u0 = 0;
    return k;
  }
  k.staged = a.stage.data && t >= s.tp;
  k.x0 = k.staged ? (t - s.tp) * kTile : (kMode & kForms ? s.begin : 0) + t * kTile;
  const int limit = k.staged ? s.X.n + 1 : a.stage.data ? s.X.S : s.X.S + s.X.n + 1;
  k.valid = min(kTile, limit - k.x0);
  k.u0 = k.staged ? k.x0 : k.x0 - s.X.S;
  k.prefix = !k.staged && (a.stage.data || k.x0 + k.valid <= s.X.S);
  return k;
}

// Whose row a row of an item is: the request (the j-th of its lot), the entry and the
// query head.
struct TcRow {
  int j, b, i, hq;
};
template <int kMode>
__device__ __forceinline__ TcRow row_of(const TcParams& P, const TcSegment& s, int row) {
  const int e = entry_of(P, row), hq = s.h * P.group + row - e * P.group;
  if (!(kMode & kShare) || s.m <= 1) return {0, s.b, e, hq};
  const int j = min(P.entries_magic ? (int)__umulhi((uint32_t)e, P.entries_magic) : e, s.m - 1);  // e < 256
  return {j, s.b + j, e - j * P.p.a.R, hq};
}

// A tile's keys as a row finds them, key numbers counted from the tile's first: it sees the
// cached positions c0 .. c1 - 1, and what the mask says of the entries, entry 0 being key
// e0; org is the key at position S, which the cached positions lead up to.
struct TcView {
  int c0, c1, e0, org;
};
template <int kMode>
__device__ __forceinline__ TcView view_of(const TcParams& P, const TcSegment& s, const TcMembers* mem, const TcTile& k, int j, bool live) {
  constexpr int kFar = 1 << 29;
  const bool staged = P.p.a.stage.data != nullptr;
  TcView v;
  if (!(kMode & kShare) || !k.own) {
    v.org = (kMode & kShare) && s.m > 0 ? mem->S[j] - k.x0 : -k.u0;
    v.c0 = 0, v.c1 = k.prefix ? k.valid : v.org;
    v.e0 = k.prefix || !live ? kFar : v.org;  // (staged entries' tiles have no cached positions: org <= 0)
    return v;
  }
  const Extent E = {mem->S[j], mem->n[j]};
  v.c0 = (mem->start[j] - k.x0) << P.box_shift;
  v.org = v.c0 + E.S - s.X.S;
  v.c1 = live ? v.org : v.c0;
  v.e0 = !live ? kFar : staged ? v.c0 + (cached_boxes(P.p.a, P.box, P.box_shift, s.X.S, E) << P.box_shift) : v.org;
  return v;
}

// What row i of request b's mask (n + 1 entries) says of keys 32 w .. 32 w + 31 of a tile
// whose key e0 is entry 0, in seen[w], by five loads that wait for nothing.
__device__ __forceinline__ void entries_seen(const sv_attention_args& a, int b, int i, int n, int e0, uint32_t (&seen)[4]) {
  const int first = -e0 >> 5, shift = -e0 & 31;
  uint32_t w[5];
#pragma unroll
  for (int x = 0; x < 5; ++x) {
    const int at = first + x, left = n - 32 * at;
    w[x] = 0u;
    if (at < 0 || left < 0) continue;
    w[x] = a.mask ? __ldg(a.mask + ((int64_t)b * a.R + i) * a.mask_ld + at) : i - 32 * at >= 31 ? 0xFFFFFFFFu : i < 32 * at ? 0u : (2u << (i - 32 * at)) - 1u;
    if (left < 31) w[x] &= (2u << left) - 1u;
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) seen[x] = __funnelshift_r(w[x], w[x + 1], shift);
}
__device__ __forceinline__ uint32_t cached_seen(const TcView& v, int ch) {
  const int lo = max(0, v.c0 - 32 * ch), hi = min(32, v.c1 - 32 * ch);
  return hi <= lo ? 0u : (hi >= 32 ? 0xFFFFFFFFu : (1u << hi) - 1u) & 0xFFFFFFFFu << lo;
}

// Whose box a box of own keys is: start[j] <= box < start[j + 1].
__device__ __forceinline__ int member_of(const TcMembers& mem, int box) {
  int lo = 0, hi = kMembers;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (mem.start[mid] <= box) lo = mid; else hi = mid;
  }
  return lo;
}

// The place past its request's S of key `x` of a tile that is no prefix's (negative:
// cached positions).
template <int kMode>
__device__ __forceinline__ int key_place(const TcParams& P, const TcPlace& s, const TcTile& k, int x) {
  const sv_attention_args& a = P.p.a;
  int b = s.seg.b, u = k.u0 + x, n = s.seg.X.n;
  if ((kMode & kShare) && k.own) {
    const int box = k.x0 + (x >> P.box_shift), lo = member_of(s.mem, box);
    const Extent E = {s.mem.S[lo], s.mem.n[lo]};
    const int in = box - s.mem.start[lo], cached = cached_boxes(a, P.box, P.box_shift, s.seg.X.S, E);
    b += lo, n = E.n, u = (in >= cached ? (in - cached) << P.box_shift : s.seg.X.S + (in << P.box_shift) - E.S) + (x & (P.box - 1));
  }
  return u < 0 || u > n ? u : depth_of(a, b, u);
}

// Rows of V in a tile, [r0, r1), that some row of the item may not see though another
// does, or that are next to such: entries, other requests' own keys, and with a window
// the positions that the deepest row no longer sees.
template <int kMode>
__device__ __forceinline__ void half_seen(const sv_attention_args& a, const TcTile& k, const TcSegment& s, int* r0, int* r1) {
  const bool tree = kMode ? !k.prefix : k.valid > -k.u0 && !(a.stage.data && !k.staged);
  *r0 = tree ? max(0, -k.u0) : k.valid;
  *r1 = k.valid;
  if ((kMode & kForms) && a.window > 0 && !k.staged) {
    const int last = (int)min((int64_t)k.valid, (int64_t)s.X.S + a.R - a.window - k.x0);
    if (last > 0) *r0 = 0, *r1 = tree ? k.valid : last;
  }
}

// Waits are bounded (1 s): one that runs out reports SV_ERR_TIMEOUT and turns
// every later wait, load and product of the CTA off, so that all roles run to
// their ends.
struct TcSync {
  volatile int* abort;
  int* err;
};

static __device__ __noinline__ void wait_long(volatile int* abort, int* err, uint32_t bar, uint32_t parity) {
  const uint64_t began = global_ns();
  for (int i = 1; !mbar_try_wait(bar, parity); ++i) {
    if (i % 64) continue;
    if (*abort) return;
    if (global_ns() - began > 1000000000ull) {
      *abort = 1;
      report(err, SV_ERR_TIMEOUT);
      return;
    }
  }
}

__device__ __forceinline__ void wait(const TcSync& s, uint32_t bar, uint32_t parity) {
  if (!mbar_try_wait(bar, parity)) wait_long(s.abort, s.err, bar, parity);
}
// The same; live becomes false in a lane that finds that a wait has run out.
__device__ __forceinline__ void wait(const TcSync& s, uint32_t bar, uint32_t parity, bool& live) {
  if (mbar_try_wait(bar, parity)) return;
  wait_long(s.abort, s.err, bar, parity);
  if (*s.abort) live = false;
}

// Two fp32 values in one register pair, one instruction for both.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Two fp16 values without their upper bytes' shares.
__device__ __forceinline__ uint32_t less_top(uint32_t v) {
  const uint32_t t = v & 0xFF00FF00u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&t));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Each row's softmax keeps a reference m of its scores (log2 units, a whole number,
// so that rescaling is exact), which moves rarely.  Over bf16 caches it moves when
// a score exceeds it by more than kSlack, and the outputs in tensor memory with it;
// weights are 2^kSlack at most and have fp32's range.  Their 8 bits are what a bf16
// product takes: V is bf16, and both operands of a product have one type.
constexpr float kSlack = 8.0f;

// Over 8-bit caches a weight is p times its key's V scale, so that V's codes are
// multiplied as they are, and weights have a reference of their own, the largest
// such product so far: V's scales may differ by any factor, and the sum of p must
// not depend on them.  (One reference for both lost every other key where a row
// that weighs much has a scale far above theirs, and the sum overflowed where the
// first scales were below 2^-112.)  m then moves when 32 p add up to more than
// kMostSum, so that one maximum is taken per score, the products'.
//
// A weight starts as fp16, in 2^(kBias - 1) .. 2^kBias for the largest when its
// reference is set and kMost at most, and is split in three: the upper byte of an
// fp16 value is an 8-bit value of 5 exponent and 2 fraction bits, and so are the
// upper bytes of what is left after the first and the second.  Their smallest step
// is 2^-16: three products of 8 bits weigh V with 9 bits down to 2^-18 of a row's
// largest weight, 5 bits at 2^-22, and are off by 2^-27 of it at most (2^-24 after
// weights were rescaled, below).  (The format of V's codes, split in two, flushes
// weights 2^-18 below the largest, and most of a long sequence's mass may lie there.)
// kMost is the largest fp16 value: a limit of 2^15 moved a reference once or twice
// more per warp and item, and a group weighed twice holds a stream up by 1500 cycles
// (64 trees of 15 nodes, scales of 2^-8 to 2^-6: 203 us; 191 as it is).
constexpr float kBias = 11.0f, kMost = 65504.0f;
constexpr float kMostSum = 0x1p7f;   // with scales of 2^120 at most, products stay finite
// log2 of what a product is multiplied by at most to become a weight: where a row's
// largest is below 2^-115, weights lose bits rather than the factor its range.
constexpr float kMaxRaise = 126.0f;

// The whole number above log2(x), -126 for zero and subnormal numbers.
__device__ __forceinline__ float above_log2(float x) { return (float)((int)(__float_as_uint(x) >> 23) - 126); }

// Adds to eight columns of a row from `col` on, fp32 of a partial result or bf16 outputs, what non-finite
// values of V that were cleared from a segment's tiles make of them: infinities or NaN.  With a list
// the tiles that had some are noted, and a row looks through its own request's keys alone.
template <bool F8, int kMode>
static __device__ __noinline__ void give_back(const TcParams& P, const TcSegment& seg, const TcPlace* place, const TcRow& row, int col,
                                              float* part, __nv_bfloat16* out) {
  const sv_attention_args& a = P.p.a;
  const TcMembers* mem = kMode ? &place->mem : nullptr;
  const bool shared = (kMode & kShare) && seg.m > 0;
  const int n = shared ? mem->n[row.j] : seg.X.n, S = shared ? mem->S[row.j] : seg.X.S;
  float sum[8] = {};
#pragma unroll 1
  for (int t = seg.t0; t < seg.t1; ++t) {
    if (kMode) {
      const int bit = spoiled_bit(seg, t);
      if (!(const_cast<const volatile uint32_t*>(place->spoiled)[bit >> 5] >> (bit & 31) & 1)) continue;
    }
    const TcTile k = tile_of<kMode>(P, seg, t);
    int r0, r1;
    half_seen<kMode>(a, k, seg, &r0, &r1);
    const TcView v = kMode ? view_of<kMode>(P, seg, mem, k, row.j, true) : TcView{0, 0, -k.u0, -k.u0};
#pragma unroll 1
    for (int entries = 0; entries < 2; ++entries) {  // cached positions, then entries
      const int end = min(r1, entries ? v.e0 + n + 1 : v.c1);
#pragma unroll 1
      for (int r = max(r0, entries ? v.e0 : v.c0); r < end; ++r) {
        const int u = entries ? r - v.e0 : r - v.org;  // past S
        if (entries && !(seen_bits(a, row.b, row.i, n, u) & 1)) continue;
        if (kMode && a.window > 0 && abs(depth_of(a, row.b, row.i) - (entries ? depth_of(a, row.b, u) : u)) >= a.window) continue;
        const bool staged = entries && a.stage.data;
        const sv_kv_place& pl = staged ? a.stage : a.cache;
        const int at = staged ? u : S + u;  // entry, or position
        const int64_t off = entry_offset(pl, row.b, at, at);
        if (off < 0) continue;
        const char* vr = static_cast<const char*>(pl.data) + off + (a.cache.heads + seg.h) * row_step(pl) + col * (F8 ? 1 : 2);
        uint32_t w[4];
        if (F8) {
          const uint2 y = *reinterpret_cast<const uint2*>(vr);
          w[0] = y.x, w[1] = y.x >> 16, w[2] = y.y, w[3] = y.y >> 16;
        } else {
          const uint4 y = *reinterpret_cast<const uint4*>(vr);
          w[0] = y.x, w[1] = y.y, w[2] = y.z, w[3] = y.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 z = F8 ? e4m3x2_values(w[e] & 0xFFFFu) : make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
          if (!(fabsf(z.x) < __builtin_huge_valf())) sum[2 * e] += z.x;
          if (!(fabsf(z.y) < __builtin_huge_valf())) sum[2 * e + 1] += z.y;
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (part)
      part[e] += sum[e];
    else
      out[e] = __float2bfloat16_rn(__bfloat162float(out[e]) + sum[e]);
  }
}

// The rare steps of a tile's softmax, as calls so that they stay out of the
// loop's instructions.
//
// Scores that row i does not see become -inf where they are.
static __device__ __noinline__ void hide_unseen(const TcParams& P, int b, int i, int n, bool prefix, int valid, int u0, int ch_a,
                                                int ch_e, uint32_t tS) {
  for (int ch = ch_a; ch < ch_e; ++ch) {
    const int left = valid - 32 * ch;
    const uint32_t bits = prefix ? (left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1u)
                          : i <= n ? seen_bits(P.p.a, b, i, n, u0 + 32 * ch)
                                   : 0u;
    uint32_t x[32];
    tmem_ld32(tS + 32 * ch, x);
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = bits >> e & 1 ? x[e] : 0xFF800000u;
    tmem_st32(tS + 32 * ch, x);
  }
  tmem_wait_st();
}

// What a row's scores get from their form.
struct TcForm {
  float factor, cap, slope;  // of the products (see form_factor; 0: steps other than kDirect); log2 units
  int at;                    // the row's position
};

// Scores become what the softmax takes, in log2 units: products times c (and K's scales),
// capped, less slope times the distance.
//   cap tanh(s / cap) = cap - 2 cap / (1 + 2^(2 s log2(e) / cap)),
// off by 3 x 2^-24 of the cap: 2^-14 of a weight up to the cap kCapNear (in log2 units).  Past
// it scores below 0.3 cap take the series of tanh to the ninth power, whose next term is 5e-8
// of it.  (The series for all scores that allow it, chosen for 32 keys of 32 rows at once: 64 trees
// capped at 50 220 us, 215 without a choice; chosen by each score 249.)  No score's form depends on
// other scores, and the functions below round alike, so that a row's result does not
// depend on which of them the other rows of its warp need.
constexpr float kCapNear = 512.0f;

// A product of codes is multiplied by the row's factor (c, or what makes the argument of a cap's
// exponential of it) before its key's scale: queries of 2^-119 and keys of 2^117 are ordinary scores,
// and 2^19, such a product, times 2^111, such a key's scale, is no fp32 value.  In factor_within neither step
// leaves fp32's range where the score does not (codes' products are 2^-18 to 2^25, or 0); for
// other factors the score is made first, of what keeps it in range, and the cap's factor is multiplied by
// after (the smallest cap's is 2^61).
constexpr float kMostFactor = 0x1p100f;
__device__ __forceinline__ bool factor_within(float f) { return f >= 0x1p-100f && f <= kMostFactor; }
// How scores are made: kDirect as shape_near does; kLarge for caps past kCapNear; kCareful where a
// row's factor is outside factor_within.
constexpr int kDirect = 0, kLarge = 1, kCareful = 2;
__device__ __forceinline__ float form_factor(float c, float cap) { return cap > 0.0f ? 2.0f * kLog2e * (c / cap) : c; }

// Those of 32 keys where they are, key e at the distance far - e, or where `apart` as the
// keys' places past S say, a lane each; -inf where `bits` are clear.  The softmax's loop has
// shape_near for keys in a row, as nearly all are.  This is for the others, and for those
// that a moved reference needs once more.
// In a pass of its own for all scores, over tensor memory and by arguments in memory, it was 3000
// cycles a group of 32 keys, mostly waits for instructions and arguments (64
// single tokens under a window of 1024, capped: 83 us).
template <bool F8, int kSteps>
static __device__ __noinline__ void shape_chunk(uint32_t tS, float c, const float* ks, float cap, float slope, int far, bool apart, int place,
                                                uint32_t bits) {
  const float f = form_factor(c, cap), inv = 1.0f / cap;
  const bool near = kSteps == kDirect || (kSteps == kCareful && cap <= kCapNear), direct = kSteps == kDirect || (near && factor_within(f));
  // a score is product * first * K's scale * last
  const float first = kSteps == kCareful && c > kMostFactor ? 1.0f : c, last = kSteps == kCareful && c > kMostFactor ? c : 1.0f;
  const float up = direct ? 1.0f : 2.0f * kLog2e;  // from y to an exponential's argument
#pragma unroll 1
  for (int g = 0; g < 32; g += 8) {
    uint32_t x[8];
    float y[8], most = 0.0f;  // the exponentials' arguments, or scores / cap
    tmem_ld8(tS + g, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = __uint_as_float(x[e]), k = F8 ? ks[g + e] : 1.0f;
      float z = __fmul_rn(__fmul_rn(s, kSteps == kDirect ? f : first), k);
      if (kSteps == kCareful) z = __fmul_rn(z, last);
      y[e] = direct ? __fmul_rn(__fmul_rn(s, f), k) : __fmul_rn(z, inv);
      if (!near) {
        const float w = y[e], w2 = __fmul_rn(w, w);
        const float t = __fmaf_rn(w2, __fmaf_rn(w2, __fmaf_rn(w2, 62.0f / 2835.0f, -17.0f / 315.0f), 2.0f / 15.0f), -1.0f / 3.0f);
        most = fmaxf(most, fabsf(w));
        z = __fmul_rn(z, __fmaf_rn(w2, t, 1.0f));
      }
      x[e] = __float_as_uint(z);
    }
    if (cap > 0.0f && (near || __any_sync(0xFFFFFFFFu, most > 0.3f))) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float large = __fmaf_rn(rcp(__fadd_rn(ex2(kSteps == kDirect ? y[e] : __fmul_rn(y[e], up)), 1.0f)), -2.0f * cap, cap);
        x[e] = near || fabsf(y[e]) > 0.3f ? __float_as_uint(large) : x[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = apart ? (float)abs(far - __shfl_sync(0xFFFFFFFFu, place, g + e)) : (float)far - (float)(g + e);
      const float z = slope == 0.0f ? __uint_as_float(x[e]) : __fmaf_rn(-slope, d, __uint_as_float(x[e]));
      x[e] = bits >> (g + e) & 1 ? __float_as_uint(z) : 0xFF800000u;
    }
    tmem_st8(tS + g, x);
  }
  tmem_wait_st();
}

// Calls of their own: as one function for all steps, the callers keep less in registers (64 8-bit
// trees with slopes 277 us, 254 so).  Caps past kCapNear have only this: the 64 trees capped at 400
// 345 us and 392 in 8 bits, at 50 202 and 272.
template <bool F8>
__device__ __forceinline__ void shape_group(bool direct, uint32_t tS, float c, const float* ks, float cap, float slope, int far, bool apart, int place,
                                            uint32_t bits) {
  if (direct)
    shape_chunk<F8, kDirect>(tS, c, ks, cap, slope, far, apart, place, bits);
  else if (cap > kCapNear && __all_sync(0xFFFFFFFFu, factor_within(c)))
    shape_chunk<F8, kLarge>(tS, c, ks, cap, slope, far, apart, place, bits);
  else
    shape_chunk<F8, kCareful>(tS, c, ks, cap, slope, far, apart, place, bits);
}

// Those of 32 keys in a row, in registers; false: they are shape_chunk's (a cap past kCapNear, factors
// outside factor_within), and x is as it was.
template <bool F8>
__device__ __forceinline__ bool shape_near(uint32_t (&x)[32], const float* ks, const TcForm& f, int far) {
  if (f.factor == 0.0f) return false;
  uint64_t v[16];
  const uint64_t f2 = pair(f.factor, f.factor);
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    v[e] = mul2(pair(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), f2);
    v[e + 1] = mul2(pair(__uint_as_float(x[2 * e + 2]), __uint_as_float(x[2 * e + 3])), f2);
    if (F8) {
      const ulonglong2 s2 = *reinterpret_cast<const ulonglong2*>(ks + 2 * e);
      v[e] = mul2(v[e], s2.x), v[e + 1] = mul2(v[e + 1], s2.y);
    }
  }
  if (f.cap > 0.0f) {
    const uint64_t cap2 = pair(f.cap, f.cap), down2 = pair(-2.0f * f.cap, -2.0f * f.cap);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 z = unpair(v[e]);
      const float2 w = unpair(add2(pair(ex2(z.x), ex2(z.y)), pair(1.0f, 1.0f)));
      v[e] = fma2(pair(rcp(w.x), rcp(w.y)), down2, cap2);
    }
  }
  if (f.slope != 0.0f) {
    const float d = (float)far;
    const uint64_t slope2 = pair(-f.slope, -f.slope), d2 = pair(d, d);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = fma2(slope2, add2(d2, pair((float)(-2 * e), (float)(-2 * e - 1))), v[e]);
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 y = unpair(v[e]);
    x[2 * e] = __float_as_uint(y.x), x[2 * e + 1] = __float_as_uint(y.y);
  }
  return true;
}

// The references (m, weights') of the rows that need others for 32 scores: a whole
// number at or above the largest score, and above the largest product of p and V's
// scale, or what kMaxRaise leaves.  Both stay -inf for a row that sees nothing.
// With forms (small windows) a row may see one key alone, and the first reference is its score
// to 2^-16, so that its weight is stored as a power of two and the output is its V: by a whole
// number one output of 12000 was off by its last bit.  Later ones are whole numbers above that.
template <bool kNear>
static __device__ __noinline__ float2 references(uint32_t tS, float c, const float* kp, const float* sc, float m, float wr, bool need) {
  uint32_t x[32];
  tmem_ld32(tS, x);
  if (!need) return make_float2(m, wr);
  float mx = m, top[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 ks = *reinterpret_cast<const float4*>(kp + e);
    const float s[4] = {__uint_as_float(x[e]) * c * ks.x, __uint_as_float(x[e + 1]) * c * ks.y, __uint_as_float(x[e + 2]) * c * ks.z,
                        __uint_as_float(x[e + 3]) * c * ks.w};
#pragma unroll
    for (int z = 0; z < 4; ++z) x[e + z] = __float_as_uint(s[z]);
    mx = fmaxf(fmaxf(mx, fmaxf(s[0], s[1])), fmaxf(s[2], s[3]));
  }
  if (!kNear)
    mx = ceilf(mx);
  else if (m != -__builtin_huge_valf())
    mx = m + ceilf(mx - m);
  else
    mx = fabsf(mx) < 128.0f ? ceilf(mx * 0x1p16f) * 0x1p-16f : ceilf(mx);
  if (mx == -__builtin_huge_valf()) return make_float2(m, wr);
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 vs = *reinterpret_cast<const float4*>(sc + kTile + e);
    const float v[4] = {vs.x, vs.y, vs.z, vs.w};
#pragma unroll
    for (int z = 0; z < 4; ++z) top[z] = fmaxf(top[z], ex2(__uint_as_float(x[e + z]) - mx) * v[z]);
  }
  const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  return make_float2(mx, fmaxf(fmaxf(wr, mx + above_log2(most)), mx + kBias - kMaxRaise));
}

// Outputs times each row's f.
static __device__ __noinline__ void rescale(uint32_t tO, int cols, float f) {
  for (int col = 0; col < cols; col += 16) {
    uint32_t o[16];
    tmem_ld16(tO + col, o);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
    tmem_st16(tO + col, o);
  }
}

// Weights times each row's f, a power of two: exact but for what the three 8-bit
// parts lose below 2^-16 each, 3 x 2^-26 of a row's largest weight.
template <bool F8>
static __device__ __noinline__ void rescale_weights(uint32_t tW, int cols, float f) {
  tmem_wait_st();
  for (int col = 0; col < cols; col += 8) {
    uint32_t w[8];
    tmem_ld8(tW + col, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (F8) {
        const __half2 f2 = __float2half2_rn(f);
        uint32_t even = w[e] << 8 & 0xFF00FF00u, odd = w[e] & 0xFF00FF00u;
        const __half2 a = __hmul2(*reinterpret_cast<const __half2*>(&even), f2), b = __hmul2(*reinterpret_cast<const __half2*>(&odd), f2);
        even = *reinterpret_cast<const uint32_t*>(&a), odd = *reinterpret_cast<const uint32_t*>(&b);
        w[e] = (even >> 8 & 0x00FF00FFu) | (odd & 0xFF00FF00u);
      } else {
        w[e] = pack_bf16(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xFFFF0000u) * f);
      }
    }
    tmem_st8(tW + col, w);
  }
}

// Rows r0 .. valid - 1 of a V tile without their non-finite values (*found is
// set where there was one), rows valid .. r1 - 1 cleared; thread of 128.
template <bool F8>
static __device__ __noinline__ void clean_rows_plain(char* v, int r0, int valid, int r1, int row_vecs, int thread, volatile int* found) {
  const int sw = row_vecs < 8 ? row_vecs : 8;  // vectors of a row per half
  for (int x = thread; x < (r1 - r0) * row_vecs; x += 128) {
    const int r = r0 + x / row_vecs, c = x % row_vecs;
    uint4* d = reinterpret_cast<uint4*>(v + (c / sw * kTile + r) * sw * 16 + c % sw * 16);
    if (r >= valid) {
      *d = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 y = *d;
    constexpr uint32_t kMax = F8 ? 0x7F7F7F7Fu : 0x7F807F80u;
    auto bad = [&](uint32_t z) { return F8 ? __vcmpeq4(z & kMax, kMax) : __vcmpeq2(z & kMax, kMax); };
    const uint32_t bx = bad(y.x), by = bad(y.y), bz = bad(y.z), bw = bad(y.w);
    if (bx | by | bz | bw) {
      y.x &= ~bx, y.y &= ~by, y.z &= ~bz, y.w &= ~bw;
      *d = y;
      *found = 1;
    }
  }
  fence_async_smem();
}

// The rows of a tile of own keys (x0: its first box) that hold none as zeros, by a whole warp: places past a
// request's last position or entry in its last boxes.  What was never written is no value of V, and must not
// look like one that has to be given back.  (Done where a tile has non-finite values at all: for every
// tile it kept the warp, for which the products wait, and shared chains took 91 us for 76.)
template <int kVecs>
static __device__ __noinline__ void clear_unheld(const TcParams& P, const TcPlace& s, int x0, int valid, char* v) {
  constexpr int kSw = kVecs < 8 ? kVecs : 8;  // vectors of a row per half
  const sv_attention_args& a = P.p.a;
  const int lane = threadIdx.x & 31, at = lane << P.box_shift;
  uint32_t held = 0;  // of a lane's box
  if (at < valid) {
    const int j = member_of(s.mem, x0 + lane), in = x0 + lane - s.mem.start[j];
    const Extent E = {s.mem.S[j], s.mem.n[j]};
    const int cached = cached_boxes(a, P.box, P.box_shift, s.seg.X.S, E);
    const int keys = in >= cached ? E.n + 1 - ((in - cached) << P.box_shift)
                                  : max(0, E.S - s.seg.X.S) + (a.stage.data ? 0 : E.n + 1) - (in << P.box_shift);
    held = (1u << min(keys, P.box)) - 1u;
  }
  bool any = false;
#pragma unroll 1
  for (int w = 0; 32 * w < valid; ++w) {
    const uint32_t all = valid - 32 * w >= 32 ? 0xFFFFFFFFu : (1u << (valid - 32 * w)) - 1u;
    uint32_t left = all & ~__reduce_or_sync(0xFFFFFFFFu, at >> 5 == w ? held << (at & 31) : 0u);
    any |= left != 0;
    for (; left; left &= left - 1) {
      const int r = 32 * w + __ffs(left) - 1;
      if (lane < kVecs) *reinterpret_cast<uint4*>(v + (lane / kSw * kTile + r) * kSw * 16 + lane % kSw * 16) = make_uint4(0, 0, 0, 0);
    }
  }
  if (any) fence_async_smem();
  __syncwarp();
}

// Whether a lane's share of rows r0 .. valid - 1 of a V tile has non-finite values.
template <bool F8, int kVecs>
__device__ __forceinline__ bool spoiled_rows(const char* v, int r0, int valid) {
  constexpr int kSw = kVecs < 8 ? kVecs : 8;  // vectors of a row per half
  // 0 times a value is NaN for bf16, an 8-bit NaN's low seven bits are ones (with the comparisons
  // below for every vector, by 128 threads: 4700 cycles a tile, 2300 of 8 bits)
  uint32_t any[4] = {0, 0, 0, 0};
#pragma unroll 8
  for (int x = threadIdx.x & 31; x < (valid - r0) * kVecs; x += 32) {
    const int r = r0 + x / kVecs, c = x % kVecs;
    const uint4 y = *reinterpret_cast<const uint4*>(v + (c / kSw * kTile + r) * kSw * 16 + c % kSw * 16);
    if (F8) {
      any[0] |= ((y.x & 0x7F7F7F7Fu) + 0x01010101u) | ((y.y & 0x7F7F7F7Fu) + 0x01010101u);
      any[1] |= ((y.z & 0x7F7F7F7Fu) + 0x01010101u) | ((y.w & 0x7F7F7F7Fu) + 0x01010101u);
    } else {
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(any[e]) : "r"(w[e]), "r"(0u));
    }
  }
  return ((any[0] | any[1] | any[2] | any[3]) & (F8 ? 0x80808080u : 0x7FFF7FFFu)) != 0;
}

// As clean_rows_plain where most tiles are looked at, by a warp that the softmax does not wait for: tile t of
// a segment.  kVecs: vectors of 16 bytes of a row.
template <bool F8, int kMode, int kVecs>
static __device__ __noinline__ void clean_rows(const TcParams& P, TcPlace* s, int t, bool own, int x0, char* v, int r0, int valid, int r1) {
  constexpr int kSw = kVecs < 8 ? kVecs : 8;
  const int lane = threadIdx.x & 31;
  auto at = [&](int x) {
    const int r = r0 + x / kVecs, c = x % kVecs;
    return reinterpret_cast<uint4*>(v + (c / kSw * kTile + r) * kSw * 16 + c % kSw * 16);
  };
  bool dirty;
#pragma unroll 1
  for (bool again = false;; again = true) {
    dirty = spoiled_rows<F8, kVecs>(v, r0, valid);
    if (!(kMode & kShare) || !own || again || !__any_sync(0xFFFFFFFFu, dirty)) break;
    clear_unheld<kVecs>(P, *s, x0, valid, v);
  }
  for (int x = lane; x < (r1 - valid) * kVecs; x += 32) *at((valid - r0) * kVecs + x) = make_uint4(0, 0, 0, 0);
  if (dirty)
#pragma unroll 1
    for (int x = lane; x < (valid - r0) * kVecs; x += 32) {
      uint4* d = at(x);
      uint4 y = *d;
      constexpr uint32_t kMax = F8 ? 0x7F7F7F7Fu : 0x7F807F80u;
      auto bad = [&](uint32_t z) { return F8 ? __vcmpeq4(z & kMax, kMax) : __vcmpeq2(z & kMax, kMax); };
      const uint32_t bx = bad(y.x), by = bad(y.y), bz = bad(y.z), bw = bad(y.w);
      if (bx | by | bz | bw) {
        y.x &= ~bx, y.y &= ~by, y.z &= ~bz, y.w &= ~bw;
        *d = y;
        const int bit = spoiled_bit(s->seg, t);
        atomicOr(&s->spoiled[bit >> 5], 1u << (bit & 31));
        *const_cast<volatile int*>(&s->found) = 1;
      }
    }
  if (dirty || r1 > valid) fence_async_smem();
}

// o = sum_x p_x V_x, p = softmax(scale q K^T), in one pass over the keys: scores
// of 128 rows and 128 keys as a product with its result in tensor memory, their
// weights against the running reference maximum back into the same columns, and
// the product of weights and V added to the outputs there; sums and maxima in
// registers, in fp32.  One persistent CTA per SM, since a CTA's products fill its
// tensor memory and its tiles its shared memory; rows are padded to 128 because
// bytes bound all but the widest calls.  64 requests of 128 to 8192 positions, 8 KV
// heads of 128, bf16: single tokens 189 us, trees of 15 nodes (60 rows a head) 199
// (5.8 and 5.6 TB/s); 8-bit 166 and 189 (3.7 and 3.3), where a stream's chain
// bounds it: with trees, a tile's softmax takes 2100 cycles (at 1.94 GHz; 750 per 32
// keys a warp) and waits 1800 for its scores, in which the products' warp issues
// both streams' 8 + 12 products and their commits (1500 a tile).  4 requests of up
// to 65536 positions, 448 rows a head, bf16: 184 us, 0.85 PFLOP/s; what the products'
// warp does between products (waits, commits: a third of its time) bounds that.  Handing scores over in halves
// of 64 keys, to have the next half's under way, doubled those steps: 249 us.
//
// Forms of the scores (kForms): 64 trees over 128 to 8192 positions, capped scores 202 us
// in bf16 as without (bytes bound both), 8-bit with a distance's share 254 (a stream's chain, which
// the form lengthens: per 32 keys some 1000 cycles of loads, factors and the form, 630 of
// weights, 1000 of stores and what is seen); under a window of 1024 single tokens 69 us: nine tiles
// an item are 22000 cycles, and 7500 more its start and end.  Prompts of up to 2041
// entries and as many cached positions under that window 233 us: 256 rows a tile take
// 7000 cycles, more than half of it the softmax of eight warps.
// Shared prefixes (kShare): rows of as many of a group's requests as lot_size has are an item's, which
// reads the prefix once for them, and their own keys are packed behind it.  A first version made
// the prefix's and each request's own parts apart and joined them in another kernel: 256 chains
// of four drafts in groups of four over 1024 shared tokens and up to 31 of their own 219 us, 77 as it is; but 64
// single tokens with 128 to 4096 own positions 157, 130 as it is, as a tile of own keys is weighed by
// one request's warps.
template <bool F8, int D, int QM, int kMode>
__global__ void __launch_bounds__(TcShape<F8, D, QM, kMode>::kThreads, 1) tc_attention_kernel(const __grid_constant__ TcParams P) {
  using C = TcShape<F8, D, QM, kMode>;
  extern __shared__ char smem_raw[];
  const sv_attention_args& a = P.p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.cache.heads, G = P.group;
  constexpr float kInf = __builtin_huge_valf();

  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  char* sm = smem_raw + pad;
  const uint32_t sQ = raw + pad, sK = sQ + C::kQAll, sV = sK + C::kK * C::kKBytes;
  char* kslots = sm + C::kQAll;
  char* vslots = kslots + C::kK * C::kKBytes;
  char* misc = vslots + C::kV * C::kTileBytes;
  const uint32_t bars = smem_u32(misc);
  // K loaded / free, V loaded / free, scores, weights, outputs, queries, scales set / read
  const uint32_t b_kf = bars, b_ke = b_kf + 8 * C::kK, b_vf = b_ke + 8 * C::kK, b_ve = b_vf + 8 * C::kV,
                 b_s = b_ve + 8 * C::kV, b_p = b_s + 16, b_o = b_s + 32, b_q = b_s + 48, b_sf = b_s + 56,
                 b_se = b_sf + 8 * kScaleRing, b_gf = b_se + 8 * kScaleRing, b_ge = b_gf + 8 * kSegments,  // places set / read
                 b_vc = b_ge + 8 * kSegments;                                                          // V without non-finite values
  int* ints = reinterpret_cast<int*>(misc + 512);  // 0 tensor memory, 1 abort, 2 non-finite entries, 3 last, 4.. walk
  float2* s_ml = reinterpret_cast<float2*>(misc + 1024);  // [256] maxima and sums exchanged or joined
  float* s_qs = reinterpret_cast<float*>(misc + 3072);    // [kRows] row scales of 8-bit queries
  float* s_sc = s_qs + C::kRows;                          // [kScaleRing][2][128] scales of a tile's entries, K's and V's
  float* s_wr = s_sc + kScaleRing * 2 * kTile;            // [256] references of 8-bit weights, exchanged
  float* s_ones = s_wr + 2 * kTile;                       // [32] K's scales of scores that have them already
  TcPlace* places = reinterpret_cast<TcPlace*>(misc + C::kMisc) - kSegments;  // [kSegments]
  int* s_at = reinterpret_cast<int*>(places) - 4 * kTile;  // [2][2][128] places of a tile's keys past their S

  if (tid == 0) {
    for (int i = 0; i < C::kK; ++i) mbar_init(b_kf + 8 * i, 1), mbar_init(b_ke + 8 * i, QM);
    for (int i = 0; i < C::kV; ++i) mbar_init(b_vf + 8 * i, 1), mbar_init(b_ve + 8 * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(b_s + 8 * i, 1), mbar_init(b_p + 8 * i, 4), mbar_init(b_o + 8 * i, 1);
    mbar_init(b_q, 8);
    for (int i = 0; i < kScaleRing; ++i) mbar_init(b_sf + 8 * i, 1), mbar_init(b_se + 8 * i, 4 * QM);
    if (kMode)
      for (int i = 0; i < kSegments; ++i) mbar_init(b_gf + 8 * i, 1), mbar_init(b_ge + 8 * i, 11);
    if (kMode)
      for (int i = 0; i < C::kV; ++i) mbar_init(b_vc + 8 * i, 1);
    ints[1] = ints[2] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&P.pages);
    if (a.stage.data) tma_prefetch_map(&P.stage);
  }
  if (warp == 9) tmem_alloc(smem_u32(&ints[0]), 512);
  if (kMode && F8 && warp == 11) s_ones[lane] = 1.0f;
  pdl_wait();
  pdl_trigger();

  // Every CTA counts the tiles of all requests and finds its share: an equal
  // number of consecutive tiles each, so no CTA waits for a longer sequence.
  TcWalk walk;
  walk.qrows = C::kRows;
  int total = 0, ctas, w0 = 0, w1 = 0;
  auto share = [&] {
    ctas = sharing_ctas(a, G, gridDim.x, total);
    if ((int)blockIdx.x < ctas) w0 = mul_div(total, blockIdx.x, ctas), w1 = mul_div(total, blockIdx.x + 1, ctas);
  };
  if (kMode) {  // a kernel before has counted
    total = __ldcg(P.list.head);
    share();  // of as many CTAs as plan_kernel has it
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  } else if (a.B <= 4) {  // every thread counts for itself
#pragma unroll 1
    for (int b = 0; b < a.B; ++b) walk_to(P, walk, b), total += walk.count();
    share();
    walk.base = 0;
    if (w1 > w0 && a.B > 1) {
#pragma unroll 1
      for (int b = 0;; walk.base += walk.count(), ++b) {
        walk_to(P, walk, b);
        if (w0 < walk.base + walk.count()) break;
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  } else {
    const int per = (a.B + C::kThreads - 1) / C::kThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; ++b) walk_to(P, walk, b), mine += walk.count();
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) ints[16 + warp] = x;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < C::kThreads / 32; ++i) {
      if (i < warp) before += ints[16 + i];
      total += ints[16 + i];
    }
    const int first = before + x - mine;  // units of the requests before mine
    share();
    if (w1 > w0 && mine > 0 && first <= w0 && w0 < first + mine) {
      int at = first;
      for (int b = b0; b < b1; ++b) {
        if (per > 1) walk_to(P, walk, b);
        if (w0 < at + walk.count()) {
          ints[4] = b, ints[5] = at, ints[8] = walk.X.S, ints[9] = walk.X.n;
          break;
        }
        at += walk.count();
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    walk.base = 0;
    if (w1 > w0) {
      walk.base = ints[5];
      plan(P, walk, ints[4], Extent{ints[8], ints[9]});
    }
  }
  walk.w = w0, walk.w1 = w1;
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&ints[0]);
  const TcSync sync{ints + 1, P.p.err};
  // `found` is written by a call, so it lives in memory, where asm statements
  // make every use a load; the roles work on a copy in registers
  TcSegment found;
  // With a list, one warp finds the items' places for all: a role takes the next one
  // and gives it back after its last tile.  (A role that finds that a wait has run out
  // ends; the softmax's warps, which meet at barriers, agree on that.)
  int taken = 0;
  auto next = [&](TcSegment& seg) {
    if (!kMode) {
      const bool any = next_segment(P, walk, found);
      seg = found;
      return any;
    }
    wait(sync, b_gf + 8 * (taken % kSegments), taken / kSegments & 1);
    if (__any_sync(0xFFFFFFFFu, *sync.abort)) return false;
    seg = places[taken % kSegments].seg;
    return seg.T > 0;
  };
  auto give_back_place = [&] {
    if (!kMode) return;
    __syncwarp();
    if (lane == 0) mbar_arrive(b_ge + 8 * (taken % kSegments));
    ++taken;
  };

  if (warp >= 8) {
    if (warp == 8 || warp == 10) {
      // ---- loads: K by one warp, V by another ------------------------------
      asm volatile("fence.proxy.async.global;" ::: "memory");  // what earlier kernels wrote, for TMA
      const int v = warp == 10, slots = v ? C::kV : C::kK;
      const uint32_t b_full = v ? b_vf : b_kf, b_empty = v ? b_ve : b_ke, ring = v ? sV : sK;
      constexpr int kElems = F8 ? C::kSw : C::kSw / 2;
      int slot = 0, lap = 0;
      TcSegment seg;
      for (; next(seg); give_back_place()) {
        const TcMembers& mem = places[taken % kSegments].mem;
        if (!v) {  // the segment's queries, on their way into L2 while the last one's tiles are worked on
          const int rows = min(C::kRows, (seg.X.n + 1) * G - seg.rb * C::kRows);
          const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(a.q) + seg.b * a.q_stride[0] + (int64_t)seg.h * G * a.q_stride[2];
#pragma unroll 1
          for (int r = lane; r < rows; r += 32) {
            const int rr = seg.rb * C::kRows + r, qi = entry_of(P, rr);
            const __nv_bfloat16* row = q0 + qi * a.q_stride[1] + (rr - qi * G) * a.q_stride[2];
            if ((kMode & kShare) && seg.m > 1) {
              const TcRow to = row_of<kMode>(P, seg, rr);
              row = static_cast<const __nv_bfloat16*>(a.q) + to.b * a.q_stride[0] + to.i * a.q_stride[1] + to.hq * a.q_stride[2];
            }
            for (int c = 0; c < D; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + c));
          }
        }
#pragma unroll 1
        for (int t = seg.t0; t < seg.t1; ++t) {
          const TcTile k = tile_of<kMode>(P, seg, t);
          const int box = k.staged ? (kMode ? P.stage_box : kStageBox) : P.box, boxes = (k.valid + box - 1) / box;
          // each lane looks up its box's block before the slot is free
          int y = k.x0 + lane * box, w = seg.b;
          bool staged = k.staged;
          if ((kMode & kShare) && k.own && lane < boxes) {  // whose box it is
            const int x = k.x0 + lane, lo = member_of(mem, x);
            const int in = x - mem.start[lo], cached = cached_boxes(a, P.box, P.box_shift, seg.X.S, {mem.S[lo], mem.n[lo]});
            staged = in >= cached;
            w = seg.b + lo, y = staged ? (in - cached) * box : seg.X.S + in * box;
          }
          if (!staged && lane < boxes) {
            const int j = block_of(P, y);
            w = __ldg(a.cache.block_table + (int64_t)w * a.cache.max_blocks + j);
            if (w < 0 || w >= a.cache.num_blocks) {
              report(P.p.err, SV_ERR_STATE);
              w = a.cache.num_blocks;  // past the last: a load gives zeros
            }
            y -= j * a.cache.block_size;
          }
          const int z = ((staged ? a.stage.layer : a.cache.layer) * 2 + v) * H + seg.h;
          const CUtensorMap* map = staged ? &P.stage : &P.pages;
          if (lap > 0) wait(sync, b_empty + 8 * slot, (lap - 1) & 1);
          if (!__any_sync(0xFFFFFFFFu, *sync.abort)) {
            const uint32_t bar = b_full + 8 * slot, at = ring + slot * (v ? C::kTileBytes : C::kKBytes), dst = at + lane * box * C::kSw;
            if (lane == 0) mbar_expect_tx(bar, boxes * box * (F8 && !v ? C::kRow + 2 * kTail : C::kRow));
            __syncwarp();
            if (lane < boxes) {
#pragma unroll
              for (int hf = 0; hf < C::kHalves; ++hf) tma_load_4d(dst + hf * C::kHalfBytes, map, bar, hf * kElems, y, z, w);
              if (F8 && !v)
                tma_load_5d(at + C::kTileBytes + lane * box * 2 * kTail, staged ? &P.stage_tails : &P.page_tails, bar, 0, y, seg.h,
                            (staged ? a.stage.layer : a.cache.layer) * 2, w);
            }
          }
          if (++slot == slots) slot = 0, ++lap;
        }
      }
    } else if (warp == 9) {
      // ---- products --------------------------------------------------------
      // The whole warp runs this and one lane issues, so that descriptors stay
      // in uniform registers; its instructions between products are kept few
      // (the softmax gives K's slots back, tiles' places are counted and not
      // divided for), since they add up with the products' own time.
      const bool one = elect_one();
      int ph_p = 0, ph_q = 0;  // ph_p: a bit per stream
      bool live = true;
      int ks = 0, klap = 0, vs = 0, vlap = 0;
      constexpr uint32_t kIdS = instr_desc(F8 ? 0 : 1, kTile, kTile, false);  // e4m3 or bf16
      constexpr uint32_t kIdO = instr_desc(F8 ? 0 : 1, kTile, D, true) | (F8 ? 1u << 7 : 0u);  // weights of 5 exponent bits
      const uint64_t q0 = smem_desc(sQ, 16, 8 * C::kSw, C::kSw), k0 = smem_desc(sK, 16, 8 * C::kSw, C::kSw);
      const uint64_t v0 = smem_desc(sV, C::kHalfBytes, 8 * C::kSw, C::kSw);
      TcSegment seg;
      for (; next(seg); give_back_place()) {
        const int units = (seg.t1 - seg.t0) * QM;
        const bool apart = a.stage.data || ((kMode & kShare) && seg.m > 0);  // no entries among the cached positions
        const int whole = ((apart ? seg.X.S : seg.X.S + seg.X.n + 1) - (kMode & kForms ? seg.begin : 0)) / kTile;  // tiles before it are full
        wait(sync, b_q, ph_q);
        ph_q ^= 1;
        // scores two units ahead of the outputs
#pragma unroll 1
        for (int x = 0; x < units + 2; ++x) {
          const int st = x & 1;
          const uint32_t tS = tmem + st * 128, tO = tmem + 256 + st * 128;
          bool k_there = QM == 2 && st == 1;
          if (x >= 2) {
            const int t = seg.t0 + (QM == 2 ? (x - 2) >> 1 : x - 2);
            const int steps = place_of<kMode>(seg, t) < whole ? kTile / C::kStep : (tile_of<kMode>(P, seg, t).valid + C::kStep - 1) / C::kStep;
            const uint64_t vd = v0 + vs * (C::kTileBytes >> 4);
            const bool first = x < 4;  // of this stream in this segment
            if (QM == 1 || st == 0) {  // the second row tile's keys are there
              if (kMode) wait(sync, b_vc + 8 * vs, vlap & 1, live);
              wait(sync, b_vf + 8 * vs, vlap & 1, live);
              k_there = x < units && mbar_test_wait(b_kf + 8 * ks, klap & 1);  // while the weights are awaited
            }
            wait(sync, b_p + 8 * st, ph_p >> st & 1, live);
            ph_p ^= 1 << st;
            tc_fence_after();
            if (one && live) {
#pragma unroll
              for (int j = 0; j < kTile / C::kStep; ++j) {
                if (j >= steps) break;
                const uint64_t d = vd + j * (C::kStep * C::kSw >> 4);
                mma_ts<F8>(tO, tS + j * (F8 ? 24 : 8), d, kIdO, !first || j > 0);
                if (F8) mma_ts<F8>(tO, tS + j * 24 + 8, d, kIdO, true), mma_ts<F8>(tO, tS + j * 24 + 16, d, kIdO, true);
              }
              if (x >= units) mma_commit(b_o + 8 * st);  // the stream's last of the segment
              if (QM == 1 || st == 1) mma_commit(b_ve + 8 * vs);
            }
            __syncwarp();
            if (QM == 1 || st == 1)
              if (++vs == C::kV) vs = 0, ++vlap;
          }
          if (x < units) {
            const uint64_t qd = q0 + (QM == 2 ? st * (C::kQBytes >> 4) : 0), kd = k0 + ks * (C::kKBytes >> 4);
            if (!k_there) wait(sync, b_kf + 8 * ks, klap & 1, live);
            tc_fence_after();
            if (one && live) {
#pragma unroll
              for (int j = 0; j < C::kRow / 32; ++j) {
                const int at = j / (C::kSw / 32) * C::kHalfBytes + j % (C::kSw / 32) * 32;
                mma_ss<F8>(tS, qd + (at >> 4), kd + (at >> 4), kIdS, j > 0);
                if (F8) mma_ss<F8>(tS, qd + ((kTile * D + at) >> 4), kd + (at >> 4), kIdS, true);  // low parts
              }
              mma_commit(b_s + 8 * st);
            }
            __syncwarp();
            if (QM == 1 || st == 1)
              if (++ks == C::kK) ks = 0, ++klap;
          }
        }
      }
      // the last arrival that the products owe this block's memory
      if (vs + vlap > 0) wait(sync, b_ve + 8 * (vs ? vs - 1 : C::kV - 1), (vs ? vlap : vlap - 1) & 1);
    } else {  // warp 11
      // ---- the items' places, one ahead of the others -----------------------
      TcWalker list;
      bool more = true;
      int set = 0;
      auto publish = [&] {
        if (set >= kSegments) wait(sync, b_ge + 8 * (set % kSegments), (set / kSegments - 1) & 1);
        if (__any_sync(0xFFFFFFFFu, *sync.abort)) {
          more = false;
          return;
        }
        more = next_place<kMode>(P, list, &places[set % kSegments]);
        __syncwarp();
        if (lane == 0) mbar_arrive(b_gf + 8 * (set % kSegments));
        ++set;
      };
      if (kMode) {
        list.w = w0, list.w1 = w1, list.count = __ldcg(P.list.head + 1), list.whole = __ldcg(P.list.head + 2);
        list.at = __ldcg(P.list.first + blockIdx.x), list.lot = load_lot(P.list.lots + list.at);
      }
      if (F8 || kMode) {
        // ---- scales of 8-bit entries, from the tails that came with K into
        // what the softmax adds and multiplies by.  (Loading four bytes of an
        // entry by cp.async kept this warp 2000 cycles a tile: 64 single tokens
        // 216 us; loading the tails itself 1500: 193.)
        // ---- and V without non-finite values, where a list has it (see below)
        int slot = 0, lap = 0, due = 0, vslot = 0, vlap = 0;
        TcSegment seg;
        for (;; ++taken) {
          if (kMode) {
            // (the next one is needed, others are as soon as there is room)
            while (more && (set <= taken || set < kSegments ||
                            __all_sync(0xFFFFFFFFu, mbar_test_wait(b_ge + 8 * (set % kSegments), (set / kSegments - 1) & 1))))
              publish();
            if (taken >= set) break;
            seg = places[taken % kSegments].seg;
            if (seg.T == 0) break;
          } else if (!next(seg)) {
            break;
          }
#pragma unroll 1
          for (int t = seg.t0; t < seg.t1; ++t, ++due) {
            const TcTile k = tile_of<kMode>(P, seg, t);
            if (F8) {
              const int box = k.staged ? (kMode ? P.stage_box : kStageBox) : P.box, ring = due % kScaleRing;
              wait(sync, b_kf + 8 * slot, lap & 1);
              const char* tails = kslots + slot * C::kKBytes + C::kTileBytes;
              float ks[4], vs[4];
              // Scales are 0 .. 2^120; what is not (and what the place of a key past the
              // valid ones held) must not reach rows that do not see the entry.  K's is
              // 2^-126 at least (0 counts as that), so that an unseen score's -inf stays.
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int r = lane + 32 * e, in = r & (box - 1);
                const char* tail = tails + ((r - in) * 2 + in) * kTail;  // a box's K, then its V
                const float x = *reinterpret_cast<const float*>(tail), z = *reinterpret_cast<const float*>(tail + box * kTail);
                ks[e] = fminf(fmaxf(x, kLeastScale), 0x1p120f);
                vs[e] = fminf(fmaxf(z, 0.0f), 0x1p120f);
              }
              if (due >= kScaleRing) wait(sync, b_se + 8 * ring, (due / kScaleRing - 1) & 1);
              float* sc = s_sc + ring * 2 * kTile + lane;
#pragma unroll
              for (int e = 0; e < 4; ++e) sc[32 * e] = ks[e], sc[kTile + 32 * e] = vs[e];
              fence_async_smem();  // the tails have been read before their place is loaded again
              __syncwarp();
              if (lane == 0) mbar_arrive(b_sf + 8 * ring);
              if (++slot == C::kK) slot = 0, ++lap;
            }
            if (kMode) {
              int r0, r1;
              half_seen<kMode>(a, k, seg, &r0, &r1);
              char* v = vslots + vslot * C::kTileBytes;
              TcPlace* place = &places[taken % kSegments];
              // (the products wait for each tile's arrival here, so that no load's phase is missed)
              wait(sync, b_vf + 8 * vslot, vlap & 1);
              if ((kMode & kForms) && r1 < k.valid) {
                clean_rows<F8, kMode, C::kRow / 16>(P, place, t, k.own, k.x0, v, r0, r1, r1);
                r0 = k.valid;
              }
              if (r0 < k.valid || k.valid % C::kStep)
                clean_rows<F8, kMode, C::kRow / 16>(P, place, t, k.own, k.x0, v, r0, k.valid, (k.valid + C::kStep - 1) / C::kStep * C::kStep);
              __syncwarp();
              if (lane == 0) mbar_arrive(b_vc + 8 * vslot);
              if (++vslot == C::kV) vslot = 0, ++vlap;
            }
          }
        }
      }
      // ---- rows past each request's entries --------------------------------
      for (int r = blockIdx.x; r < a.B * a.R; r += gridDim.x) {
        const int b = r / a.R, i = r - b * a.R;
        if (i <= extent_of(a, b, P.p.err).n) continue;
        const float zero[8] = {};
        for (int c = lane; c < a.Hq * (D / 8); c += 32)
          store8<false>(a.out, b * a.out_stride[0] + i * a.out_stride[1] + c / (D / 8) * a.out_stride[2] + c % (D / 8) * 8, zero);
      }
    }
  } else {
    // ---- softmax ------------------------------------------------------------
    const int st = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t tS = tmem + (quad << 21) + st * 128, tO = tmem + (quad << 21) + 256 + st * 128;
    int kbase = 0, ph_s = 0, ph_o = 0, place_next = 0;
    TcSegment seg;
    for (;; give_back_place()) {
      if (kMode) {
        if (warp == 0) {
          const bool any = next(seg);
          if (lane == 0) ints[14] = any;
        }
        named_barrier(1, 256);
        if (!*reinterpret_cast<volatile int*>(&ints[14])) break;
        seg = places[taken % kSegments].seg;
      } else if (!next(seg)) {
        break;
      }
      const TcPlace& place = places[taken % kSegments];  // (of a list)
      const int n = seg.t1 - seg.t0, units = n * QM;
      const int i0 = seg.rb * C::kRows;
      // copies of the block's rows in the tile: this thread's copy weighs the
      // 32-key groups ch_a .. ch_b - 1 of each key tile
      const int rows = min(C::kRows, (seg.X.n + 1) * G - i0);
      const int fold = QM == 2 || rows > 64 ? 0 : rows > 32 ? 1 : 2, copies = 1 << fold, apart = kTile >> fold;
      const int copy = row >> (7 - fold), ch_a = copy << (2 - fold), ch_b = ch_a + (4 >> fold);
      const int lrow = QM == 2 ? st * kTile + row : row - copy * apart;  // row of the CTA's block
      const TcRow me = row_of<kMode>(P, seg, i0 + lrow);
      const int i = me.i, hq = me.hq;
      const bool live = (kMode & kShare) && seg.m > 0 ? lrow < rows && i <= place.mem.n[me.j] : i <= seg.X.n;
      TcForm form = {};
      int deepest = 0;  // row of the warp
      if (kMode & kForms) {
        form.cap = a.softcap * kLog2e;
        if (live) {
          const int depth = depth_of(a, me.b, i);
          form.at = ((kMode & kShare) && seg.m > 0 ? place.mem.S[me.j] : seg.X.S) + depth;
          form.slope = a.slopes ? a.slopes[hq] * kLog2e : 0.0f;
          deepest = depth;
        }
        deepest = __reduce_max_sync(0xFFFFFFFFu, deepest);
      }
      const bool warp_live = lrow - lane < rows;
      // queries: rows of this CTA's block, read once and written to each copy,
      // swizzled as the products read them
      {
        constexpr int kChunks = D / 8, kGroup = QM == 2 ? 128 : 256;
        const int each = apart * kChunks / kGroup;
        const int qt = QM == 2 ? row : tid, part0 = i0 + (QM == 2 ? st * kTile : 0);
        char* q = sm + (QM == 2 ? st * C::kQBytes : 0);
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;  // scores are compared before they are scaled
        const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(a.q) + seg.b * a.q_stride[0] + (int64_t)seg.h * G * a.q_stride[2];
        constexpr int kAt = F8 ? 4 : 8;  // loads in flight
#pragma unroll 1
        for (int it0 = 0; it0 < each; it0 += kAt) {
          uint4 x8[kAt];
#pragma unroll
          for (int it = 0; it < kAt; ++it) {
            const int idx = (it0 + it) * kGroup + qt, rr = part0 + idx / kChunks, qi = entry_of(P, rr);
            x8[it] = make_uint4(0, 0, 0, 0);
            if ((kMode & kShare) && seg.m > 0) {
              const TcRow to = row_of<kMode>(P, seg, rr);
              if (it0 + it < each && qi <= seg.X.n && to.i <= place.mem.n[to.j])
                x8[it] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + to.b * a.q_stride[0] + to.i * a.q_stride[1] +
                                                         to.hq * a.q_stride[2] + idx % kChunks * 8);
            } else if (it0 + it < each && qi <= seg.X.n)
              x8[it] = *reinterpret_cast<const uint4*>(q0 + qi * a.q_stride[1] + (rr - qi * G) * a.q_stride[2] + idx % kChunks * 8);
          }
#pragma unroll
          for (int it = 0; it < kAt; ++it) {
            if (it0 + it >= each) break;
            const int idx = (it0 + it) * kGroup + qt, r = idx / kChunks, c = idx % kChunks;  // r: row of the tile
            const uint4 v = make_uint4(x8[it].x ^ flip, x8[it].y ^ flip, x8[it].z ^ flip, x8[it].w ^ flip);
            if (!F8) {
              const int hf = c * 16 / C::kSw, in = c - hf * (C::kSw / 16);
              char* d = q + hf * C::kHalfBytes + r * C::kSw + ((in ^ (r & 7)) << 4);
#pragma unroll 1
              for (int x = 0; x < copies; ++x, d += apart * C::kSw) *reinterpret_cast<uint4*>(d) = v;
            } else {
              // q = scale (hi + lo): hi rounds to the 8-bit format's 4 significant
              // bits, and the rest of a bf16 value is at most 4 bits more, so the
              // two parts are exact (but for parts below 2^-10 of a row maximum
              // scaled to 224 .. 448)
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
              float x[8], m = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                x[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
                m = fmaxf(m, fabsf(x[e]));
              }
#pragma unroll
              for (int o = 1; o < kChunks; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
              const float qs = e4m3_scale(m, 1.0f);
              // 1 / qs by its exponent; an infinite query's codes are NaN, as its scores
              const float inv = m < kInf ? __uint_as_float(0x7F000000u - __float_as_uint(qs)) : __uint_as_float(0x7FC00000u);
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 y = make_float2(x[2 * e] * inv, x[2 * e + 1] * inv);
                hi[e] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
                const float2 z = e4m3x2_values(hi[e]);
                lo[e] = __nv_cvt_float2_to_fp8x2(make_float2(y.x - z.x, y.y - z.y), __NV_SATFINITE, __NV_E4M3);
              }
              const int in = c >> 1;
              const int sw = C::kSw == 128 ? in ^ (r & 7) : in ^ ((r >> 1) & 3);
              char* d = q + r * C::kSw + sw * 16 + (c & 1) * 8;
#pragma unroll 1
              for (int x = 0; x < copies; ++x, d += apart * C::kSw) {
                *reinterpret_cast<uint2*>(d) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                *reinterpret_cast<uint2*>(d + kTile * D) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                if (c == 0) s_qs[(QM == 2 ? st * kTile : 0) + r + x * apart] = qs;
              }
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_q);
        if (F8) named_barrier(QM == 2 ? 2 + st : 1, kGroup);  // the rows' scales
      }
      // positive (a subnormal at least), so that what is not seen stays -inf when it is scaled
      const float c_raw = fmaxf(fabsf(a.scale) * kLog2e * (F8 ? s_qs[(QM == 2 ? st * kTile : 0) + row] : 1.0f), 0x1p-149f);
      const bool shape = (kMode & kForms) && (F8 || a.softcap > 0.0f || a.slopes);
      const float c = shape ? 1.0f : c_raw;  // shaped scores have it already
      form.factor = form_factor(c_raw, form.cap);
      if ((kMode & kForms) && shape) form.factor = form.cap <= kCapNear && __all_sync(0xFFFFFFFFu, factor_within(form.factor)) ? form.factor : 0.0f;
      const uint64_t c2 = pair(c, c);
      // wr: reference of 8-bit weights, log2 units; raise = 2^(kBias + m - wr)
      float m = -kInf, l = 0.0f, wr = -kInf, raise = 0.0f;
      for (int u = st; u < units; u += 2) {
        const int tt = QM == 2 ? u >> 1 : u;
        const TcTile k = tile_of<kMode>(P, seg, seg.t0 + tt);
        const int kt = kbase + tt;
        const bool full = k.prefix && k.valid == kTile;
        // keys in a row that all rows of the warp see; else what they see, looked up while
        // the scores are under way, the places of keys by a thread each
        const bool clear = full && (!(kMode & kForms) || a.window == 0 || seg.X.S + deepest - k.x0 < a.window);
        uint32_t seen[4] = {0, 0, 0, 0};
        TcView view = {};
        // (a warp may still read those of the stream's last tile)
        int* places_at = s_at + (st * 2 + ((QM == 2 ? kt : kt >> 1) & 1)) * kTile;
        if (kMode) {
          if (warp_live && !clear) {
            view = view_of<kMode>(P, seg, &place.mem, k, me.j, live);
            if (!k.prefix) entries_seen(a, me.b, live ? i : 0, live ? (kMode & kShare) && seg.m > 0 ? place.mem.n[me.j] : seg.X.n : -1, view.e0, seen);
          }
          if ((kMode & kForms) && (a.window > 0 || a.slopes)) {
            // (the next tile's are on their way while this one is weighed)
            if (!k.prefix) {
              places_at[row] = u == st ? key_place<kMode>(P, place, k, row) : place_next;
              named_barrier(4 + st, 128);
            }
            if (u + 2 < units) {
              const TcTile next = tile_of<kMode>(P, seg, seg.t0 + (QM == 2 ? (u + 2) >> 1 : u + 2));
              if (!next.prefix) place_next = key_place<kMode>(P, place, next, row);
            }
          }
        }
        wait(sync, b_s + 8 * st, ph_s);
        ph_s ^= 1;
        if (F8) wait(sync, b_sf + 8 * (kt % kScaleRing), (kt / kScaleRing) & 1);
        if (quad == 0 && lane == 0) mbar_arrive(b_ke + 8 * (kt % C::kK));  // the scores' product is done with its keys, and their tails are read
        tc_fence_after();
        const float* sc = s_sc + (kt % kScaleRing) * 2 * kTile;
        if (warp_live) {
          const int chunks = (k.valid + 31) / 32, ch_e = min(ch_b, chunks);
          if (!kMode && !full) hide_unseen(P, seg.b, i, seg.X.n, k.prefix, k.valid, k.u0, ch_a, ch_e, tS);
          // One pass over the tile's scores, 32 columns at a time, so that the
          // loop stays short.  A group of 32 that exceeds the reference by too
          // much rescales what is there, the weights before it included.
          uint64_t ls[2] = {0, 0};
#pragma unroll 1
          for (int ch = 0; ch < chunks; ++ch) {
            constexpr int kW = F8 ? 24 : 16;  // columns of 32 weights
            uint32_t w[kW];
            // keys that the row sees, the distance of the first, and whether the others'
            // distances do not follow from it (then their places, a lane each)
            uint32_t bits = 0xFFFFFFFFu;
            int far = 0, at = 0;
            bool apart = false;
            if (kMode && ch >= ch_a && ch < ch_b) {
              if (clear) {
                far = form.at - k.x0 - 32 * ch;
              } else {
                const uint32_t of_mask = ch == 0 ? seen[0] : ch == 1 ? seen[1] : ch == 2 ? seen[2] : seen[3];
                bits = of_mask | cached_seen(view, ch);
                if (kMode & kForms) {
                  const int d = form.at - ((kMode & kShare) && seg.m > 0 ? place.mem.S[me.j] : seg.X.S);
                  far = d + view.org - 32 * ch;
                  if (!k.prefix && (a.window > 0 || a.slopes) && __any_sync(0xFFFFFFFFu, of_mask != 0)) {
                    at = places_at[32 * ch + lane];
                    // a chain's depths follow one another: distances do for keys up to the row
                    const int at0 = __shfl_sync(0xFFFFFFFFu, at, 0);
                    const bool in_row = __all_sync(0xFFFFFFFFu, at == at0 + lane) && !((kMode & kShare) && k.own);
                    if (in_row) far = d - at0;
                    apart = !in_row || __any_sync(0xFFFFFFFFu, bits != 0 && far < 31 - __clz(bits));
                  }
                  if (a.window > 0) {
                    if (!apart) {
                      if (far >= a.window) bits &= far - a.window >= 31 ? 0u : 0xFFFFFFFEu << (far - a.window);
                    } else {
                      const int least = __reduce_min_sync(0xFFFFFFFFu, at), most = __reduce_max_sync(0xFFFFFFFFu, at);
                      if (__any_sync(0xFFFFFFFFu, bits != 0 && max(abs(d - least), abs(d - most)) >= a.window))
#pragma unroll 8
                        for (int e = 0; e < 32; ++e)
                          if (abs(d - __shfl_sync(0xFFFFFFFFu, at, e)) >= a.window) bits &= ~(1u << e);
                    }
                  }
                  if (apart) far = d;
                }
              }
            }
            if (ch < ch_a || ch >= ch_b || (kMode && !__any_sync(0xFFFFFFFFu, bits != 0))) {  // another copy's keys, or no one's
#pragma unroll
              for (int e = 0; e < kW; ++e) w[e] = 0u;
              tmem_st(tS + kW * ch, w);
              continue;
            }
            if (F8) {
              // Weights by the references so far; where a row's sum or largest shows that
              // one is too low, once more after they have moved.
              const float* kp = kMode & kForms ? s_ones : sc + 32 * ch;
              bool bad = m == -kInf, again = false;
              bool shaped = kMode == 0;  // the scores in tensor memory are what the softmax takes
              uint64_t gs[2];
#pragma unroll 1
              while (true) {
                if (kMode && !shaped && (__any_sync(0xFFFFFFFFu, bad) || apart)) {
                  shaped = true;
                  if ((kMode & kForms) && shape)
                    shape_group<F8>(form.factor != 0.0f, tS + 32 * ch, c_raw, sc + 32 * ch, form.cap, form.slope, far, apart, at, bits);
                  else if (__any_sync(0xFFFFFFFFu, ~bits))
                    shape_chunk<false, kDirect>(tS + 32 * ch, 1.0f, nullptr, 0.0f, 0.0f, 0, false, 0, bits);
                }
                if (__any_sync(0xFFFFFFFFu, bad)) {
                  const float2 n = references<(kMode & kForms) != 0>(tS + 32 * ch, c, kp, sc + 32 * ch, m, wr, bad);
                  const float f = n.x > m ? ex2(m - n.x) : 1.0f, fw = n.y > wr ? ex2(wr - n.y) : 1.0f;
                  l *= f, ls[0] = mul2(ls[0], pair(f, f)), ls[1] = mul2(ls[1], pair(f, f));
                  m = n.x, wr = n.y;
                  raise = m == -kInf ? 0.0f : ex2(kBias + m - wr);
                  if (__any_sync(0xFFFFFFFFu, fw != 1.0f)) {
                    if (ch > ch_a) rescale_weights<F8>(tS + kW * ch_a, kW * (ch - ch_a), fw);
                    if (u >= 2) rescale(tO, D, fw);  // these scores were issued, and are done, after the last outputs
                  }
                }
                uint32_t x[32];
                tmem_ld32(tS + 32 * ch, x);
                if (kMode && !shaped) {
                  if ((kMode & kForms) && shape && !shape_near<F8>(x, sc + 32 * ch, form, far)) {
                    shape_group<F8>(form.factor != 0.0f, tS + 32 * ch, c_raw, sc + 32 * ch, form.cap, form.slope, far, false, 0, bits);
                    shaped = true;
                    tmem_ld32(tS + 32 * ch, x);
                  } else if (__any_sync(0xFFFFFFFFu, ~bits)) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = bits >> e & 1 ? x[e] : 0xFF800000u;
                  }
                }
                const float base = m == -kInf ? -kInf : -m;  // nothing seen: p is 0
                const uint64_t base2 = pair(base, base), raise2 = pair(raise, raise);
                float t4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                gs[0] = gs[1] = 0;
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  const ulonglong2 ks = kMode & kForms ? ulonglong2() : *reinterpret_cast<const ulonglong2*>(kp + 2 * e);
                  const ulonglong2 vs = *reinterpret_cast<const ulonglong2*>(sc + kTile + 32 * ch + 2 * e);
                  float2 y[2];
#pragma unroll
                  for (int z = 0; z < 2; ++z) {
                    const uint64_t s = pair(__uint_as_float(x[2 * (e + z)]), __uint_as_float(x[2 * (e + z) + 1]));
                    const float2 d = unpair(kMode & kForms ? add2(s, base2) : fma2(mul2(s, c2), z ? ks.y : ks.x, base2));  // -inf stays
                    const uint64_t p2 = pair(ex2(d.x), ex2(d.y));
                    gs[z] = add2(gs[z], p2);
                    y[z] = unpair(mul2(mul2(p2, z ? vs.y : vs.x), raise2));
                    float& top = t4[(e & 2) + z];
                    top = fmaxf(top, fmaxf(y[z].x, y[z].y));
                  }
                  const __half2 h0 = __floats2half2_rn(y[0].x, y[0].y), h1 = __floats2half2_rn(y[1].x, y[1].y);
                  uint32_t a0 = *reinterpret_cast<const uint32_t*>(&h0), a1 = *reinterpret_cast<const uint32_t*>(&h1);
                  w[e / 2] = __byte_perm(a0, a1, 0x7531);
                  a0 = less_top(a0), a1 = less_top(a1);
                  w[8 + e / 2] = __byte_perm(a0, a1, 0x7531);
                  a0 = less_top(a0) + 0x00800080u, a1 = less_top(a1) + 0x00800080u;
                  w[16 + e / 2] = __byte_perm(a0, a1, 0x7531);
                }
                const float2 g2 = unpair(add2(gs[0], gs[1]));
                bad = !(g2.x + g2.y <= kMostSum) || fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) > kMost;
                if (again || !__any_sync(0xFFFFFFFFu, bad)) break;
                again = true;
              }
              ls[0] = add2(ls[0], gs[0]), ls[1] = add2(ls[1], gs[1]);
            } else {
              uint32_t x[32];
              uint64_t v[16];
              if ((kMode & kForms) && shape) {
                if (!apart) tmem_ld32(tS + 32 * ch, x);
                if (apart || !shape_near<F8>(x, nullptr, form, far)) {
                  shape_group<F8>(form.factor != 0.0f, tS + 32 * ch, c_raw, nullptr, form.cap, form.slope, far, apart, at, bits);
                  tmem_ld32(tS + 32 * ch, x);
                }
              } else {
                tmem_ld32(tS + 32 * ch, x);
              }
              if (kMode && __any_sync(0xFFFFFFFFu, ~bits)) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = bits >> e & 1 ? x[e] : 0xFF800000u;
              }
              float mx4[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                v[e] = pair(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                mx4[e & 3] = fmaxf(mx4[e & 3], fmaxf(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])));
              }
              const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * c;
              if (__any_sync(0xFFFFFFFFu, mx > m + kSlack)) {
                // (A weight's argument rounds by its reference: with a list a row's moves for the row's own
                // scores alone.  In plain calls all lanes' move at once, and last bits may tell.)
                const float mn = kMode && !(mx > m + kSlack) ? m : fmaxf(m, ceilf(mx)), f = mn == -kInf ? 1.0f : ex2(m - mn);
                m = mn, l *= f;
                const uint64_t f2 = pair(f, f);
                ls[0] = mul2(ls[0], f2), ls[1] = mul2(ls[1], f2);
                if (ch > ch_a) rescale_weights<F8>(tS + kW * ch_a, kW * (ch - ch_a), f);
                if (u >= 2) rescale(tO, D, f);  // these scores were issued, and are done, after the last outputs
              }
              const float base = m == -kInf ? 0.0f : m;
              const uint64_t base2 = pair(-base, -base);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
#pragma unroll
                for (int z = e; z < e + 2; ++z) {
                  v[z] = fma2(v[z], c2, base2);
                  const float2 y = unpair(v[z]);
                  v[z] = pair(ex2(y.x), ex2(y.y));
                }
                const float2 y0 = unpair(v[e]), y1 = unpair(v[e + 1]);
                w[e] = pack_bf16(y0.x, y0.y);
                w[e + 1] = pack_bf16(y1.x, y1.y);
                if (kMode) {  // the weights as they are multiplied: a row of few keys keeps what rounding moved between them
                  ls[0] = add2(ls[0], pair(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u)));
                  ls[1] = add2(ls[1], pair(__uint_as_float(w[e + 1] << 16), __uint_as_float(w[e + 1] & 0xFFFF0000u)));
                } else {
                  ls[0] = add2(ls[0], v[e]), ls[1] = add2(ls[1], v[e + 1]);
                }
              }
            }
            tmem_st(tS + kW * ch, w);
          }
          const float2 l2 = unpair(add2(ls[0], ls[1]));
          l += l2.x + l2.y;
        }
        // The last product of a short tile takes whole steps of keys: the rows
        // past the valid ones are cleared.  Entries some rows do not see must
        // not ruin them through 0 * NaN: non-finite values of V are cleared and
        // given back to the rows that see them at the end.
        // With a list, most tiles are looked at in some calls (1400 of 8400 cycles of a prompt's
        // tile), and the warp that makes the items' places does it.
        if (!kMode) {
          int r0, r1;
          half_seen<kMode>(a, k, seg, &r0, &r1);
          if (r0 < r1 || k.valid % C::kStep) {
            const int slot = kt % C::kV, end = (k.valid + C::kStep - 1) / C::kStep * C::kStep;
            wait(sync, b_vf + 8 * slot, (kt / C::kV) & 1);
            clean_rows_plain<F8>(vslots + slot * C::kTileBytes, r0, k.valid, end, C::kRow / 16, row, &ints[2]);
          }
        }
        if (warp_live) tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_p + 8 * st);
          if (F8) mbar_arrive(b_se + 8 * (kt % kScaleRing));
        }
      }
      kbase += n;

      // ---- the segment's outputs -------------------------------------------
      if (st < units) {
        wait(sync, b_o + 8 * st, ph_o);
        ph_o ^= 1;
      }
      const bool both = QM == 1 && units > 1;  // stream 1 had a tile too
      if (QM == 1) s_ml[st * kTile + row] = make_float2(m, l);
      const float unit = F8 ? wr - kBias : m;  // of the outputs, log2
      if (F8 && QM == 1) s_wr[st * kTile + row] = unit;
      tc_fence_before();
      named_barrier(1, 256);
      tc_fence_after();
      const bool spoiled = *reinterpret_cast<const volatile int*>(kMode ? &place.found : &ints[2]) != 0;
      float f0 = 1.0f, f1 = 0.0f;  // of this copy's outputs in the two streams
      if (F8 && QM == 2) f0 = ex2(unit - (m == -kInf ? 0.0f : m));
      if (QM == 1) {
        float M = -kInf, L = 0.0f;
        const int parts = both ? 2 * copies : copies;  // a copy every `apart` rows, the second stream after the first
        float2 o[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          o[x] = x < parts ? s_ml[lrow + x * apart] : make_float2(-kInf, 0.0f);
          M = fmaxf(M, o[x].x);
        }
        const float Mb = M == -kInf ? 0.0f : M;
#pragma unroll
        for (int x = 0; x < 8; ++x) L += o[x].y * ex2(o[x].x - Mb);
        f0 = ex2((F8 ? s_wr[row] : s_ml[row].x) - Mb);
        f1 = both ? ex2((F8 ? s_wr[kTile + row] : s_ml[kTile + row].x) - Mb) : 0.0f;
        m = M, l = L;
      }
      const int c_first = QM == 1 ? st * (D / 2) : 0;
      constexpr int kCols = QM == 1 ? D / 2 : D;
      const int lead = kMode ? P.list.lead : kLead;
      const bool split = seg.t0 > 0 || seg.t1 + lead < seg.T;  // other CTAs have tiles of this item
      // a CTA has two partial results at most: of the item it starts in, and of its last
      float* part = P.p.part + (int64_t)(2 * blockIdx.x + (w0 >= seg.item0 ? 0 : 1)) * C::kPart;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int64_t out = me.b * a.out_stride[0] + i * a.out_stride[1] + (int64_t)hq * a.out_stride[2];
      float4* gather = reinterpret_cast<float4*>(sm);  // the queries' place: every score is done
#pragma unroll 1
      for (int col = c_first; col < c_first + kCols; col += 32) {
        float y[32];
        if (warp_live) {
          uint32_t o[32];
          const uint32_t t0 = tmem + (quad << 21) + 256 + col;
          tmem_ld32(QM == 1 ? t0 : t0 + st * 128, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(o[e]) * f0;
          if (both) {
            tmem_ld32(t0 + 128, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] += __uint_as_float(o[e]) * f1;
          }
        }
        auto put = [&](int at, const float* z) {  // eight columns of a row
          if (!split) {
            __nv_bfloat16* d = static_cast<__nv_bfloat16*>(a.out) + out + at;
            *reinterpret_cast<uint4*>(d) = make_uint4(pack_bf16(z[0] * inv, z[1] * inv), pack_bf16(z[2] * inv, z[3] * inv),
                                                      pack_bf16(z[4] * inv, z[5] * inv), pack_bf16(z[6] * inv, z[7] * inv));
            if (spoiled) give_back<F8, kMode>(P, kMode ? place.seg : found, &place, me, at, nullptr, d);
          } else {
            float* d = part + lrow * D + at;
            *reinterpret_cast<float4*>(d) = make_float4(z[0], z[1], z[2], z[3]);
            *reinterpret_cast<float4*>(d + 4) = make_float4(z[4], z[5], z[6], z[7]);
            if (spoiled) give_back<F8, kMode>(P, kMode ? place.seg : found, &place, me, at, d, nullptr);
          }
        };
        if (copies > 1) {  // each copy adds all shares of 32 / copies columns
          if (warp_live)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              gather[(copy * 16 + st * 8 + e) * apart + lrow] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          named_barrier(1, 256);
          if (live)
#pragma unroll 1
            for (int g = copy; g < 4; g += copies) {
              float z[8] = {};
#pragma unroll 2
              for (int x = 0; x < copies; ++x) {
                const float4* from = gather + (x * 16 + st * 8 + 2 * g) * apart + lrow;
                const float4 u = from[0], v = from[apart];
                z[0] += u.x, z[1] += u.y, z[2] += u.z, z[3] += u.w, z[4] += v.x, z[5] += v.y, z[6] += v.z, z[7] += v.w;
              }
              put(col + 8 * g, z);
            }
          named_barrier(1, 256);
        } else if (live) {
#pragma unroll
          for (int g = 0; g < 4; ++g) put(col + 8 * g, y + 8 * g);
        }
      }
      if (split && live && copy == 0 && (QM == 2 || st == 0))
        reinterpret_cast<float2*>(part + C::kRows * D)[lrow] = make_float2(m, l);
      if (split) {
        // the last of the item's CTAs joins the partial results, in the order
        // of the CTAs, so that results do not depend on who was last
        __threadfence();
        named_barrier(1, 256);
        if (tid == 0) {
          const int ca = share_of(seg.item0 + lead, total, ctas), cb = share_of(seg.item0 + seg.T - 1, total, ctas);
          ints[12] = ca, ints[13] = cb;
          uint32_t* ticket = P.p.ticket + ca;  // one item at most starts in a CTA and goes on in the next
          const bool last = atomicAdd(ticket, 1u) == (uint32_t)(cb - ca);
          if (last) *ticket = 0;
          ints[3] = last;
        }
        named_barrier(1, 256);
        if (*reinterpret_cast<volatile int*>(&ints[3])) {
          __threadfence();
          const int ca = ints[12], cb = ints[13];
          const float* first = P.p.part + (int64_t)(2 * ca + (mul_div(total, ca, ctas) >= seg.item0 ? 0 : 1)) * C::kPart;
          auto slot = [&](int x) { return x == ca ? first : P.p.part + (int64_t)(2 * x) * C::kPart; };
          auto part_ml = [&](int x, int r) { return __ldcg(reinterpret_cast<const float2*>(slot(x) + C::kRows * D) + r); };
          // With a list, each part's factor of a row, where the queries were (the outputs are
          // stored): so that the loads below wait for nothing (joining 256 rows of three parts with
          // factors made beside them: 42000 cycles, 28000 so)
          float* factor = reinterpret_cast<float*>(sm);
          const bool held = kMode && (cb - ca + 1) * rows * 4 <= C::kQAll;
          for (int r = tid; r < rows; r += 256) {
            float M = -kInf, L = 0.0f;
#pragma unroll 4
            for (int x = ca; x <= cb; ++x) M = fmaxf(M, part_ml(x, r).x);
            const float Mb = M == -kInf ? 0.0f : M;
#pragma unroll 4
            for (int x = ca; x <= cb; ++x) {
              const float2 v = part_ml(x, r);
              const float f = ex2(v.x - Mb);
              L += v.y * f;
              if (held) factor[(x - ca) * rows + r] = f;
            }
            s_ml[r] = make_float2(Mb, L);
          }
          named_barrier(1, 256);
          auto join = [&](int z) {
            const int r = z / (D / 8), col = z % (D / 8) * 8;
            const float2 ML = s_ml[r];
            float y[8] = {};
#pragma unroll 4
            for (int x = ca; x <= cb; ++x) {
              const float f = held ? factor[(x - ca) * rows + r] : ex2(part_ml(x, r).x - ML.x);
              const float4* v = reinterpret_cast<const float4*>(slot(x) + r * D + col);
              const float4 v0 = __ldcg(v), v1 = __ldcg(v + 1);
              y[0] += v0.x * f, y[1] += v0.y * f, y[2] += v0.z * f, y[3] += v0.w * f;
              y[4] += v1.x * f, y[5] += v1.y * f, y[6] += v1.z * f, y[7] += v1.w * f;
            }
            const TcRow to = row_of<kMode>(P, seg, i0 + r);
            if ((kMode & kShare) && seg.m > 0 && to.i > place.mem.n[to.j]) return;
            const float iv = 1.0f / ML.y;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = ML.y == 0.0f ? 0.0f : y[e] * iv;
            store8<false>(a.out, to.b * a.out_stride[0] + to.i * a.out_stride[1] + to.hq * a.out_stride[2] + col, y);
          };
          if (kMode) {
#pragma unroll 2
            for (int z = tid; z < rows * (D / 8); z += 256) join(z);
          } else {
            for (int z = tid; z < rows * (D / 8); z += 256) join(z);
          }
        }
      }
      // outputs, flags and exchanged maxima are free again
      tc_fence_before();
      named_barrier(1, 256);
      if (tid == 0) ints[2] = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*sync.abort) __nanosleep(1000000);  // copies already under way land before the block's memory is given up
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// One kernel as the host sees it.
struct TcKernel {
  void (*fn)(TcParams);
  int threads, smem, part;  // block, dynamic shared memory, floats of a partial result
};

// head_dim 64 or 128; tiles: row tiles per CTA, 1 or 2 (1 where requests share prefixes and scores have a form).
TcKernel tc_kernel_bf16(int head_dim, int tiles);
TcKernel tc_kernel_e4m3(int head_dim, int tiles);
TcKernel tc_kernel_bf16_forms(int head_dim, int tiles);
TcKernel tc_kernel_e4m3_forms(int head_dim, int tiles);
TcKernel tc_kernel_bf16_shared(int head_dim, int tiles);
TcKernel tc_kernel_e4m3_shared(int head_dim, int tiles);
TcKernel tc_kernel_bf16_both(int head_dim, int tiles);
TcKernel tc_kernel_e4m3_both(int head_dim, int tiles);

template <bool F8, int kMode>
TcKernel tc_kernel(int head_dim, int tiles) {
  auto k = [](auto shape, void (*fn)(TcParams)) { return TcKernel{fn, shape.kThreads, shape.kSmem, shape.kPart}; };
  if constexpr (kMode != (kForms | kShare))
    if (tiles == 2)
      return head_dim == 64 ? k(TcShape<F8, 64, 2, kMode>(), tc_attention_kernel<F8, 64, 2, kMode>)
                            : k(TcShape<F8, 128, 2, kMode>(), tc_attention_kernel<F8, 128, 2, kMode>);
  return head_dim == 64 ? k(TcShape<F8, 64, 1, kMode>(), tc_attention_kernel<F8, 64, 1, kMode>)
                        : k(TcShape<F8, 128, 1, kMode>(), tc_attention_kernel<F8, 128, 1, kMode>);
}

}  // namespace sv
