// Attention of a verify pass on the tensor cores: scores and outputs by
// tcgen05.mma with accumulators in tensor memory, K and V by TMA, for bf16 and
// 8-bit caches with heads of 64 or 128.
#pragma once

#include <cuda_fp16.h>

#include "attention.cuh"
#include "tcgen05.cuh"

namespace sv {

constexpr int kTile = 128;        // keys of a tile, and rows of a product
constexpr int kTcThreads = 384;   // two softmax groups of four warps, loads, products, two converting warps
constexpr int kStageBox = 16;     // staged entries per TMA box
constexpr int kScaleRing = 8;     // tiles whose scales are held

struct TcParams {
  AttnParams p;
  CUtensorMap pages, stage;
  int box;   // cached positions per TMA box: the largest power of two up to 128 that divides block_size
};

// F8: an 8-bit cache.  D: head_dim.  QM: row tiles of 128 per CTA.
//   QM = 1: up to 128 rows; the two streams (score, probability and output
//           regions of tensor memory, each with its softmax group) take the
//           even and the odd key tiles and are merged at the end.
//   QM = 2: more rows; the streams are two row tiles that share every key tile.
template <bool F8, int D, int QM>
struct TcShape {
  static constexpr int kRow = F8 ? D : 2 * D;                // bytes of a row without its tail
  static constexpr int kSw = kRow < 128 ? kRow : 128;        // swizzle = bytes of a row per half
  static constexpr int kHalves = kRow / kSw;
  static constexpr int kHalfBytes = kTile * kSw;
  static constexpr int kTileBytes = kTile * kRow;
  static constexpr int kQBytes = kTile * 2 * D;              // bf16 rows, or two 8-bit parts
  static constexpr int kWide = kTile * 128;                  // a half (64 columns) of a tile of 16-bit rows
  static constexpr int kV16 = F8 ? kTile * 2 * D : 0;        // V of a tile, converted
  static constexpr int kStep = 16;                           // keys of one product of weights and V
  static constexpr int kRows = kTile * QM;
  static constexpr int kMisc = 3072 + 4 * kRows + (F8 ? kScaleRing * 3 * kTile * 4 : 0);
  static constexpr int kRoom = 232448 - 1024 - kMisc - QM * kQBytes - 2 * kV16;
  static constexpr int kSlots = kRoom / kTileBytes < 10 ? kRoom / kTileBytes : 10;
  static constexpr int kSmem = 1024 + kMisc + QM * kQBytes + 2 * kV16 + kSlots * kTileBytes;
  static constexpr int kPart = kRows * (D + 2);              // floats of a partial result
};

// A CTA's share of the work: tiles [w, w1) of the list of all requests' items
// (head, row block) and their key tiles, in order.
struct TcWalk {
  const TcParams& P;
  int* err;
  int qrows, w, w1, b, base, T, items, tp, blocks;
  Extent X;
  __device__ __forceinline__ TcWalk(const TcParams& P_, int* err_, int qrows_) : P(P_), err(err_), qrows(qrows_) {}
  __device__ __forceinline__ void request(int b_) {
    const sv_attention_args& a = P.p.a;
    b = b_;
    X = extent_of(a, b, err);
    if (X.n < 0) {
      T = 0, items = 0, tp = 0, blocks = 1;
      return;
    }
    const int G = a.Hq / a.cache.heads;
    blocks = ((X.n + 1) * G + qrows - 1) / qrows;
    items = a.cache.heads * blocks;
    if (a.stage.data) {
      tp = (X.S + kTile - 1) / kTile;
      T = tp + (X.n + kTile) / kTile;
    } else {
      T = tp = (X.S + X.n + kTile) / kTile;
    }
  }
  __device__ __forceinline__ int count() const { return T * items; }
};

struct TcSegment {
  int b, h, rb, t0, t1, T, tp, item0;  // item0: where the item starts in the list
  Extent X;
};

// The next segment (one item's consecutive tiles); false at the end.
__device__ __forceinline__ bool next_segment(TcWalk& k, TcSegment& s) {
  if (k.w >= k.w1) return false;
  while (k.w >= k.base + k.count()) {
    k.base += k.count();
    k.request(k.b + 1);
  }
  const int at = k.w - k.base, item = at / k.T;
  s.b = k.b, s.h = item / k.blocks, s.rb = item % k.blocks;
  s.T = k.T, s.tp = k.tp, s.X = k.X;
  s.t0 = at % k.T;
  s.t1 = min(k.T, s.t0 + k.w1 - k.w);
  s.item0 = k.base + item * k.T;
  k.w += s.t1 - s.t0;
  return true;
}

// What a tile holds: `valid` keys, and u0, the entry number of its first key
// (negative: cached positions before entry 0).  prefix: cached positions only,
// all of them seen.
struct TcTile {
  bool staged, prefix;
  int x0, valid, u0;
};

__device__ __forceinline__ TcTile tile_of(const sv_attention_args& a, const TcSegment& s, int t) {
  TcTile k;
  k.staged = a.stage.data && t >= s.tp;
  k.x0 = k.staged ? (t - s.tp) * kTile : t * kTile;
  const int limit = k.staged ? s.X.n + 1 : a.stage.data ? s.X.S : s.X.S + s.X.n + 1;
  k.valid = min(kTile, limit - k.x0);
  k.u0 = k.staged ? k.x0 : k.x0 - s.X.S;
  k.prefix = !k.staged && (a.stage.data || k.x0 + k.valid <= s.X.S);
  return k;
}

// Ring position of a tile's K and V, counted from the segment's first load.
// Loads follow the order in which the products use them: with QM = 1,
// K0 K1 V0 K2 V1 ..; with QM = 2, K0 V0 K1 V1 ..
template <int QM>
__device__ __forceinline__ int k_pos(int t) {
  return QM == 2 ? 2 * t : t < 1 ? 0 : 2 * t - 1;
}
template <int QM>
__device__ __forceinline__ int v_pos(int t, int n) {
  return QM == 2 ? 2 * t + 1 : t + min(t + 2, n);
}

// Waits are bounded (1 s): one that runs out reports SV_ERR_TIMEOUT and turns
// every later wait, load and product of the CTA off, so that all roles run to
// their ends.
struct TcSync {
  volatile int* abort;
  int* err;
  __device__ __forceinline__ void wait(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return;
    uint64_t began = 0;
    for (int i = 1;; ++i) {
      if (mbar_try_wait(bar, parity)) return;
      if (i % 64 == 0) {
        if (*abort) return;
        const uint64_t t = global_ns();
        if (began == 0) began = t;
        if (t - began > 1000000000ull) {
          *abort = 1;
          report(err, SV_ERR_TIMEOUT);
          return;
        }
      }
    }
  }
};

// Each row's softmax keeps a reference maximum m (log2 units); it moves only
// when a tile exceeds it by more than kSlack, so that outputs in tensor memory
// are rescaled rarely.  Weights are 2^(kBias + kSlack) at most.  bf16 weights
// have fp32's range.  Over 8-bit caches they are fp16: 2^15 at most, so 11 bits
// hold down to 2^-25 of a row's largest weight and 8 bits to 2^-28.
template <bool F8>
struct TcSoft {
  static constexpr float kSlack = F8 ? 4.0f : 8.0f, kBias = F8 ? 11.0f : 0.0f;
};

template <bool F8, int D, int QM>
__global__ void __launch_bounds__(kTcThreads, 1) tc_attention_kernel(const __grid_constant__ TcParams P) {
  using C = TcShape<F8, D, QM>;
  extern __shared__ char smem_raw[];
  const sv_attention_args& a = P.p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.cache.heads, G = a.Hq / H;
  constexpr float kInf = __builtin_huge_valf();

  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  char* sm = smem_raw + pad;
  const uint32_t s0 = raw + pad;
  const uint32_t sQ = s0, sV16 = s0 + QM * C::kQBytes, sKV = sV16 + 2 * C::kV16;
  char* kv = sm + QM * C::kQBytes + 2 * C::kV16;
  char* misc = kv + C::kSlots * C::kTileBytes;
  const uint32_t bars = smem_u32(misc);
  const uint32_t b_full = bars, b_empty = bars + 8 * C::kSlots, b_s = bars + 16 * C::kSlots, b_p = b_s + 16,
                 b_o = b_s + 32, b_q = b_s + 48, b_vf = b_s + 56, b_ve = b_s + 72, b_sf = b_s + 88,
                 b_se = b_sf + 8 * kScaleRing;
  int* ints = reinterpret_cast<int*>(misc + 512);  // 0 tensor memory, 1 abort, 3 last, 4.. walk, 8.. non-finite entries by segment
  float2* s_ml = reinterpret_cast<float2*>(misc + 1024);  // [2][128] maxima and sums the streams exchange
  float* s_qs = reinterpret_cast<float*>(misc + 3072);    // [kRows] row scales of 8-bit queries
  float* s_sc = s_qs + C::kRows;                          // [kScaleRing][3][128] of a tile's entries: K's scale,
                                                          // log2 of V's, 1 / V's

  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) mbar_init(b_full + 8 * i, 1), mbar_init(b_empty + 8 * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(b_s + 8 * i, 1), mbar_init(b_p + 8 * i, 4), mbar_init(b_o + 8 * i, 1), mbar_init(b_vf + 8 * i, 2), mbar_init(b_ve + 8 * i, 1);
    mbar_init(b_q, 8);
    for (int i = 0; i < kScaleRing; ++i) mbar_init(b_sf + 8 * i, 2), mbar_init(b_se + 8 * i, 4 * QM);
    ints[1] = ints[8] = ints[9] = ints[10] = ints[11] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&P.pages);
    if (a.stage.data) tma_prefetch_map(&P.stage);
  }
  if (warp == 9) tmem_alloc(smem_u32(&ints[0]), 512);
  pdl_wait();
  pdl_trigger();

  // Every CTA counts the tiles of all requests and finds its share: an equal
  // number of consecutive tiles each, so no CTA waits for a longer sequence.
  TcWalk walk(P, P.p.err, C::kRows);
  {
    const int per = (a.B + kTcThreads - 1) / kTcThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; ++b) walk.request(b), mine += walk.count();
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) ints[16 + warp] = x;
    __syncthreads();
    int before = 0, total = 0;
    for (int i = 0; i < kTcThreads / 32; ++i) {
      if (i < warp) before += ints[16 + i];
      total += ints[16 + i];
    }
    const int first = before + x - mine;  // tiles of the requests before mine
    const int ctas = min((int)gridDim.x, total);
    int w0 = 0, w1 = 0;
    if ((int)blockIdx.x < ctas) {
      w0 = (int)((int64_t)total * blockIdx.x / ctas);
      w1 = (int)((int64_t)total * (blockIdx.x + 1) / ctas);
      if (mine > 0 && first <= w0 && w0 < first + mine) {
        int at = first;
        for (int b = b0; b < b1; ++b) {
          walk.request(b);
          if (w0 < at + walk.count()) {
            ints[4] = b, ints[5] = at;
            break;
          }
          at += walk.count();
        }
      }
    }
    if (tid == 0) ints[6] = total, ints[7] = ctas;  // for the joining of partial results
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    walk.w = w0, walk.w1 = w1, walk.base = 0;
    if (w1 > w0) {
      walk.base = ints[5];
      walk.request(ints[4]);
    }
  }
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&ints[0]);
  const TcSync sync{ints + 1, P.p.err};
  TcSegment seg;

  if (warp == 8) {
    asm volatile("fence.proxy.async.global;" ::: "memory");  // what earlier kernels wrote, for TMA
    // ---- loads ------------------------------------------------------------
    int pos = 0;
    auto load = [&](int t, int v) {
      const int slot = pos % C::kSlots, use = pos / C::kSlots;
      ++pos;
      const TcTile k = tile_of(a, seg, t);
      if (use > 0) sync.wait(b_empty + 8 * slot, (use - 1) & 1);
      if (__any_sync(0xFFFFFFFFu, *sync.abort)) return;
      const int box = k.staged ? kStageBox : P.box;
      const int boxes = (k.valid + box - 1) / box;
      const uint32_t bar = b_full + 8 * slot, dst = sKV + slot * C::kTileBytes + lane * box * C::kSw;
      if (lane == 0) mbar_expect_tx(bar, boxes * box * C::kRow);
      __syncwarp();
      if (lane >= boxes) return;
      constexpr int kElems = F8 ? C::kSw : C::kSw / 2;
      if (k.staged) {
        const int run = (a.stage.layer * 2 + v) * H + seg.h;
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_4d(dst + hf * C::kHalfBytes, &P.stage, bar, hf * kElems, k.x0 + lane * box, run, seg.b);
      } else {
        const int x = k.x0 + lane * box, j = x / a.cache.block_size;
        const int blk = __ldg(a.cache.block_table + (int64_t)seg.b * a.cache.max_blocks + j);
        const bool ok = blk >= 0 && blk < a.cache.num_blocks;
        if (!ok) report(P.p.err, SV_ERR_STATE);
        // outside the pool: past the last run, where a load gives zeros
        const int run = ((ok ? blk : a.cache.num_blocks) * a.cache.layers + a.cache.layer) * 2 * H + v * H + seg.h;
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(dst + hf * C::kHalfBytes, &P.pages, bar, hf * kElems, x - j * a.cache.block_size, run);
      }
    };
    while (next_segment(walk, seg)) {
      const int n = seg.t1 - seg.t0;
      load(seg.t0, 0);
      if (QM == 1 && n > 1) load(seg.t0 + 1, 0);
      for (int t = 0; t < n; ++t) {
        load(seg.t0 + t, 1);
        const int ahead = t + (QM == 1 ? 2 : 1);
        if (ahead < n) load(seg.t0 + ahead, 0);
      }
    }
  } else if (warp == 9) {
    // ---- products ---------------------------------------------------------
    if (lane == 0) {
      int pos = 0, kbase = 0, ph_p = 0, ph_q = 0;  // ph_p: a bit per stream
      constexpr uint32_t kIdS = instr_desc(F8 ? 0 : 1, kTile, kTile, false);  // e4m3 or bf16
      constexpr uint32_t kIdO = instr_desc(F8 ? 0 : 1, kTile, D, true);       // fp16 or bf16
      while (next_segment(walk, seg)) {
        const int n = seg.t1 - seg.t0, units = n * QM;
        sync.wait(b_q, ph_q);
        ph_q ^= 1;
        auto scores = [&](int u) {
          const int st = u & 1, t = QM == 2 ? u >> 1 : u, at = pos + k_pos<QM>(t), slot = at % C::kSlots;
          sync.wait(b_full + 8 * slot, (at / C::kSlots) & 1);
          if (*sync.abort) return;
          tc_fence_after();
          const uint32_t q = sQ + (QM == 2 ? st * C::kQBytes : 0), k = sKV + slot * C::kTileBytes;
#pragma unroll
          for (int j = 0; j < C::kRow / 32; ++j) {
            const int hf = j / (C::kSw / 32), in = (j % (C::kSw / 32)) * 32;
            const uint64_t kd = smem_desc(k + hf * C::kHalfBytes + in, 16, 8 * C::kSw, C::kSw);
            const uint64_t qd = smem_desc(q + hf * C::kHalfBytes + in, 16, 8 * C::kSw, C::kSw);
            mma_ss<F8>(tmem + st * 128, qd, kd, kIdS, j > 0);
            if (F8)  // the queries' low parts
              mma_ss<F8>(tmem + st * 128, smem_desc(q + kTile * D + in, 16, 8 * C::kSw, C::kSw), kd, kIdS, true);
          }
          mma_commit(b_s + 8 * st);
          if (QM == 1 || st == 1) mma_commit(b_empty + 8 * slot);
        };
        scores(0);
        if (units > 1) scores(1);
        for (int u = 0; u < units; ++u) {
          const int st = u & 1, t = QM == 2 ? u >> 1 : u, at = pos + v_pos<QM>(t, n), slot = at % C::kSlots;
          sync.wait(b_p + 8 * st, ph_p >> st & 1);
          ph_p ^= 1 << st;
          const int vt = kbase + t;
          if (F8)
            sync.wait(b_vf + 8 * (vt & 1), vt >> 1 & 1);
          else
            sync.wait(b_full + 8 * slot, (at / C::kSlots) & 1);
          if (!*sync.abort) {
            tc_fence_after();
            const uint32_t v = F8 ? sV16 + (vt & 1) * C::kV16 : sKV + slot * C::kTileBytes;
            const int steps = (tile_of(a, seg, seg.t0 + t).valid + C::kStep - 1) / C::kStep;
            const bool first = u < 2;  // of this stream in this segment
            for (int j = 0; j < steps; ++j)
              mma_ts<false>(tmem + 256 + st * 128, tmem + st * 128 + j * 8,
                            smem_desc(v + j * C::kStep * 128, C::kWide, 1024, 128), kIdO, !first || j > 0);
            mma_commit(b_o + 8 * st);
            if (QM == 1 || st == 1) mma_commit(F8 ? b_ve + 8 * (vt & 1) : b_empty + 8 * slot);
          }
          if (u + 2 < units) scores(u + 2);
        }
        pos += 2 * n;
        kbase += n;
      }
    }
  } else if (warp >= 10) {
    // ---- 8-bit entries: scales, V to fp16; and the rows past each request's entries
    const int me = warp - 10;
    if (F8) {
      // Weights times V is an fp16 product: 8-bit weights would lose what lies
      // 2^-18 below a row's maximum, and a long sequence has most of its mass
      // there.  The scores' product takes the codes of K as they are.
      int pos = 0, kbase = 0, index = 0;
      const int ct = me * 32 + lane;
      float ks[2], vs[2];
      auto fetch = [&](int t) {  // this thread's two entries of a tile: scales of K and V
        const TcTile tl = tile_of(a, seg, t);
        const sv_kv_place& pl = tl.staged ? a.stage : a.cache;
        const int64_t step = row_step(pl);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = e * 64 + ct;
          ks[e] = vs[e] = 1.0f;
          if (r < tl.valid) {
            const int64_t off = entry_offset(pl, seg.b, tl.x0 + r, tl.x0 + r);
            if (off >= 0) {
              const char* row = static_cast<const char*>(pl.data) + off + seg.h * step + D;
              ks[e] = __ldg(reinterpret_cast<const float*>(row));
              vs[e] = __ldg(reinterpret_cast<const float*>(row + H * step));
            }
          }
        }
      };
      auto publish = [&](int k) {
        const int slot = k % kScaleRing, use = k / kScaleRing;
        if (use > 0) sync.wait(b_se + 8 * slot, (use - 1) & 1);
        float* sc = s_sc + slot * 3 * kTile;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float v = fmaxf(vs[e], 1.17549435e-38f);  // a NaN counts as the least here and as itself in the weight
          sc[e * 64 + ct] = ks[e];
          sc[kTile + e * 64 + ct] = vs[e] == vs[e] ? lg2(v) : vs[e];
          sc[2 * kTile + e * 64 + ct] = 1.0f / v;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b_sf + 8 * slot);
      };
      auto convert = [&](int t, int n) {
        const TcTile tl = tile_of(a, seg, seg.t0 + t);
        const int at = pos + v_pos<QM>(t, n), slot = at % C::kSlots, vt = kbase + t, use = vt >> 1;
        sync.wait(b_full + 8 * slot, (at / C::kSlots) & 1);
        if (use > 0) sync.wait(b_ve + 8 * (vt & 1), (use - 1) & 1);
        const char* src = kv + slot * C::kTileBytes;
        char* dst = sm + QM * C::kQBytes + (vt & 1) * C::kV16;
        const int tree = a.stage.data && !tl.staged ? kTile : max(0, -tl.u0);  // first entry some row may not see
        const int rows = (tl.valid + C::kStep - 1) / C::kStep * C::kStep;
        constexpr int kVecs = D / 16;
#pragma unroll 4
        for (int x = ct; x < rows * kVecs; x += 64) {
          const int r = x / kVecs, c = x % kVecs;
          uint4 y = *reinterpret_cast<const uint4*>(src + r * C::kSw + ((c ^ (C::kSw == 128 ? r & 7 : r >> 1 & 3)) << 4));
          if (r >= tl.valid) {
            y = make_uint4(0, 0, 0, 0);
          } else if (r >= tree) {
            // entries some rows do not see must not ruin them through 0 * NaN
            auto bad = [](uint32_t z) { return __vcmpeq4(z & 0x7F7F7F7Fu, 0x7F7F7F7Fu); };
            const uint32_t bx = bad(y.x), by = bad(y.y), bz = bad(y.z), bw = bad(y.w);
            if (bx | by | bz | bw) {
              y.x &= ~bx, y.y &= ~by, y.z &= ~bz, y.w &= ~bw;
              *reinterpret_cast<volatile int*>(&ints[8 + (index & 3)]) = 1;
            }
          }
          const uint32_t w[4] = {y.x, y.y, y.z, y.w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[e >> 1] >> (e & 1) * 16), __NV_E4M3);
            o[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          char* d = dst + (c >> 2) * C::kWide + r * 128;
          const int cc = (c & 3) * 2;
          *reinterpret_cast<uint4*>(d + ((cc ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(d + (((cc + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_async_smem();
        named_barrier(4, 64);  // both warps have read the slot
        if (ct == 0) mbar_arrive(b_empty + 8 * slot);
        if (lane == 0) mbar_arrive(b_vf + 8 * (vt & 1));
      };
      while (next_segment(walk, seg)) {
        const int n = seg.t1 - seg.t0;
        fetch(seg.t0);
        publish(kbase);
        if (n > 1) fetch(seg.t0 + 1), publish(kbase + 1);
        for (int t = 0; t < n; ++t) {
          if (t + 2 < n) fetch(seg.t0 + t + 2);  // on its way while V is converted
          convert(t, n);
          if (t + 2 < n) publish(kbase + t + 2);
        }
        pos += 2 * n;
        kbase += n;
        ++index;
      }
    }
    for (int r = blockIdx.x * 2 + me; r < a.B * a.R; r += gridDim.x * 2) {
      const int b = r / a.R, i = r - b * a.R;
      if (i <= extent_of(a, b, P.p.err).n) continue;
      const float zero[8] = {};
      for (int c = lane; c < a.Hq * (D / 8); c += 32)
        store8<false>(a.out, b * a.out_stride[0] + i * a.out_stride[1] + c / (D / 8) * a.out_stride[2] + c % (D / 8) * 8, zero);
    }
  } else {
    // ---- softmax ----------------------------------------------------------
    const int st = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t tS = tmem + (quad << 21) + st * 128, tO = tmem + (quad << 21) + 256 + st * 128;
    const int total = ints[6], ctas = ints[7];
    int pos = 0, kbase = 0, ph_s = 0, done = 0;  // done: outputs committed by this stream so far
    int index = 0;  // of the segment
    while (next_segment(walk, seg)) {
      const int n = seg.t1 - seg.t0, units = n * QM;
      const int lrow = (QM == 2 ? st * kTile : 0) + row;        // row of the CTA's block
      const int i0 = seg.rb * C::kRows;
      const int i = (i0 + lrow) / G, hq = seg.h * G + (i0 + lrow) % G;
      const bool live = i <= seg.X.n;
      const bool warp_live = (i0 + lrow - lane) / G <= seg.X.n;
      // queries: rows of this CTA's block, swizzled as the products read them
      {
        constexpr int kChunks = D / 8, kThreads = QM == 2 ? 128 : 256;
        const int qt = QM == 2 ? row : tid;
        char* q = sm + (QM == 2 ? st * C::kQBytes : 0);
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;  // scores are compared before they are scaled
#pragma unroll
        for (int it = 0; it < kTile * kChunks / kThreads; ++it) {
          const int idx = it * kThreads + qt, r = idx / kChunks, c = idx % kChunks;
          const int rr = i0 + (QM == 2 ? st * kTile : 0) + r, qi = rr / G;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (qi <= seg.X.n)
            v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + seg.b * a.q_stride[0] +
                                                qi * a.q_stride[1] + (seg.h * G + rr % G) * a.q_stride[2] + c * 8);
          v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
          if (!F8) {
            const int hf = c * 16 / C::kSw, in = c - hf * (C::kSw / 16);
            *reinterpret_cast<uint4*>(q + hf * C::kHalfBytes + r * C::kSw + ((in ^ (r & 7)) << 4)) = v;
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
            const float qs = e4m3_scale(m), inv = 1.0f / qs;
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
            *reinterpret_cast<uint2*>(d) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2*>(d + kTile * D) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
            if (c == 0) s_qs[(QM == 2 ? st * kTile : 0) + r] = qs;
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_q);
        if (F8) named_barrier(QM == 2 ? 2 + st : 1, kThreads);  // the rows' scales
      }
      const float c = fabsf(a.scale) * kLog2e * (F8 ? s_qs[lrow] : 1.0f);
      float m = -kInf, l = 0.0f;
      for (int u = st; u < units; u += 2) {
        const int tt = QM == 2 ? u >> 1 : u;
        const TcTile k = tile_of(a, seg, seg.t0 + tt);
        const int ring = kbase + tt;
        sync.wait(b_s + 8 * st, ph_s);
        ph_s ^= 1;
        if (F8) sync.wait(b_sf + 8 * (ring % kScaleRing), (ring / kScaleRing) & 1);
        tc_fence_after();
        const float* sc = s_sc + (ring % kScaleRing) * 3 * kTile;
        if (warp_live) {
          auto bits_of = [&](int ch) -> uint32_t {
            if (k.prefix) {
              const int left = k.valid - 32 * ch;
              return left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
            }
            return live ? seen_bits(a, seg.b, i, seg.X.n, k.u0 + 32 * ch) : 0u;
          };
          const int chunks = (k.valid + 31) / 32;
          const bool full = k.prefix && k.valid == kTile;
          float mx = -kInf;
          for (int ch = 0; ch < chunks; ++ch) {
            uint32_t s[32];
            tmem_ld32(tS + 32 * ch, s);
            const uint32_t bits = full ? 0xFFFFFFFFu : bits_of(ch);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float y[4];
              if (F8) {
                const float4 ks = *reinterpret_cast<const float4*>(sc + 32 * ch + e);
                const float4 lv = *reinterpret_cast<const float4*>(sc + kTile + 32 * ch + e);
                y[0] = __uint_as_float(s[e]) * (ks.x * c) + lv.x, y[1] = __uint_as_float(s[e + 1]) * (ks.y * c) + lv.y;
                y[2] = __uint_as_float(s[e + 2]) * (ks.z * c) + lv.z, y[3] = __uint_as_float(s[e + 3]) * (ks.w * c) + lv.w;
              } else {
#pragma unroll
                for (int z = 0; z < 4; ++z) y[z] = __uint_as_float(s[e + z]);
              }
              if (full) {
#pragma unroll
                for (int z = 0; z < 4; ++z) mx = fmaxf(mx, y[z]);
              } else {
#pragma unroll
                for (int z = 0; z < 4; ++z) mx = fmaxf(mx, bits >> (e + z) & 1 ? y[z] : -kInf);
              }
            }
          }
          if (!F8) mx = mx == -kInf ? mx : mx * c;
          const float mn = fmaxf(m, mx);
          if (__any_sync(0xFFFFFFFFu, mn > m + TcSoft<F8>::kSlack || (m == -kInf && mn > m))) {
            if (u >= 2) {
              const float f = mn == -kInf ? 1.0f : ex2(m - mn);
              l *= f;
              sync.wait(b_o + 8 * st, (done - 1) & 1);
              tc_fence_after();
#pragma unroll
              for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t o[32];
                tmem_ld32(tO + 32 * ch, o);
    #pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(tO + 32 * ch, o);
              }
            }
            m = mn;
          }
          const float base = (m == -kInf ? 0.0f : m) - TcSoft<F8>::kBias;
          float ls[4] = {};
          for (int ch = 0; ch < chunks; ++ch) {
            uint32_t s[32];
            tmem_ld32(tS + 32 * ch, s);
            const uint32_t bits = full ? 0xFFFFFFFFu : bits_of(ch);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float y[4];
              if (F8) {
                const float4 ks = *reinterpret_cast<const float4*>(sc + 32 * ch + e);
                const float4 lv = *reinterpret_cast<const float4*>(sc + kTile + 32 * ch + e);
                const float4 iv = *reinterpret_cast<const float4*>(sc + 2 * kTile + 32 * ch + e);
                const float ksv[4] = {ks.x, ks.y, ks.z, ks.w}, lvv[4] = {lv.x, lv.y, lv.z, lv.w};
                const float ivv[4] = {iv.x, iv.y, iv.z, iv.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  y[z] = ex2(__uint_as_float(s[e + z]) * (ksv[z] * c) + lvv[z] - base);
                  if (!full) y[z] = bits >> (e + z) & 1 ? y[z] : 0.0f;
                  ls[z] += y[z] * ivv[z];
                }
                const __half2 h0 = __floats2half2_rn(y[0], y[1]), h1 = __floats2half2_rn(y[2], y[3]);
                w[e / 2] = *reinterpret_cast<const uint32_t*>(&h0);
                w[e / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
              } else {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  y[z] = ex2(__uint_as_float(s[e + z]) * c - base);
                  if (!full) y[z] = bits >> (e + z) & 1 ? y[z] : 0.0f;
                  ls[z] += y[z];
                }
                w[e / 2] = pack_bf16(y[0], y[1]);
                w[e / 2 + 1] = pack_bf16(y[2], y[3]);
              }
            }
            tmem_st16(tS + 16 * ch, w);
          }
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        }
        // The last product of a short tile takes whole steps of keys: the rows
        // past the valid ones are cleared.  Entries some rows do not see must
        // not ruin them through 0 * NaN: non-finite values of V are cleared and
        // given back to the rows that see them at the end.  (The converting
        // warps do this for 8-bit entries.)
        const bool tree = k.valid > -k.u0 && !(a.stage.data && !k.staged);
        if (!F8 && (tree || k.valid % C::kStep)) {
          const int at = pos + v_pos<QM>(tt, n), slot = at % C::kSlots;
          sync.wait(b_full + 8 * slot, (at / C::kSlots) & 1);
          char* v = kv + slot * C::kTileBytes;
          constexpr int kVecs = C::kRow / 16, kPer = C::kSw / 16;
          const int r0 = tree ? max(0, -k.u0) : k.valid;
          const int r1 = (k.valid + C::kStep - 1) / C::kStep * C::kStep;
          for (int x = row; x < (r1 - r0) * kVecs; x += 128) {
            const int r = r0 + x / kVecs, cc = x % kVecs;
            uint4* d = reinterpret_cast<uint4*>(v + cc / kPer * C::kHalfBytes + r * C::kSw + cc % kPer * 16);
            if (r >= k.valid) {
              *d = make_uint4(0, 0, 0, 0);
            } else {
              uint4 y = *d;
              auto bad = [](uint32_t z) { return __vcmpeq2(z & 0x7F807F80u, 0x7F807F80u); };
              const uint32_t bx = bad(y.x), by = bad(y.y), bz = bad(y.z), bw = bad(y.w);
              if (bx | by | bz | bw) {
                y.x &= ~bx, y.y &= ~by, y.z &= ~bz, y.w &= ~bw;
                *d = y;
                *reinterpret_cast<volatile int*>(&ints[8 + (index & 3)]) = 1;
              }
            }
          }
          fence_async_smem();
        }
        if (warp_live) tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_p + 8 * st);
          if (F8) mbar_arrive(b_se + 8 * (ring % kScaleRing));
        }
        ++done;
      }
      pos += 2 * n;
      kbase += n;

      // ---- the segment's outputs -------------------------------------------
      const bool mine = st < units;  // this stream had a tile
      if (mine) sync.wait(b_o + 8 * st, (done - 1) & 1);
      if (QM == 1) s_ml[st * kTile + row] = make_float2(m, l);
      tc_fence_before();
      named_barrier(1, 256);
      tc_fence_after();
      const bool spoiled = *reinterpret_cast<volatile int*>(&ints[8 + (index & 3)]) != 0;
      const bool both = QM == 1 && units > 1;
      float f0 = 1.0f, f1 = 0.0f;
      if (QM == 1) {
        // both groups need both streams' m and l
        const float2 o = st == 1 || both ? s_ml[(st ^ 1) * kTile + row] : make_float2(-kInf, 0.0f);
        const float M = fmaxf(m, o.x), Mb = M == -kInf ? 0.0f : M;
        const float fm = ex2(m - Mb), fo = ex2(o.x - Mb);
        l = l * fm + o.y * fo;
        f0 = st == 0 ? fm : fo, f1 = st == 0 ? fo : fm;
        m = M;
      }
      const int c_first = QM == 1 ? st * (D / 2) : 0;
      constexpr int kCols = QM == 1 ? D / 2 : D;
      const int64_t T0 = seg.item0, T1 = seg.item0 + seg.T;
      auto cta_of = [&](int64_t x) { return (int)(((x + 1) * ctas - 1) / total); };
      const int ca = cta_of(T0), cb = cta_of(T1 - 1);
      const bool split = ca != cb;
      float* part = P.p.part + (int64_t)(2 * blockIdx.x + (index == 0 ? 0 : 1)) * C::kPart;
      const float inv = split ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
      const int64_t out = seg.b * a.out_stride[0] + i * a.out_stride[1] + (int64_t)hq * a.out_stride[2];
      auto put = [&](int col, const float (&y)[32]) {
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          const float z[8] = {y[e], y[e + 1], y[e + 2], y[e + 3], y[e + 4], y[e + 5], y[e + 6], y[e + 7]};
          store8<false>(a.out, out + col + e, z);
        }
      };
      if (warp_live) {
        for (int ch = 0; ch < kCols / 32; ++ch) {
          const int col = c_first + 32 * ch;
          float y[32];
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
          if (spoiled && live) {
            for (int t = seg.t0; t < seg.t1; ++t) {
              const TcTile k = tile_of(a, seg, t);
              if (a.stage.data && !k.staged) continue;
              const sv_kv_place& pl = k.staged ? a.stage : a.cache;
              for (int r = max(0, -k.u0); r < k.valid; ++r) {
                if (!(seen_bits(a, seg.b, i, seg.X.n, k.u0 + r) & 1)) continue;
                const int64_t off = entry_offset(pl, seg.b, k.x0 + r, k.x0 + r);
                if (off < 0) continue;
                const char* vr = static_cast<const char*>(pl.data) + off + (H + seg.h) * row_step(pl);
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                  float x[8];
                  load_entry8(vr, pl.format, col + e, 1.0f, x);
#pragma unroll
                  for (int z = 0; z < 8; ++z)
                    if (!(fabsf(x[z]) < kInf)) y[e + z] += x[z];
                }
              }
            }
          }
          if (!split) {
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = l == 0.0f ? 0.0f : y[e] * inv;
            if (live) put(col, y);
          } else if (live) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              reinterpret_cast<float4*>(part)[((col + e) / 4) * C::kRows + lrow] = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        }
        if (split && live && (QM == 2 || st == 0))
          reinterpret_cast<float2*>(part + C::kRows * D)[lrow] = make_float2(m, l);
      }
      if (split) {
        // the last of the item's CTAs joins the partial results, in the order
        // of the CTAs, so that results do not depend on who was last
        __threadfence();
        named_barrier(1, 256);
        if (tid == 0) {
          uint32_t* ticket = P.p.ticket + ca;  // one item at most starts in a CTA and goes on in the next
          const bool last = atomicAdd(ticket, 1u) == (uint32_t)(cb - ca);
          if (last) *ticket = 0;
          ints[3] = last;
        }
        named_barrier(1, 256);
        if (*reinterpret_cast<volatile int*>(&ints[3]) && live) {
          __threadfence();
          auto slot = [&](int x) {
            const int w0 = (int)((int64_t)total * x / ctas);
            return P.p.part + (int64_t)(2 * x + (w0 >= T0 ? 0 : 1)) * C::kPart;
          };
          float M = -kInf, L = 0.0f;
          for (int x = ca; x <= cb; ++x) M = fmaxf(M, __ldcg(reinterpret_cast<const float2*>(slot(x) + C::kRows * D) + lrow).x);
          const float Mb = M == -kInf ? 0.0f : M;
          for (int x = ca; x <= cb; ++x) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(slot(x) + C::kRows * D) + lrow);
            L += v.y * ex2(v.x - Mb);
          }
          const float iv = L == 0.0f ? 0.0f : 1.0f / L;
          for (int ch = 0; ch < kCols / 32; ++ch) {
            const int col = c_first + 32 * ch;
            float y[32] = {};
            for (int x = ca; x <= cb; ++x) {
              const float* sp = slot(x);
              const float f = ex2(__ldcg(reinterpret_cast<const float2*>(sp + C::kRows * D) + lrow).x - Mb);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(sp) + ((col + e) / 4) * C::kRows + lrow);
                y[e] += v.x * f, y[e + 1] += v.y * f, y[e + 2] += v.z * f, y[e + 3] += v.w * f;
              }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = L == 0.0f ? 0.0f : y[e] * iv;
            put(col, y);
          }
        }
      }
      // outputs, flags and exchanged maxima are free again
      tc_fence_before();
      named_barrier(1, 256);
      if (tid == 0) ints[8 + (index & 3)] = 0;  // the converting warps are two segments ahead at most
      ++index;
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
  int smem, part;  // dynamic shared memory, floats of a partial result
};

// head_dim 64 or 128; tiles: row tiles per CTA, 1 or 2.
TcKernel tc_kernel_bf16(int head_dim, int tiles);
TcKernel tc_kernel_e4m3(int head_dim, int tiles);

template <bool F8, int D, int QM>
TcKernel tc_kernel() {
  return {tc_attention_kernel<F8, D, QM>, TcShape<F8, D, QM>::kSmem, TcShape<F8, D, QM>::kPart};
}

}  // namespace sv
