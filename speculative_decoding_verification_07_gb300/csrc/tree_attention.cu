// Attention of a verify pass over the paged cache and the pass's own entries:
// the host entry, and the kernel for fp32 and for shapes outside the tensor
// kernel's.
#include "attention_tc.cuh"

namespace sv {

constexpr int kSimtWarps = 4, kSimtKeys = 32;
constexpr int kSimtThreads = 32 * kSimtWarps;

// o = sum_x p_x V_x with the running maximum and sum of a softmax: one pass
// over the keys, 32 at a time.  One CTA takes 4 RPW rows (entry, head of the
// group) of one KV head, so the keys are read once for all of them, and one of
// `splits` shares of the keys; the share that arrives last joins the others in
// share order, which keeps results the same from call to call.  A tile's K and
// V are decoded to fp32 in shared memory; a lane is a key for the scores and
// four columns (per 128) for the output.  fp32 products bound it with many
// rows (16 FMA to five shared-memory reads), latency with few: fewer rows a warp
// then.  One request of 6 rows over 38 keys, 4 heads of 64: 18.8 us with 4 rows a
// warp and a tile's loads one after another, 10.2 us as it is.
// X: the scores may have a form (capped, less with the distance, a window).
template <bool F32, int RPW, bool X>
__global__ void __launch_bounds__(kSimtThreads) simt_attention_kernel(const __grid_constant__ AttnParams P) {
  pdl_wait();
  pdl_trigger();
  constexpr int kRowsPerWarp = RPW, kSimtRows = RPW * kSimtWarps;
  constexpr float kUnit = X ? kLog2e : 1.0f;  // scores with a form stay as they are, the others are in log2 units
  extern __shared__ float smem[];
  const sv_attention_args& a = P.a;
  const int D = a.cache.head_dim, DP = D + 4, H = a.cache.heads, G = a.Hq / H;
  float* sK = smem;                  // [32][DP]
  float* sV = sK + kSimtKeys * DP;   // [32][DP]
  float* sQ = sV + kSimtKeys * DP;   // [16][DP]
  __shared__ int s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = (a.R * G + kSimtRows - 1) / kSimtRows;
  const int item = blockIdx.x, rb = item % blocks, h = item / blocks % H, b = item / blocks / H;
  const int split = blockIdx.y;
  const Extent E = extent_of(a, b, P.err);
  const int row0 = rb * kSimtRows;
  const int64_t q0 = b * a.q_stride[0], o0 = b * a.out_stride[0];
  // rows of this block that are past the request's entries are zero
  if (split == 0)
    for (int c = threadIdx.x; c < kSimtRows * (D / 8); c += kSimtThreads) {
      const int r = row0 + c / (D / 8), i = r / G;
      const float zero[8] = {};
      if (i < a.R && i > E.n)
        store8<F32>(a.out, o0 + i * a.out_stride[1] + (h * G + r % G) * a.out_stride[2] + c % (D / 8) * 8, zero);
    }
  if (row0 / G > E.n) return;
  const int begin = X ? first_seen(a, E.S) : 0;
  const int keys = E.S + E.n + 1, tiles = (keys - begin + kSimtKeys - 1) / kSimtKeys;
  const int per = (tiles + P.splits - 1) / P.splits;
  const int t0 = split * per, t1 = min(tiles, t0 + per);
  const int used = (tiles + per - 1) / per;  // shares with work
  if (split >= used) return;
  const int64_t cstep = row_step(a.cache), sstep = a.stage.data ? row_step(a.stage) : 0;
  for (int c = threadIdx.x; c < kSimtRows * (D / 8); c += kSimtThreads) {
    const int r = row0 + c / (D / 8), i = r / G, d = c % (D / 8) * 8;
    float x[8] = {};
    if (i <= E.n) load8<F32>(a.q, q0 + i * a.q_stride[1] + (h * G + r % G) * a.q_stride[2] + d, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) sQ[c / (D / 8) * DP + d + e] = x[e] * (X ? a.scale : a.scale * kLog2e);
  }
  float m[kRowsPerWarp], l[kRowsPerWarp], o[kRowsPerWarp][kMaxHeadDim / 32];
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    m[r] = -__int_as_float(0x7F800000), l[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < kMaxHeadDim / 32; ++e) o[r][e] = 0.0f;
  }
  const float* q = sQ + warp * kRowsPerWarp * DP;
  for (int t = t0; t < t1; ++t) {
    const int x0 = begin + t * kSimtKeys;
    __syncthreads();
    constexpr int kAt = 2;  // vectors of K and of V on their way
    for (int c0 = threadIdx.x; c0 < kSimtKeys * (D / 8); c0 += kAt * kSimtThreads) {
      float k[kAt][8], v[kAt][8];
#pragma unroll
      for (int u = 0; u < kAt; ++u) {
        const int c = c0 + u * kSimtThreads, j = c / (D / 8), d = c % (D / 8) * 8, x = x0 + j;
#pragma unroll
        for (int e = 0; e < 8; ++e) k[u][e] = v[u][e] = 0.0f;
        if (j >= kSimtKeys || x >= keys) continue;
        const bool staged = a.stage.data && x >= E.S;
        const sv_kv_place& pl = staged ? a.stage : a.cache;
        const int64_t off = entry_offset(pl, b, x - E.S, x);
        if (off >= 0) {
          const int64_t step = staged ? sstep : cstep;
          const char* kr = static_cast<const char*>(pl.data) + off + h * step;
          const char* vr = kr + H * step;
          load_entry8(kr, pl.format, d, entry_scale(kr, pl.format, D), k[u]);
          load_entry8(vr, pl.format, d, entry_scale(vr, pl.format, D), v[u]);
        } else if (d == 0) {
          report(P.err, SV_ERR_STATE);
        }
      }
#pragma unroll
      for (int u = 0; u < kAt; ++u) {
        const int c = c0 + u * kSimtThreads, j = c / (D / 8), d = c % (D / 8) * 8;
        if (j >= kSimtKeys) continue;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          *reinterpret_cast<float4*>(&sK[j * DP + d + e]) = make_float4(k[u][e], k[u][e + 1], k[u][e + 2], k[u][e + 3]);
          *reinterpret_cast<float4*>(&sV[j * DP + d + e]) = make_float4(v[u][e], v[u][e + 1], v[u][e + 2], v[u][e + 3]);
        }
      }
    }
    __syncthreads();
    float s[kRowsPerWarp] = {};
    for (int d = 0; d < D; d += 4) {
      const float4 k = *reinterpret_cast<const float4*>(&sK[lane * DP + d]);
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) {
        const float4 v = *reinterpret_cast<const float4*>(&q[r * DP + d]);
        s[r] += v.x * k.x, s[r] += v.y * k.y, s[r] += v.z * k.z, s[r] += v.w * k.w;
      }
    }
    float p[kRowsPerWarp];
    // where this lane's key is, past S
    const int at = !X || x0 + lane < E.S || x0 + lane >= keys ? x0 + lane - E.S : depth_of(a, b, x0 + lane - E.S);
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      const int i = (row0 + warp * kRowsPerWarp + r) / G;
      const uint32_t bits = i > E.n ? 0u : seen_bits(a, b, i, E.n, x0 - E.S);
      bool see = bits >> lane & 1;
      if (X) {
        const int hq = h * G + (row0 + warp * kRowsPerWarp + r) % G, far = i > E.n ? 0 : abs(depth_of(a, b, i) - at);
        if (a.softcap > 0.0f) s[r] = a.softcap * tanhf(s[r] / a.softcap);
        if (a.slopes) s[r] -= a.slopes[hq] * (float)far;
        if (a.window > 0 && far >= a.window) see = false;
      }
      // a key that is not seen takes no part, whatever its score is; a NaN
      // score that is seen stays NaN through the sums
      float mx = see ? s[r] : -__int_as_float(0x7F800000);
#pragma unroll
      for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, w));
      const float mn = fmaxf(m[r], mx);
      const float base = mn == -__int_as_float(0x7F800000) ? 0.0f : mn;
      p[r] = see ? exp2f((s[r] - base) * kUnit) : 0.0f;
      const float alpha = exp2f((m[r] - base) * kUnit);
      m[r] = mn;
      l[r] = l[r] * alpha + p[r];  // a lane's share of the sum
#pragma unroll
      for (int e = 0; e < kMaxHeadDim / 32; ++e) o[r][e] *= alpha;
      p[r] = see ? p[r] : -1.0f;  // marks what is not seen
    }
#pragma unroll 4
    for (int j = 0; j < kSimtKeys; ++j) {
      float w[kRowsPerWarp];
#pragma unroll
      for (int r = 0; r < kRowsPerWarp; ++r) w[r] = __shfl_sync(0xFFFFFFFFu, p[r], j);
#pragma unroll
      for (int c = 0; c < kMaxHeadDim / 128; ++c) {
        if (c * 128 + lane * 4 >= D) continue;
        const float4 v = *reinterpret_cast<const float4*>(&sV[j * DP + c * 128 + lane * 4]);
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) {
          if (w[r] != -1.0f) {  // seen
            o[r][4 * c] += w[r] * v.x, o[r][4 * c + 1] += w[r] * v.y;
            o[r][4 * c + 2] += w[r] * v.z, o[r][4 * c + 3] += w[r] * v.w;
          }
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r)
#pragma unroll
    for (int w = 16; w; w >>= 1) l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], w);
  // partial results: [item][split][row][2 + D]
  const int stride = D + 4;
  auto slot = [&](int s, int r) {
    return P.part + (((int64_t)item * P.splits + s) * kSimtRows + warp * kRowsPerWarp + r) * stride;
  };
  if (used > 1) {
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      float* w = slot(split, r);
      if (lane == 0) w[D] = m[r], w[D + 1] = l[r];
#pragma unroll
      for (int c = 0; c < kMaxHeadDim / 128; ++c)
        if (c * 128 + lane * 4 < D)
          *reinterpret_cast<float4*>(w + c * 128 + lane * 4) =
              make_float4(o[r][4 * c], o[r][4 * c + 1], o[r][4 * c + 2], o[r][4 * c + 3]);
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      s_last = atomicAdd(&P.ticket[item], 1u) == (uint32_t)used - 1;
      if (s_last) P.ticket[item] = 0;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
      float mm = -__int_as_float(0x7F800000);
      for (int s = 0; s < used; ++s) mm = fmaxf(mm, __ldcg(slot(s, r) + D));
      const float base = mm == -__int_as_float(0x7F800000) ? 0.0f : mm;
      l[r] = 0.0f;
#pragma unroll
      for (int e = 0; e < kMaxHeadDim / 32; ++e) o[r][e] = 0.0f;
      for (int s = 0; s < used; ++s) {
        const float* w = slot(s, r);
        const float f = exp2f((__ldcg(w + D) - base) * kUnit);
        l[r] += f * __ldcg(w + D + 1);
#pragma unroll
        for (int c = 0; c < kMaxHeadDim / 128; ++c)
          if (c * 128 + lane * 4 < D) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(w + c * 128 + lane * 4));
            o[r][4 * c] += f * v.x, o[r][4 * c + 1] += f * v.y;
            o[r][4 * c + 2] += f * v.z, o[r][4 * c + 3] += f * v.w;
          }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsPerWarp; ++r) {
    const int row = row0 + warp * kRowsPerWarp + r, i = row / G;
    if (i > E.n) continue;
    const float inv = l[r] == 0.0f ? 0.0f : 1.0f / l[r];
    const int64_t at = o0 + i * a.out_stride[1] + (h * G + row % G) * a.out_stride[2];
#pragma unroll
    for (int c = 0; c < kMaxHeadDim / 128; ++c) {
      const int d = c * 128 + lane * 4;
      if (d >= D) continue;
      const float y[4] = {o[r][4 * c] * inv, o[r][4 * c + 1] * inv, o[r][4 * c + 2] * inv, o[r][4 * c + 3] * inv};
      if (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + d) = make_float4(y[0], y[1], y[2], y[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at + d) =
            make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    }
  }
}

// Tickets sit at the workspace's start whatever the shape, so that a call never
// finds another shape's partial results in them.  Few are ever in use: only
// items that are shared by CTAs have one, and there are fewer of them than
// CTAs that fill the GPU twice.
constexpr int kTickets = 1024;
constexpr size_t kTicketBytes = kTickets * 4;
static_assert(kTicketBytes == SV_ATTENTION_CLEAR, "the tickets are all that a call reads before it wrote it");

// Shares of the keys: enough CTAs to fill the GPU twice, none below 64 keys.
static int simt_splits(const sv_handle* h, const sv_attention_args* a, int64_t items) {
  const int64_t keys = (int64_t)a->cache.max_blocks * a->cache.block_size + a->R;
  int64_t s = (2 * (int64_t)h->num_sms + items - 1) / (items > 0 ? items : 1);
  const int64_t most = (keys + 63) / 64;
  if (s > most) s = most;
  if (items > kTickets) s = 1;
  return s < 1 ? 1 : s > 64 ? 64 : (int)s;
}

// Rows of a CTA: 4, 8 or 16.
static int simt_rows(const sv_attention_args* a) {
  const int64_t rows = (int64_t)a->R * (a->Hq / a->cache.heads);
  return rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
}

static int64_t simt_items(const sv_attention_args* a) {
  const int64_t rows = (int64_t)a->R * (a->Hq / a->cache.heads);
  return (int64_t)a->B * a->cache.heads * ((rows + simt_rows(a) - 1) / simt_rows(a));
}

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// ---------------------------------------------------------------------------
// The tensor kernel's host side
// ---------------------------------------------------------------------------
static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct TcPlan {
  bool use;
  bool sharing;  // requests of a group share items
  int tiles, ctas;  // row tiles per CTA, grid
  TcKernel k;
  size_t list, ranges, bytes;  // where the list and the ranges start in the workspace, and its bytes
};

static bool has_form(const sv_attention_args* a) { return a->softcap > 0.0f || a->slopes || a->window > 0; }

// Whether a call looks at its groups.  Two requests at least have to fit an item's 128 rows: where
// each has one of its own the prefix is read for each all the same, by smaller boxes, and with a form a
// prompt's hidden tiles are gone through.  16 groups of four trees of 15 nodes, 8 query heads a KV head,
// over 8192 positions 337 us without groups and 350 so (8-bit 428 and 474), four capped prompts of
// 1024 entries 257 and 295; 64 rows 322 and 196.  Prompts without a form are listed all the same
// where their entries are a good part of their keys, since the list has a warp of its own for clearing V:
// four of 1024 entries over 1024 positions 292 us without groups and 198 so (8-bit 339 and 286), 400
// entries 169 and 111, but 200 of one head a KV head 54 and 58 in 8 bits, and 400 over 8192 468 and 482.
static bool looks_at_groups(const sv_attention_args* a, int64_t rows) {
  if (!a->shared_len || a->window > 0) return false;
  if (2 * rows <= kTile) return true;
  return !has_form(a) && a->R > 2 * kTile && 5 * (int64_t)a->R >= (int64_t)a->cache.max_blocks * a->cache.block_size;
}

// bf16 and 8-bit caches with heads of 64 or 128 and blocks of whole 8-row
// groups (the swizzle's unit, so that a TMA box can start at any block) run on
// the tensor cores, from one row up: padding 4 rows to 128 costs no bytes, and
// bytes bound them.
static TcPlan tc_plan(const sv_handle* h, const sv_attention_args* a) {
  TcPlan p = {};
  const sv_kv_place& c = a->cache;
  if (a->dtype != SV_BF16 || (c.head_dim != 64 && c.head_dim != 128) || c.block_size % 8 || c.num_blocks < 1)
    return p;
  const int64_t rows = (int64_t)a->R * (a->Hq / c.heads);
  const bool forms = has_form(a);
  // a group's rows are its members' R entries each, and it has no more items than they
  p.sharing = looks_at_groups(a, rows);
  p.tiles = rows > kTile ? 2 : 1;
  const int64_t blocks = cdiv(rows, p.tiles * kTile);
  const int64_t tiles = (int64_t)a->B * c.heads * blocks * (cdiv((int64_t)c.max_blocks * c.block_size, kTile) + cdiv(a->R, kTile) + 1 + kLead);
  if (tiles > INT32_MAX || (rows + 2 * kTile) * (a->Hq / c.heads) > INT32_MAX || c.num_blocks == INT32_MAX) return p;
  p.use = true;
  typedef TcKernel (*Of)(int, int);
  static const Of of[2][4] = {{tc_kernel_bf16, tc_kernel_bf16_forms, tc_kernel_bf16_shared, tc_kernel_bf16_both},
                              {tc_kernel_e4m3, tc_kernel_e4m3_forms, tc_kernel_e4m3_shared, tc_kernel_e4m3_both}};
  p.ctas = (int)(tiles < h->num_sms ? tiles : h->num_sms);
  if (p.ctas > kTickets) p.ctas = kTickets;
  p.k = of[c.format == SV_KV_E4M3][(forms ? kForms : 0) + (p.sharing ? kShare : 0)](c.head_dim, p.tiles);
  p.list = p.bytes = kTicketBytes + up256((size_t)p.ctas * 2 * p.k.part * 4);
  if (forms || p.sharing) {
    p.ranges = p.bytes += 256 + up256((size_t)p.ctas * 4) + up256((size_t)a->B * sizeof(TcLot));
    if (forms && !p.sharing && blocks > 1) p.bytes += up256((size_t)a->B * (2 * (size_t)blocks + 1) * 4);
  }
  return p;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// A place's rows; rows of an 8-bit entry without their tails, which have a map
// of their own, {byte, slot or entry, head, (layer, K or V), block or request},
// and come for K and V at once.
struct Rows {
  int64_t n, step, other, outer, step_outer;  // of the second and the last dimension, and from row to row of a layer
};
static bool make_maps(CUtensorMap* m, CUtensorMap* tails, const sv_kv_place& pl, const Rows& r, int box_rows) {
  const bool f8 = pl.format == SV_KV_E4M3;
  const int row = f8 ? pl.head_dim : 2 * pl.head_dim, sw = row < 128 ? row : 128;
  const cuuint64_t D = (cuuint64_t)pl.head_dim, n = (cuuint64_t)r.n, H = (cuuint64_t)pl.heads, L2 = (cuuint64_t)pl.layers * 2,
                   outer = (cuuint64_t)r.outer;
  const cuuint64_t step = (cuuint64_t)r.step, other = (cuuint64_t)r.other, step_outer = (cuuint64_t)r.step_outer;
  const cuuint32_t rows = (cuuint32_t)box_rows, one[5] = {1, 1, 1, 1, 1};
  if (f8) {
    const cuuint64_t dims[5] = {kTail, n, H, L2, outer}, strides[4] = {step, other, other * H, step_outer};
    const cuuint32_t box[5] = {kTail, rows, 1, 2, 1};
    if (encode_tiled()(tails, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, static_cast<char*>(pl.data) + row, dims, strides, box, one,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  // a bf16 row of 128 comes as two halves: the first brings all of it into L2 (64
  // single tokens 192.4 us without, 189.4 so; 64 trees over 8192 positions 359 and 354)
  const cuuint64_t dims[4] = {D, n, L2 * H, outer}, strides[3] = {step, other, step_outer};
  const cuuint32_t box[4] = {(cuuint32_t)(f8 ? sw : sw / 2), rows, 1, 1};
  return encode_tiled()(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pl.data, dims,
                        strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        sw == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static sv_status tc_launch(sv_handle* h, const sv_attention_args* a, const TcPlan& plan, void* ws, cudaStream_t stream) {
  if (!encode_tiled()) return SV_ERR_CUDA;
  TcParams P = {};
  P.p.a = *a;
  P.p.ticket = static_cast<uint32_t*>(ws);
  P.p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kTicketBytes);
  P.p.err = h->d_err;
  const sv_kv_place& c = a->cache;
  P.box = 8;
  while (P.box < (plan.sharing ? kStageBox : kTile) && c.block_size % (2 * P.box) == 0) P.box *= 2;
  P.stage_box = plan.sharing ? P.box : kStageBox;
  P.block_shift = -1;
  for (int s = 3; s < 31; ++s)
    if (c.block_size == 1 << s) P.block_shift = s;
  const uint32_t G = (uint32_t)(a->Hq / c.heads);
  P.group = (int)G;
  P.group_magic = G == 1 ? 0u : (uint32_t)((0x100000000ull + G - 1) / G);
  const int64_t row = row_bytes(c), per = row * 2 * c.heads;  // bytes of a row, and of an entry's layer
  if (!make_maps(&P.pages, &P.page_tails, c,
                 {c.block_size, row, row * c.block_size, c.num_blocks, per * c.layers * c.block_size}, P.box))
    return SV_ERR_CUDA;
  const sv_kv_place& g = a->stage;
  if (g.data && !make_maps(&P.stage, &P.stage_tails, g, {g.rows, per * g.layers, row, a->B, per * g.layers * g.rows}, P.stage_box))
    return SV_ERR_CUDA;
  const bool forms = has_form(a), listed = forms || plan.sharing;
  TcPlanning L = {};
  if (listed) {
    char* at = static_cast<char*>(ws);
    P.entries_magic = a->R == 1 ? 0u : (uint32_t)((0x100000000ull + a->R - 1) / a->R);
    while (P.box >> (P.box_shift + 1)) ++P.box_shift;
    P.down = a->slopes != nullptr;
    L.a = *a, L.rows = plan.tiles * kTile, L.lead = plan.tiles == 2 ? kLeadWide : kLead, L.box = P.box, L.shift = P.box_shift, L.group = P.group, L.ctas = plan.ctas;
    L.sharing = plan.sharing, L.err = h->d_err;
    L.head = reinterpret_cast<int*>(at + plan.list), L.first = reinterpret_cast<int*>(at + plan.list + 256);
    L.lots = reinterpret_cast<TcLot*>(at + plan.list + 256 + up256((size_t)plan.ctas * 4));
    if (plan.bytes > plan.ranges) {
      L.ranges = reinterpret_cast<int*>(at + plan.ranges);
      L.words = 2 * (int)cdiv((int64_t)a->R * P.group, L.rows) + 1;
    }
    const sv_status rp = plan_launch(L, stream);
    if (rp != SV_OK) return rp;
  }
  P.list = {L.lots, L.head, L.first, L.ranges, L.words, L.lead};
  const sv_status rr = sv_raise_dyn_smem((const void*)plan.k.fn, (size_t)plan.k.smem);
  if (rr != SV_OK) return rr;
  if (sv_launch_pdl(plan.k.fn, dim3((unsigned)plan.ctas), dim3((unsigned)plan.k.threads), (size_t)plan.k.smem, stream, P) != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return SV_OK;
}

static sv_status simt_launch(sv_handle* h, const sv_attention_args* a, void* ws, cudaStream_t stream) {
  const int64_t items = simt_items(a);
  AttnParams P = {};
  P.a = *a;
  P.ticket = static_cast<uint32_t*>(ws);
  P.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kTicketBytes);
  P.err = h->d_err;
  P.splits = simt_splits(h, a, items);
  const size_t smem = (size_t)(2 * kSimtKeys + simt_rows(a)) * (a->cache.head_dim + 4) * 4;
  typedef void (*Fn)(AttnParams);
#define SV_SIMT(x) {{simt_attention_kernel<false, 1, x>, simt_attention_kernel<false, 2, x>, simt_attention_kernel<false, 4, x>}, \
                    {simt_attention_kernel<true, 1, x>, simt_attention_kernel<true, 2, x>, simt_attention_kernel<true, 4, x>}}
  static const Fn fns[2][2][3] = {SV_SIMT(false), SV_SIMT(true)};
#undef SV_SIMT
  const Fn fn = fns[has_form(a)][a->dtype == SV_FP32][simt_rows(a) / 8];
  const sv_status rr = sv_raise_dyn_smem((const void*)fn, smem);
  if (rr != SV_OK) return rr;
  if (sv_launch_pdl(fn, dim3((unsigned)items, (unsigned)P.splits), dim3(kSimtThreads), smem, stream, P) != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return SV_OK;
}

}  // namespace sv

using namespace sv;

static sv_status check(const sv_handle* h, const sv_attention_args* a) {
  if (!h || !a || a->B < 0 || a->R < 1 || a->Hq < 1 || (a->dtype != SV_BF16 && a->dtype != SV_FP32)) return SV_ERR_INVALID;
  if (a->B == 0) return SV_OK;
  const int eb = a->dtype == SV_BF16 ? 2 : 4;
  if (bad_place(&a->cache) || !a->cache.block_table || a->Hq % a->cache.heads || !a->seq_len) return SV_ERR_INVALID;
  if ((int64_t)a->cache.max_blocks * a->cache.block_size + a->R > INT32_MAX) return SV_ERR_INVALID;
  if (bad_strides(a->q, a->q_stride, eb) || bad_strides(a->out, a->out_stride, eb)) return SV_ERR_INVALID;
  if (a->stage.data &&
      (bad_place(&a->stage) || a->stage.block_table || a->stage.rows < a->R || a->stage.heads != a->cache.heads ||
       a->stage.head_dim != a->cache.head_dim || a->stage.format != a->cache.format))
    return SV_ERR_INVALID;
  if (a->mask && a->mask_ld < (a->R + 31) / 32) return SV_ERR_INVALID;
  if (!(a->scale == a->scale)) return SV_ERR_INVALID;
  if (!(a->softcap == 0.0f || (a->softcap >= 0x1p-60f && a->softcap <= 0x1p60f)) || a->window < 0) return SV_ERR_INVALID;
  if (!a->shared_len != !a->shared_members) return SV_ERR_INVALID;
  if ((a->dtype == SV_FP32) != (a->cache.format == SV_KV_FP32)) return SV_ERR_UNSUPPORTED;
  if (simt_items(a) > INT32_MAX) return SV_ERR_UNSUPPORTED;
  return SV_OK;
}

extern "C" size_t sv_attention_args_size(void) { return sizeof(sv_attention_args); }

extern "C" sv_status sv_attention_workspace_size(sv_handle* h, const sv_attention_args* a, size_t* bytes) {
  if (!bytes) return SV_ERR_INVALID;
  const sv_status rs = check(h, a);
  if (rs != SV_OK) return rs;
  *bytes = 256;
  if (a->B == 0) return SV_OK;
  const TcPlan plan = tc_plan(h, a);
  if (plan.use) {
    *bytes = plan.bytes;
    return SV_OK;
  }
  const int64_t items = simt_items(a);
  const int splits = simt_splits(h, a, items);
  *bytes = kTicketBytes + up256((size_t)items * splits * simt_rows(a) * (a->cache.head_dim + 4) * 4);
  return SV_OK;
}

extern "C" sv_status sv_tree_attention(sv_handle* h, const sv_attention_args* a, void* ws, size_t ws_bytes,
                                       sv_stream_t stream) {
  size_t need = 0;
  const sv_status rs = sv_attention_workspace_size(h, a, &need);
  if (rs != SV_OK) return rs;
  if (a->B == 0) return SV_OK;
  if (!ws || ((uintptr_t)ws & 255u) || ws_bytes < need) return SV_ERR_INVALID;
  const TcPlan plan = tc_plan(h, a);
  return plan.use ? tc_launch(h, a, plan, ws, (cudaStream_t)stream) : simt_launch(h, a, ws, (cudaStream_t)stream);
}
