// The entries of a verify pass: rotary positions, formats, write and read back.
#include "entries.cuh"

namespace sv {

// 8164 entries of 32 + 2 x 8 heads of 128, 8-bit (186 MB): written in 52 us by
// 256 threads, 38 by 128, 37 by 64; 960 entries 6.1, 5.9 and 6.2 us: what a
// thread does before its first row is shared by more rows.  (39.6, 4.7 TB/s, and
// 5.8 since columns past the rotated ones are left alone; bf16 38.8, 5.2 TB/s,
// fp32 65.4, 6.1.)
constexpr int kAppendThreads = 128;

// Lanes of a warp that share a row of head_dim values, eight values a lane;
// rows never straddle warps, so in-place rotation and the row maximum need
// warp-level exchange only.
struct RowLanes {
  int cpr, rpw, c, slot, nslots;
  bool on;
  uint32_t group;  // lanes of this row
  __device__ __forceinline__ RowLanes(int head_dim) {
    const int lane = threadIdx.x & 31;
    cpr = head_dim >> 3;
    rpw = 32 / cpr;
    const int r = lane / cpr;
    c = lane - r * cpr;
    on = r < rpw;
    slot = (threadIdx.x >> 5) * rpw + r;
    nslots = (blockDim.x >> 5) * rpw;
    group = (cpr == 32 ? 0xFFFFFFFFu : ((1u << cpr) - 1u)) << (on ? r * cpr : 0);
  }
};

struct AppendParams {
  sv_append_args a;
  int* err;
};

// Eight values as they are stored.
template <bool F32>
struct Raw8 {
  uint4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> raw8(const char* p) {
  Raw8<F32> r;
  r.w[0] = reinterpret_cast<const uint4*>(p)[0];
  if (F32) r.w[F32 ? 1 : 0] = reinterpret_cast<const uint4*>(p)[1];
  return r;
}
template <bool F32>
__device__ __forceinline__ void values8(const Raw8<F32>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
  if (F32) {
    const uint4 h = r.w[F32 ? 1 : 0];
    const uint32_t v[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(w[e]), x[4 + e] = __uint_as_float(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[2 * e] = __uint_as_float(w[e] << 16), x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

// How the other half of a rotary pair is reached: not at all, in the same eight
// columns (neighbours), in another lane's (halves that are whole lanes), or in
// memory (halves that end inside a lane's columns).
enum Turn { kNone, kPairs, kLanes, kMemory };

// x' = x cos + other * sin in the first `turned` of the eight columns, with the
// sign of the pair's half in sin; the others stay as they are, whatever they and
// their neighbours hold.
template <bool F32, int TURN>
__device__ __forceinline__ void turn8(float (&x)[8], const Raw8<F32>& now, const char* row, int d0, int half, int turned, int other, uint32_t group,
                                      const float (&co)[8], const float (&si)[8]) {
  if (TURN == kNone) return;
  float o[8];
  if (TURN == kPairs) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = x[e ^ 1];
  } else if (TURN == kLanes) {
    Raw8<F32> t;
#pragma unroll
    for (int k = 0; k < (F32 ? 2 : 1); ++k)
      t.w[k] = make_uint4(__shfl_sync(group, now.w[k].x, other), __shfl_sync(group, now.w[k].y, other),
                          __shfl_sync(group, now.w[k].z, other), __shfl_sync(group, now.w[k].w, other));
    values8<F32>(t, o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = d0 + e, q = d < half ? d + half : d < 2 * half ? d - half : d;
      o[e] = F32 ? reinterpret_cast<const float*>(row)[q] : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[q]);
    }
    __syncwarp(group);  // queries may be rotated in place: every lane has its operands
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (TURN == kLanes ? 0 : e) < turned ? x[e] * co[e] + o[e] * si[e] : x[e];
}

// One CTA per (request, entry): its queries, keys and values are rows of
// head_dim, and a thread has the same eight columns of all its rows, with their
// cos / sin in registers.  Each value is read and written once, the table's row
// once per entry; instructions bound it as much as bytes do, so what differs
// between calls is settled at compile time and rows are reached by one stride.
// A row does not depend on where its entry goes: a thread's first three are on
// their way before the entry's length, block and position are known.
template <bool F32, int TURN>
__global__ void __launch_bounds__(kAppendThreads, 8) kv_append_kernel(const __grid_constant__ AppendParams P) {
  pdl_wait();
  pdl_trigger();
  const sv_append_args& a = P.a;
  const sv_kv_place& dst = a.dst;
  constexpr int eb = F32 ? 4 : 2;
  const int b = blockIdx.x / a.R, i = blockIdx.x - b * a.R;
  const RowLanes L(dst.head_dim);
  const int Hq = a.q ? a.Hq : 0, H = dst.heads, d0 = 8 * L.c;
  auto base = [&](const void* p, const int64_t* st) { return static_cast<const char*>(p) + (b * st[0] + i * st[1]) * eb; };
  const char *q = base(a.q, a.q_stride), *k = base(a.k, a.k_stride), *v = base(a.v, a.v_stride);
  const int64_t qs = a.q_stride[2] * eb, ks = a.k_stride[2] * eb, vs = a.v_stride[2] * eb;
  auto kv_row = [&](int r) { return r < H ? k + r * ks : v + (r - H) * vs; };
  Raw8<F32> q0, q1, kv0;
  if (L.on) {
    if (L.slot < Hq) q0 = raw8<F32>(q + L.slot * qs + d0 * eb);
    if (L.slot + L.nslots < Hq) q1 = raw8<F32>(q + (L.slot + L.nslots) * qs + d0 * eb);
    if (L.slot < 2 * H) kv0 = raw8<F32>(kv_row(L.slot) + d0 * eb);
  }
  int n = a.n_nodes ? a.n_nodes[b] : a.R - 1;
  if (n >= a.R) {
    if (threadIdx.x == 0 && i == 0) report(P.err, SV_ERR_STATE);
    n = a.R - 1;
  }
  const int64_t S = a.seq_len[b];
  bool live = i <= n;
  int64_t off = -1, pos = 0;
  if (live) {
    if (TURN != kNone) pos = S + (a.depth ? a.depth[(int64_t)b * a.R + i] : i);
    off = entry_offset(dst, b, i, S + i);
    live = off >= 0 && (TURN == kNone || (pos >= 0 && pos < a.max_pos));
    if (!live && threadIdx.x == 0) report(P.err, SV_ERR_STATE);
  }
  if (!L.on) return;
  char* out = static_cast<char*>(a.q_out) + (b * a.q_out_stride[0] + i * a.q_out_stride[1] + d0) * eb;
  const int64_t os = a.q_out_stride[2] * eb;
  if (!live) {
    const float zero[8] = {};
    for (int h = L.slot; h < Hq; h += L.nslots) store8<F32>(out + h * os, 0, zero);
    return;
  }
  const int half = a.rot_dim >> 1, turned = a.rot_dim - d0;
  const int other = TURN == kLanes && d0 < a.rot_dim ? (threadIdx.x & 31) + (d0 < half ? half >> 3 : -(half >> 3)) : threadIdx.x & 31;
  float co[8], si[8];
  if (TURN != kNone) {
    const float2* cs = reinterpret_cast<const float2*>(a.rope + pos * a.rot_dim);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = d0 + e;
      co[e] = si[e] = 0.0f;
      if (d < a.rot_dim) {
        const float2 t = cs[TURN == kPairs ? d >> 1 : d < half ? d : d - half];
        co[e] = t.x, si[e] = (TURN == kPairs ? !(d & 1) : d < half) ? -t.y : t.y;
      }
    }
  }
#pragma unroll 1
  for (int h = L.slot; h < Hq; h += 2 * L.nslots) {
    if (h != L.slot) {
      q0 = raw8<F32>(q + h * qs + d0 * eb);
      if (h + L.nslots < Hq) q1 = raw8<F32>(q + (h + L.nslots) * qs + d0 * eb);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int hu = h + u * L.nslots;
      if (hu >= Hq) break;
      float x[8];
      const Raw8<F32>& now = u ? q1 : q0;
      values8<F32>(now, x);
      turn8<F32, TURN>(x, now, q + hu * qs, d0, half, turned, other, L.group, co, si);
      store8<F32>(out + hu * os, 0, x);
    }
  }
  const int64_t step = row_step(dst);
#pragma unroll 1
  for (int r = L.slot; r < 2 * H; r += L.nslots) {
    if (r != L.slot) kv0 = raw8<F32>(kv_row(r) + d0 * eb);
    float x[8];
    values8<F32>(kv0, x);
    if (r < H) turn8<F32, TURN>(x, kv0, kv_row(r), d0, half, turned, other, L.group, co, si);
    char* row = static_cast<char*>(dst.data) + off + r * step;
    if (dst.format == SV_KV_FP32) {
      store8<true>(row, d0, x);
    } else if (dst.format == SV_KV_BF16) {
      store8<false>(row, d0, x);
    } else {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));  // NaN is left out
      const float scale = e4m3_scale(__uint_as_float(__reduce_max_sync(L.group, __float_as_uint(m))), r < H ? 1.0f : kLeastScale);
      const float inv = __uint_as_float(0x7F000000u - __float_as_uint(scale));  // scales are 2^-126 .. 2^120
      uint32_t w[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * g] * inv, x[4 * g + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * g + 2] * inv, x[4 * g + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        w[g] = lo | hi << 16;
      }
      *reinterpret_cast<uint2*>(row + d0) = make_uint2(w[0], w[1]);
      if (L.c == 0) *reinterpret_cast<uint4*>(row + dst.head_dim) = make_uint4(__float_as_uint(scale), 0, 0, 0);
    }
  }
}

// One CTA per (request, entry), kReadRows rows of a thread under way at once;
// bytes bound it.  8164 entries of 2 x 8 rows of 128, 8-bit to bf16 (52 MB),
// with 256 threads for four entries 15.4 us, 64 for one and one row at a time
// 9.3, two rows 9.6 (5.4 TB/s), four 10.0; 960 entries 3.3, 3.0, 2.8 and 2.7 us.
constexpr int kReadThreads = 64, kReadRows = 2;

template <bool F32>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(int R, const int32_t* seq_len, const int32_t* n_nodes,
                                                               const __grid_constant__ sv_kv_place src, void* out, int* err) {
  pdl_wait();
  pdl_trigger();
  const RowLanes L(src.head_dim);
  const int64_t step = row_step(src);
  const int b = blockIdx.x / R, i = blockIdx.x - b * R, rows = 2 * src.heads;
  int n = n_nodes ? n_nodes[b] : R - 1;
  if (n >= R) {
    if (threadIdx.x == 0 && i == 0) report(err, SV_ERR_STATE);
    n = R - 1;
  }
  int64_t off = -1;
  if (i <= n) {
    off = entry_offset(src, b, i, (int64_t)seq_len[b] + i);
    if (off < 0 && threadIdx.x == 0) report(err, SV_ERR_STATE);
  }
  if (!L.on) return;
  for (int r0 = L.slot; r0 < rows; r0 += kReadRows * L.nslots) {
    float x[kReadRows][8] = {};
#pragma unroll
    for (int u = 0; u < kReadRows; ++u) {
      const int r = r0 + u * L.nslots;
      if (off < 0 || r >= rows) continue;
      const char* row = static_cast<const char*>(src.data) + off + r * step;
      load_entry8(row, src.format, 8 * L.c, entry_scale(row, src.format, src.head_dim), x[u]);
    }
#pragma unroll
    for (int u = 0; u < kReadRows; ++u) {
      const int r = r0 + u * L.nslots;
      if (r < rows) store8<F32>(out, ((int64_t)blockIdx.x * rows + r) * src.head_dim + 8 * L.c, x[u]);
    }
  }
}

}  // namespace sv

using namespace sv;

extern "C" size_t sv_append_args_size(void) { return sizeof(sv_append_args); }

extern "C" sv_status kv_append(sv_handle* h, const sv_append_args* a, sv_stream_t stream) {
  if (!h || !a || a->B < 0 || a->R < 1 || (a->dtype != SV_BF16 && a->dtype != SV_FP32)) return SV_ERR_INVALID;
  if (a->B == 0) return SV_OK;
  const int eb = a->dtype == SV_BF16 ? 2 : 4;
  if (bad_place(&a->dst) || !a->seq_len || (int64_t)a->B * a->R > INT32_MAX) return SV_ERR_INVALID;
  if (!a->dst.block_table && a->dst.rows < a->R) return SV_ERR_INVALID;
  if (bad_strides(a->k, a->k_stride, eb) || bad_strides(a->v, a->v_stride, eb)) return SV_ERR_INVALID;
  if (a->q && (a->Hq < 1 || bad_strides(a->q, a->q_stride, eb) || bad_strides(a->q_out, a->q_out_stride, eb)))
    return SV_ERR_INVALID;
  if (a->rope && (a->rot_dim < 2 || a->rot_dim % 2 || a->rot_dim > a->dst.head_dim || a->max_pos < 0 ||
                  ((uintptr_t)a->rope & 7u)))
    return SV_ERR_INVALID;
  const AppendParams P = {*a, h->d_err};
  const int turn = !a->rope ? kNone : (a->flags & SV_APPEND_PAIRS) ? kPairs : a->rot_dim % 16 == 0 ? kLanes : kMemory;
  typedef void (*Fn)(AppendParams);
  static const Fn fns[2][4] = {
      {kv_append_kernel<false, kNone>, kv_append_kernel<false, kPairs>, kv_append_kernel<false, kLanes>, kv_append_kernel<false, kMemory>},
      {kv_append_kernel<true, kNone>, kv_append_kernel<true, kPairs>, kv_append_kernel<true, kLanes>, kv_append_kernel<true, kMemory>}};
  const cudaError_t e = sv_launch_pdl(fns[a->dtype == SV_FP32][turn], dim3((unsigned)(a->B * a->R)), dim3(kAppendThreads), 0,
                                      (cudaStream_t)stream, P);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return SV_OK;
}

extern "C" sv_status kv_read(sv_handle* h, int32_t B, int32_t R, const int32_t* seq_len,
                             const int32_t* n_nodes, const sv_kv_place* src, void* out,
                             int32_t out_dtype, sv_stream_t stream) {
  if (!h || B < 0 || R < 1 || (out_dtype != SV_BF16 && out_dtype != SV_FP32)) return SV_ERR_INVALID;
  if (B == 0) return SV_OK;
  if (bad_place(src) || !seq_len || !out || ((uintptr_t)out & 15u) || (int64_t)B * R > INT32_MAX) return SV_ERR_INVALID;
  if (!src->block_table && src->rows < R) return SV_ERR_INVALID;
  const dim3 grid((unsigned)(B * R)), block(kReadThreads);
  const cudaError_t e =
      out_dtype == SV_FP32
          ? sv_launch_pdl(kv_read_kernel<true>, grid, block, 0, (cudaStream_t)stream, (int)R, seq_len, n_nodes, *src, out, h->d_err)
          : sv_launch_pdl(kv_read_kernel<false>, grid, block, 0, (cudaStream_t)stream, (int)R, seq_len, n_nodes, *src, out, h->d_err);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return SV_OK;
}
