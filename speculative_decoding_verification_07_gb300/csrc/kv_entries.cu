// The entries of a verify pass: rotary positions, formats, write and read back.
#include "entries.cuh"

namespace sv {

constexpr int kEntryThreads = 256;

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

// One CTA per (request, entry): its queries, keys and values are rows of
// head_dim; a thread keeps its eight columns' cos / sin in registers for all
// heads.  Bound by memory: each value is read once and written once, the
// table's row once per entry.
template <bool F32>
__global__ void __launch_bounds__(kEntryThreads) kv_append_kernel(const __grid_constant__ AppendParams P) {
  pdl_wait();
  pdl_trigger();
  const sv_append_args& a = P.a;
  const sv_kv_place& dst = a.dst;
  const int b = blockIdx.x / a.R, i = blockIdx.x - b * a.R;
  int n = a.n_nodes ? a.n_nodes[b] : a.R - 1;
  if (n >= a.R) {
    if (threadIdx.x == 0 && i == 0) report(P.err, SV_ERR_STATE);
    n = a.R - 1;
  }
  const RowLanes L(dst.head_dim);
  const int Hq = a.q ? a.Hq : 0, H = dst.heads, d0 = 8 * L.c;
  const int64_t S = a.seq_len[b];
  bool live = i <= n;
  int64_t off = -1;
  const float* cs = nullptr;
  if (live) {
    off = entry_offset(dst, b, i, S + i);
    live = off >= 0;
    if (a.rope) {
      const int64_t pos = S + (a.depth ? a.depth[(int64_t)b * a.R + i] : i);
      live = live && pos >= 0 && pos < a.max_pos;
      cs = a.rope + pos * a.rot_dim;
    }
    if (!live && threadIdx.x == 0) report(P.err, SV_ERR_STATE);
  }
  if (!L.on) return;
  if (!live) {
    const float zero[8] = {};
    for (int h = L.slot; h < Hq; h += L.nslots)
      store8<F32>(a.q_out, b * a.q_out_stride[0] + i * a.q_out_stride[1] + h * a.q_out_stride[2] + d0, zero);
    return;
  }
  // cos and (signed) sin of this thread's eight columns, and where the other
  // half of each pair is: x' = x cos + other * sin
  const bool pairs = a.flags & SV_APPEND_PAIRS;
  const int half = a.rot_dim >> 1;
  float co[8], si[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = d0 + e;
    co[e] = 1.0f, si[e] = 0.0f;
    if (cs && d < a.rot_dim) {
      const int p = pairs ? d >> 1 : d < half ? d : d - half;
      const bool first = pairs ? !(d & 1) : d < half;
      const float2 v = reinterpret_cast<const float2*>(cs)[p];
      co[e] = v.x, si[e] = first ? -v.y : v.y;
    }
  }
  const int64_t step = row_step(dst);
  const int rows = Hq + 2 * H;
  for (int r = L.slot; r < rows; r += L.nslots) {
    const bool is_q = r < Hq, is_v = r >= Hq + H;
    const int h = is_q ? r : is_v ? r - Hq - H : r - Hq;
    const void* src = is_q ? a.q : is_v ? a.v : a.k;
    const int64_t* st = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
    const int64_t at = b * st[0] + i * st[1] + h * st[2];
    float x[8], o[8];
    load8<F32>(src, at + d0, x);
    const bool rot = cs && !is_v && d0 < a.rot_dim;
    if (rot) {
      if (pairs) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = x[e ^ 1];
      } else if (half % 8 == 0) {
        load8<F32>(src, at + (d0 < half ? d0 + half : d0 - half), o);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int d = d0 + e;
          const int64_t q = at + (d < half ? d + half : d < a.rot_dim ? d - half : d);
          o[e] = F32 ? static_cast<const float*>(src)[q]
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(src)[q]);
        }
      }
    }
    __syncwarp(L.group);  // q may be rotated in place: every lane has its operands
    if (rot) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (d0 + e < a.rot_dim) x[e] = x[e] * co[e] + o[e] * si[e];
    }
    if (is_q) {
      store8<F32>(a.q_out, b * a.q_out_stride[0] + i * a.q_out_stride[1] + h * a.q_out_stride[2] + d0, x);
      continue;
    }
    char* row = static_cast<char*>(dst.data) + off + (is_v ? H + h : h) * step;
    if (dst.format == SV_KV_FP32) {
      store8<true>(row, d0, x);
    } else if (dst.format == SV_KV_BF16) {
      store8<false>(row, d0, x);
    } else {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));  // NaN is left out
      const float scale = e4m3_scale(__uint_as_float(__reduce_max_sync(L.group, __float_as_uint(m))));
      // scales are 2^-126 .. 2^120, so 1 / scale is exact
      const float inv = 1.0f / scale;
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

template <bool F32>
__global__ void __launch_bounds__(kEntryThreads) kv_read_kernel(int R, const int32_t* seq_len,
                                                                const int32_t* n_nodes,
                                                                const __grid_constant__ sv_kv_place src,
                                                                void* out, int* err) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / R, i = blockIdx.x - b * R;
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
  const RowLanes L(src.head_dim);
  if (!L.on) return;
  const int64_t step = row_step(src);
  for (int r = L.slot; r < 2 * src.heads; r += L.nslots) {
    float x[8] = {};
    if (off >= 0) {
      const char* row = static_cast<const char*>(src.data) + off + r * step;
      load_entry8(row, src.format, 8 * L.c, entry_scale(row, src.format, src.head_dim), x);
    }
    store8<F32>(out, ((int64_t)blockIdx.x * 2 * src.heads + r) * src.head_dim + 8 * L.c, x);
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
  const dim3 grid((unsigned)(a->B * a->R)), block(kEntryThreads);
  const cudaError_t e = a->dtype == SV_FP32
                            ? sv_launch_pdl(kv_append_kernel<true>, grid, block, 0, (cudaStream_t)stream, P)
                            : sv_launch_pdl(kv_append_kernel<false>, grid, block, 0, (cudaStream_t)stream, P);
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
  const dim3 grid((unsigned)(B * R)), block(kEntryThreads);
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
