// K/V entries as device code sees them: a place (paged or staged), its row
// addresses, and the three formats' conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace sv {

constexpr int kTail = 16;  // bytes after an 8-bit entry's codes: its fp32 scale, then zeros
constexpr int kMaxHeadDim = 256;

__host__ __device__ __forceinline__ int row_bytes(const sv_kv_place& p) {
  return p.format == SV_KV_FP32 ? 4 * p.head_dim
                                : p.format == SV_KV_BF16 ? 2 * p.head_dim : p.head_dim + kTail;
}

// Host check of a place; B is only needed to know that it may be empty.
static inline bool bad_place(const sv_kv_place* p) {
  if (!p || !p->data || ((uintptr_t)p->data & 15u)) return true;
  if (p->layers < 1 || p->heads < 1 || p->layer < 0 || p->layer >= p->layers) return true;
  if (p->format != SV_KV_BF16 && p->format != SV_KV_FP32 && p->format != SV_KV_E4M3) return true;
  if (p->head_dim < 8 || p->head_dim > kMaxHeadDim || p->head_dim % (p->format == SV_KV_E4M3 ? 16 : 8))
    return true;
  if (p->block_table) return p->num_blocks < 0 || p->block_size < 1 || p->max_blocks < 1;
  return p->rows < 1;
}

// Strides {request, entry, head} in elements of eb bytes: multiples of 16 bytes.
static inline bool bad_strides(const void* p, const int64_t* st, int eb) {
  return !p || ((uintptr_t)p & 15u) || (st[0] * eb) % 16 || (st[1] * eb) % 16 || (st[2] * eb) % 16;
}

// Byte offset of head 0's K row of entry i of request b (position S + i when
// paged), or -1 when it has no block.  Other heads and V follow at
// row_step(p) and heads * row_step(p).  64-bit throughout: a cache may exceed
// 2^32 bytes.
__device__ __forceinline__ int64_t entry_offset(const sv_kv_place& p, int b, int i, int64_t pos) {
  const int rb = row_bytes(p);
  if (!p.block_table)
    return ((((int64_t)b * p.rows + i) * p.layers + p.layer) * 2) * p.heads * (int64_t)rb;
  if (pos < 0 || pos > INT32_MAX) return -1;
  const uint32_t at = (uint32_t)pos, bs = (uint32_t)p.block_size;
  const uint32_t j = (bs & (bs - 1)) ? at / bs : at >> (31 - __clz(bs));
  if (j >= (uint32_t)p.max_blocks) return -1;
  const int blk = p.block_table[(int64_t)b * p.max_blocks + j];
  if (blk < 0 || blk >= p.num_blocks) return -1;
  return (((int64_t)blk * p.layers + p.layer) * 2 * p.heads * p.block_size + (at - j * bs)) * rb;
}

__device__ __forceinline__ int64_t row_step(const sv_kv_place& p) {
  return (int64_t)row_bytes(p) * (p.block_table ? p.block_size : 1);
}

// Eight consecutive values at element d of a row.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t elem, float (&x)[8]) {
  if (F32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + elem);
    const float4 a = s[0], b = s[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + elem);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t elem, const float (&x)[8]) {
  if (F32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + elem);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + elem) = make_uint4(
        pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
}

// Two 8-bit codes (low byte first) -> their values.
__device__ __forceinline__ float2 e4m3x2_values(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight values at element d of an entry's row, decoded; scale is 1 but for
// the 8-bit format.
__device__ __forceinline__ void load_entry8(const char* row, int format, int d, float scale, float (&x)[8]) {
  if (format == SV_KV_FP32) {
    load8<true>(row, d, x);
  } else if (format == SV_KV_BF16) {
    load8<false>(row, d, x);
  } else {
    const uint2 c = *reinterpret_cast<const uint2*>(row + d);
    const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = e4m3x2_values(w[i]);
      x[2 * i] = v.x * scale, x[2 * i + 1] = v.y * scale;
    }
  }
}

__device__ __forceinline__ float entry_scale(const char* row, int format, int head_dim) {
  return format == SV_KV_E4M3 ? *reinterpret_cast<const float*>(row + head_dim) : 1.0f;
}

// The smallest power of two with amax <= 448 * scale: amax = f * 2^x with f in
// [1, 2) and 448 = 1.75 * 2^8, so 2^(x - 8), or 2^(x - 7) where f > 1.75.  A
// power of two makes x / scale exact (but for underflow), so codes do not
// depend on how the division rounds, and the format's relative precision is
// the same at every scale.  Clamped to normal numbers; infinity gives 2^120, zero
// what the caller says.
constexpr float kLeastScale = 0x1p-126f;

__device__ __forceinline__ float e4m3_scale(float amax, float of_zeros) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return of_zeros;
  const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u && u < 0x7F800000u ? 1 : 0);
  return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}

}  // namespace sv
