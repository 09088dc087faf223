// Rules on the target's rows before they are verified: penalties for repeated
// tokens, biases, grammar masks.
#include "entries.cuh"

namespace sv {

constexpr int kRuleThreads = 256;
constexpr int kSlice = 4096;         // tokens of one CTA
constexpr int kGroups = kSlice / 8;  // eight tokens to a 16-byte bf16 vector

struct RuleSmem {
  int count[kSlice];        // occurrences in the history (and, while a row is worked, its path)
  float bias[kSlice];
  uint8_t touched[kGroups]; // the group has a count or a bias
};

// One CTA per (request, slice of 4096 tokens) works on the slice of every row of
// the request: the history and the biases are looked through once, into counts
// and sums in shared memory, and the rows stream past them.  Bound by memory:
// each logit is read and written once.
template <bool F32>
__global__ void __launch_bounds__(kRuleThreads) logit_rules_kernel(const __grid_constant__ sv_logits_args a, int* err) {
  pdl_wait();
  pdl_trigger();
  __shared__ RuleSmem s;
  const int b = blockIdx.y, t = threadIdx.x, lane = t & 31;
  const int v0 = blockIdx.x * kSlice, len = min(kSlice, a.V - v0);
  int n = a.n_nodes ? a.n_nodes[b] : a.R - 1;
  const float rep = a.rep_penalty ? a.rep_penalty[b] : 1.0f;
  const float pres = a.presence ? a.presence[b] : 0.0f, freq = a.frequency ? a.frequency[b] : 0.0f;
  const bool bad = !(rep > 0.0f && rep < __int_as_float(0x7F800000)) || n >= a.R;
  if (bad) {
    if (t == 0 && blockIdx.x == 0) report(err, SV_ERR_STATE);
    n = -1;
  }
  for (int i = t; i < kSlice; i += kRuleThreads) s.count[i] = 0, s.bias[i] = 0.0f;
  for (int i = t; i < kGroups; i += kRuleThreads) s.touched[i] = 0;
  __syncthreads();
  if (n >= 0) {
    for (int i = t; i < a.history_ld; i += kRuleThreads) {
      const int x = a.history[b * a.history_ld + i] - v0;
      if (x >= 0 && x < len) atomicAdd(&s.count[x], 1), s.touched[x >> 3] = 1;
    }
    // one warp adds the biases, so that a token named several times gets its
    // values in list order
    if (t < 32)
      for (int i0 = 0; i0 < a.bias_ld; i0 += 32) {
        const bool in = i0 + lane < a.bias_ld;
        const int x = in ? a.bias_ids[b * a.bias_ld + i0 + lane] - v0 : -1;
        const float v = in ? a.bias_values[b * a.bias_ld + i0 + lane] : 0.0f;
        const bool hit = x >= 0 && x < len;
        uint32_t hits = __ballot_sync(0xFFFFFFFFu, hit);
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, hit ? x : -1 - lane);
        if (__all_sync(0xFFFFFFFFu, same == 1u << lane)) {
          if (hit) s.bias[x] += v, s.touched[x >> 3] = 1;
        } else {
          for (; hits; hits &= hits - 1) {
            if (lane == __ffs(hits) - 1) s.bias[x] += v, s.touched[x >> 3] = 1;
            __syncwarp();
          }
        }
        __syncwarp();
      }
  }
  const int eb = F32 ? 4 : 2;
  for (int i = 0; i < a.R; ++i) {
    const bool live = i <= n;
    if (!live && a.logits == a.out) break;  // unchanged, and so is every later row
    const int64_t row = (int64_t)b * a.R + i;
    if (i == 0) __syncthreads();
    const int np = !live ? 0 : a.mask ? n : i;  // drafted nodes that may be on the path
    if (np > 0) {
      __syncthreads();
      for (int j = t; j < np; j += kRuleThreads) {
        const int node = j + 1;
        if (a.mask && !(a.mask[row * a.mask_ld + (node >> 5)] >> (node & 31) & 1)) continue;
        const int x = a.tokens[(int64_t)b * (a.R - 1) + j] - v0;
        if (x >= 0 && x < len) atomicAdd(&s.count[x], 1), s.touched[x >> 3] = 1;
      }
      __syncthreads();
    }
    const char* src = static_cast<const char*>(a.logits) + (row * a.ld + v0) * eb;
    char* dst = static_cast<char*>(a.out) + (row * a.out_ld + v0) * eb;
    const uint8_t* allow =
        a.allowed && live ? reinterpret_cast<const uint8_t*>(a.allowed + row * a.allowed_ld) + v0 / 8 : nullptr;
    for (int g = t; g * 8 < len; g += kRuleThreads) {
      float x[8];
      const bool whole = 8 * g + 8 <= len;  // a row may end right after its last token
      if (whole) {
        load8<F32>(src, 8 * g, x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[e] = 8 * g + e >= len ? 0.0f
                 : F32            ? reinterpret_cast<const float*>(src)[8 * g + e]
                                  : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src)[8 * g + e]);
      }
      const uint32_t bits = allow ? allow[g] : 0xFFu;
      if (live && s.touched[g]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = s.count[8 * g + e];
          if (c > 0) x[e] = (x[e] > 0.0f ? x[e] / rep : x[e] * rep) - (freq * (float)c + pres);
          x[e] += s.bias[8 * g + e];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(bits >> e & 1)) x[e] = __int_as_float(0xFF800000);
      if (whole) {
        store8<F32>(dst, 8 * g, x);
      } else {
        for (int e = 0; 8 * g + e < len; ++e) {
          if (F32)
            reinterpret_cast<float*>(dst)[8 * g + e] = x[e];
          else
            reinterpret_cast<__nv_bfloat16*>(dst)[8 * g + e] = __float2bfloat16_rn(x[e]);
        }
      }
    }
    if (np > 0) {
      __syncthreads();
      for (int j = t; j < np; j += kRuleThreads) {
        const int node = j + 1;
        if (a.mask && !(a.mask[row * a.mask_ld + (node >> 5)] >> (node & 31) & 1)) continue;
        const int x = a.tokens[(int64_t)b * (a.R - 1) + j] - v0;
        if (x >= 0 && x < len) atomicSub(&s.count[x], 1);
      }
    }
  }
}

}  // namespace sv

using namespace sv;

extern "C" size_t sv_logits_args_size(void) { return sizeof(sv_logits_args); }

extern "C" sv_status sv_adjust_logits(sv_handle* h, const sv_logits_args* a, sv_stream_t stream) {
  if (!h || !a || a->B < 0 || a->R < 1 || a->V < 1 || (a->dtype != SV_BF16 && a->dtype != SV_FP32)) return SV_ERR_INVALID;
  if (a->B == 0) return SV_OK;
  const int eb = a->dtype == SV_BF16 ? 2 : 4;
  if (!a->logits || !a->out || ((uintptr_t)a->logits & 15u) || ((uintptr_t)a->out & 15u)) return SV_ERR_INVALID;
  if (a->ld < a->V || a->out_ld < a->V || (a->ld * eb) % 16 || (a->out_ld * eb) % 16) return SV_ERR_INVALID;
  if (a->logits == a->out && a->ld != a->out_ld) return SV_ERR_INVALID;
  if (a->history_ld < 0 || a->history_ld > (1 << 24) || (a->history_ld > 0 && !a->history)) return SV_ERR_INVALID;
  if (a->bias_ld < 0 || a->bias_ld > (1 << 24) || (a->bias_ld > 0 && (!a->bias_ids || !a->bias_values))) return SV_ERR_INVALID;
  if (a->R > 1 && !a->tokens) return SV_ERR_INVALID;
  if (a->mask && a->mask_ld < (a->R + 31) / 32) return SV_ERR_INVALID;
  if (a->allowed && a->allowed_ld < ((int64_t)a->V + 31) / 32) return SV_ERR_INVALID;
  if (a->B > 65535) return SV_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)((a->V + kSlice - 1) / kSlice), (unsigned)a->B), block(kRuleThreads);
  const cudaError_t e = a->dtype == SV_FP32
                            ? sv_launch_pdl(logit_rules_kernel<true>, grid, block, 0, (cudaStream_t)stream, *a, h->d_err)
                            : sv_launch_pdl(logit_rules_kernel<false>, grid, block, 0, (cudaStream_t)stream, *a, h->d_err);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return SV_OK;
}
