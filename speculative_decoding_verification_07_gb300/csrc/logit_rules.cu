// Rules on the target's rows before they are verified: penalties for repeated
// tokens, biases, grammar masks.
#include "entries.cuh"

namespace sv {

constexpr int kRuleThreads = 256;
constexpr int kSlice = 4096;  // tokens of one CTA
constexpr int kFlight = 4;    // vectors a thread has on their way

struct RuleSmem {
  int count[kSlice];       // occurrences in the history (and, while a row is patched, in its path)
  float bias[kSlice];
  uint16_t listed[kSlice]; // tokens with a count or a bias; a row's own ones after them
  uint8_t known[kSlice];   // in the list
  int n, n_row, n_path;    // listed, with the row's own ones, drafted tokens of this slice
};

// One CTA takes a slice of 4096 tokens of one request's rows, or of `per` of
// them.  The grammar mask touches every logit, the other rules a few: so the
// rows are streamed with the mask alone (out = allowed ? logit : -inf, 16 bytes
// a thread, four in flight, no look-up), and then the tokens that a penalty or
// a bias concerns, listed once per slice from the history and the biases, are
// written again from the row's logits.  Bound by memory: each logit is read and
// written once.  Looking up counts and biases for every logit as it passed took
// 109 us instead of 45 for 64 x 7 rows of 128256 (bf16).
template <bool F32>
__global__ void __launch_bounds__(kRuleThreads) logit_rules_kernel(const __grid_constant__ sv_logits_args a, int per, int* err) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) RuleSmem s;
  constexpr int eb = F32 ? 4 : 2;
  const int b = blockIdx.y, t = threadIdx.x, lane = t & 31;
  const int v0 = blockIdx.x * kSlice, len = min(kSlice, a.V - v0), groups = (len + 7) / 8;
  const int r0 = blockIdx.z * per, r1 = min(a.R, r0 + per);
  int n = a.n_nodes ? a.n_nodes[b] : a.R - 1;
  const float rep = a.rep_penalty ? a.rep_penalty[b] : 1.0f;
  const float pres = a.presence ? a.presence[b] : 0.0f, freq = a.frequency ? a.frequency[b] : 0.0f;
  if (!(rep > 0.0f && rep < __builtin_huge_valf()) || n >= a.R) {
    if (t == 0 && blockIdx.x == 0 && blockIdx.z == 0) report(err, SV_ERR_STATE);
    n = -1;
  }
  const int live = min(r1, n + 1) - r0;  // rows of this CTA that the rules apply to
  const bool in_place = a.logits == a.out;
  const char* src0 = static_cast<const char*>(a.logits) + ((int64_t)b * a.R * a.ld + v0) * eb;
  char* dst0 = static_cast<char*>(a.out) + ((int64_t)b * a.R * a.out_ld + v0) * eb;

  // ---- the tokens the rules concern ----------------------------------------
  if (live > 0) {
    for (int i = t; i < kSlice / 4; i += kRuleThreads) {
      reinterpret_cast<int4*>(s.count)[i] = make_int4(0, 0, 0, 0);
      if (a.bias_ld > 0) reinterpret_cast<float4*>(s.bias)[i] = make_float4(0, 0, 0, 0);
      reinterpret_cast<uint32_t*>(s.known)[i] = 0;
    }
    if (t == 0) s.n = s.n_path = 0;
    __syncthreads();
    auto list = [&](int x, int* n) { s.listed[atomicAdd(n, 1)] = (uint16_t)x; };
    for (int i = t; i < a.history_ld; i += kRuleThreads) {
      const int x = a.history[b * a.history_ld + i] - v0;
      if (x >= 0 && x < len && atomicAdd(&s.count[x], 1) == 0) s.known[x] = 1, list(x, &s.n);
    }
    const int np = a.mask ? n : min(n, r1 - 1);
    for (int j = t; j < np; j += kRuleThreads) {
      const int x = a.tokens[(int64_t)b * (a.R - 1) + j] - v0;
      if (x >= 0 && x < len) s.n_path = 1;
    }
    __syncthreads();
    // one warp adds the biases, so that a token named several times gets its
    // values in list order
    if (t < 32)
      for (int i0 = 0; i0 < a.bias_ld; i0 += 32) {
        const bool in = i0 + lane < a.bias_ld;
        const int x = in ? a.bias_ids[b * a.bias_ld + i0 + lane] - v0 : -1;
        const float v = in ? a.bias_values[b * a.bias_ld + i0 + lane] : 0.0f;
        const bool hit = x >= 0 && x < len;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, hit ? x : -1 - lane);
        auto add = [&] {
          s.bias[x] += v;
          if (!s.known[x]) s.known[x] = 1, list(x, &s.n);
        };
        if (__all_sync(0xFFFFFFFFu, same == 1u << lane)) {
          if (hit) add();
        } else {
          for (uint32_t hits = __ballot_sync(0xFFFFFFFFu, hit); hits; hits &= hits - 1) {
            if (lane == __ffs(hits) - 1) add();
            __syncwarp();
          }
        }
        __syncwarp();
      }
  }

  // ---- every logit: copied, or -inf ----------------------------------------
  const int rows = in_place ? live : r1 - r0;  // rows without rules are copied
  if (!in_place || a.allowed) {
    const int total = rows * groups;
    auto row_of = [&](int k) { return groups == kSlice / 8 ? k / (kSlice / 8) : k / groups; };
    for (int g0 = t; g0 < total; g0 += kFlight * kRuleThreads) {
      uint4 lo[kFlight], hi[kFlight];
      uint32_t bits[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int k = g0 + u * kRuleThreads, r = row_of(k), g = k - r * groups;
        if (k >= total) continue;
        const char* p = src0 + (int64_t)(r0 + r) * a.ld * eb + g * 8 * eb;
        bits[u] = 0xFFu;
        if (a.allowed && r < live)
          bits[u] = reinterpret_cast<const uint8_t*>(a.allowed + ((int64_t)b * a.R + r0 + r) * a.allowed_ld)[v0 / 8 + g];
        if (8 * g + 8 <= len) {
          lo[u] = *reinterpret_cast<const uint4*>(p);
          if (F32) hi[u] = reinterpret_cast<const uint4*>(p)[1];
        } else {  // a row may end right after its last token
          uint32_t w[8] = {};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (8 * g + e >= len) break;
            if (F32)
              w[e] = reinterpret_cast<const uint32_t*>(p)[e];
            else
              w[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << 16 * (e & 1);
          }
          lo[u] = make_uint4(w[0], w[1], w[2], w[3]), hi[u] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int k = g0 + u * kRuleThreads, r = row_of(k), g = k - r * groups;
        if (k >= total || (in_place && bits[u] == 0xFFu)) continue;
        char* p = dst0 + (int64_t)(r0 + r) * a.out_ld * eb + g * 8 * eb;
        uint32_t w[8] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w, hi[u].x, hi[u].y, hi[u].z, hi[u].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool ban = !(bits[u] >> e & 1);
          if (F32)
            w[e] = ban ? 0xFF800000u : w[e];
          else if (ban)
            w[e >> 1] = e & 1 ? (w[e >> 1] & 0xFFFFu) | 0xFF800000u : (w[e >> 1] & 0xFFFF0000u) | 0xFF80u;
        }
        if (8 * g + 8 <= len) {
          *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
          if (F32) reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (8 * g + e >= len) break;
            if (F32)
              reinterpret_cast<uint32_t*>(p)[e] = w[e];
            else
              reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e >> 1] >> 16 * (e & 1));
          }
        }
      }
    }
  }
  if (live <= 0) return;
  __syncthreads();

  // ---- the listed tokens again ---------------------------------------------
  auto patch = [&](int r, int x) {
    const int64_t row = (int64_t)b * a.R + r0 + r;
    const int v = v0 + x;
    if (a.allowed && !(a.allowed[row * a.allowed_ld + (v >> 5)] >> (v & 31) & 1)) return;
    const int64_t at = (int64_t)(r0 + r) * a.ld + x, to = (int64_t)(r0 + r) * a.out_ld + x;
    float l = F32 ? reinterpret_cast<const float*>(src0)[at]
                  : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src0)[at]);
    const int c = s.count[x];
    if (c > 0) l = (l > 0.0f ? l / rep : l * rep) - (freq * (float)c + pres);
    if (a.bias_ld > 0) l += s.bias[x];
    if (F32)
      reinterpret_cast<float*>(dst0)[to] = l;
    else
      reinterpret_cast<__nv_bfloat16*>(dst0)[to] = __float2bfloat16_rn(l);
  };
  const int listed = s.n;
  if (!s.n_path) {  // no drafted token is in this slice: every row has the same list
    for (int k = t; k < live * listed; k += kRuleThreads) patch(k / listed, s.listed[k % listed]);
    return;
  }
  for (int r = 0; r < live; ++r) {
    const int64_t row = (int64_t)b * a.R + r0 + r;
    const int np = a.mask ? n : r0 + r;  // drafted nodes that may be on the path
    auto on_path = [&](int j) -> int {   // the node's token in this slice, or -1
      const int node = j + 1;
      if (a.mask && !(a.mask[row * a.mask_ld + (node >> 5)] >> (node & 31) & 1)) return -1;
      const int x = a.tokens[(int64_t)b * (a.R - 1) + j] - v0;
      return x >= 0 && x < len ? x : -1;
    };
    if (t == 0) s.n_row = listed;
    __syncthreads();
    for (int j = t; j < np; j += kRuleThreads) {
      const int x = on_path(j);
      if (x >= 0 && atomicAdd(&s.count[x], 1) == 0 && !s.known[x]) s.listed[atomicAdd(&s.n_row, 1)] = (uint16_t)x;
    }
    __syncthreads();
    for (int k = t; k < s.n_row; k += kRuleThreads) patch(r, s.listed[k]);
    __syncthreads();
    for (int j = t; j < np; j += kRuleThreads) {
      const int x = on_path(j);
      if (x >= 0) atomicSub(&s.count[x], 1);
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
  // Rows share a CTA's lists where there are CTAs enough without it; a small
  // call gives each row its own, so that rows do not wait for one another.
  const int64_t slices = (a->V + kSlice - 1) / kSlice, wanted = 2 * (int64_t)h->num_sms;
  int parts = (int)((wanted + slices * a->B - 1) / (slices * a->B));
  parts = parts < 1 ? 1 : parts > a->R ? a->R : parts;
  const int per = (a->R + parts - 1) / parts;
  const dim3 grid((unsigned)slices, (unsigned)a->B, (unsigned)((a->R + per - 1) / per)), block(kRuleThreads);
  const cudaError_t e =
      a->dtype == SV_FP32
          ? sv_launch_pdl(logit_rules_kernel<true>, grid, block, 0, (cudaStream_t)stream, *a, per, h->d_err)
          : sv_launch_pdl(logit_rules_kernel<false>, grid, block, 0, (cudaStream_t)stream, *a, per, h->d_err);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return SV_ERR_CUDA;
  }
  return SV_OK;
}
