// Rules on the target's rows before they are verified: penalties for repeated
// tokens, biases, grammar masks.
#include "entries.cuh"

namespace sv {

constexpr int kRuleThreads = 512, kListThreads = 64;  // of them, those that make the lists
constexpr int kSlice = 4096;  // tokens of one CTA
constexpr int kNodes = 256;   // drafted tokens of a slice that are kept at hand

struct RuleSmem {
  int count[kSlice];       // occurrences in the history
  float bias[kSlice];
  uint16_t listed[kSlice]; // tokens with a count or a bias
  uint8_t known[kSlice];   // in the list
  int node[kNodes];  // drafted nodes whose token is in this slice, and the token
  uint16_t token[kNodes];
  int n, n_path;           // listed tokens, such nodes (more than kNodes: look through all)
};

static __device__ __forceinline__ void list_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kListThreads) : "memory"); }

// One CTA takes a slice of 4096 tokens of one request's rows, or of `per` of
// them.  The grammar mask touches every logit, the other rules a few: so the
// rows are streamed with the mask alone (out = allowed ? logit : -inf, 16 bytes
// a thread, no look-up), and then the tokens that a penalty or a bias concerns,
// listed once per slice from the history and the biases, are written again from
// the row's logits; a row's own path only adds to their counts, so all rows are
// written at once.  Bound by memory: each logit is read and written once.  64 x 7
// rows of 128256 (bf16): looking up counts and biases for every logit as it
// passed 109 us, a list 71, rows patched together 55, half as many lists (slices
// of 4096 for 512 threads, not 2048 for 256) 50, lists made by two warps while
// the others stream 48 (by one 53, by four 51), 4.9 TB/s; the copy alone 41.
// Larger CTAs or two vectors on their way leave fewer threads on an SM: 68 and 52.
template <bool F32>
__global__ void __launch_bounds__(kRuleThreads, 4) logit_rules_kernel(const __grid_constant__ sv_logits_args a, int per, int* err) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) RuleSmem s;
  constexpr int eb = F32 ? 4 : 2;
  // slices outermost: the first, where frequent tokens are, take longest
  const int b = blockIdx.x, t = threadIdx.x, lane = t & 31;
  const int v0 = blockIdx.y * kSlice, len = min(kSlice, a.V - v0), groups = (len + 7) / 8;
  const int r0 = blockIdx.z * per, r1 = min(a.R, r0 + per);
  int n = a.n_nodes ? a.n_nodes[b] : a.R - 1;
  const float rep = a.rep_penalty ? a.rep_penalty[b] : 1.0f;
  const float pres = a.presence ? a.presence[b] : 0.0f, freq = a.frequency ? a.frequency[b] : 0.0f;
  if (!(rep > 0.0f && rep < __builtin_huge_valf()) || n >= a.R) {
    if (t == 0 && blockIdx.y == 0 && blockIdx.z == 0) report(err, SV_ERR_STATE);
    n = -1;
  }
  const int live = min(r1, n + 1) - r0;  // rows of this CTA that the rules apply to
  const bool in_place = a.logits == a.out;
  const char* src0 = static_cast<const char*>(a.logits) + ((int64_t)b * a.R * a.ld + v0) * eb;
  char* dst0 = static_cast<char*>(a.out) + ((int64_t)b * a.R * a.out_ld + v0) * eb;

  const int total = !in_place ? (r1 - r0) * groups : a.allowed ? live * groups : 0;  // rows without rules are copied
  auto row_of = [&](int k) { return groups == kSlice / 8 ? k / (kSlice / 8) : k / groups; };
  struct Vector {
    uint4 lo, hi;  // eight logits; hi of fp32 alone
    uint32_t bits;
  };
  auto fetch = [&](Vector& q, int k) {
    if (k >= total) return;
    const int r = row_of(k), g = k - r * groups;
    const char* p = src0 + (int64_t)(r0 + r) * a.ld * eb + g * 8 * eb;
    q.bits = 0xFFu;
    if (a.allowed && r < live)
      q.bits = reinterpret_cast<const uint8_t*>(a.allowed + ((int64_t)b * a.R + r0 + r) * a.allowed_ld)[v0 / 8 + g];
    if (8 * g + 8 <= len) {
      q.lo = *reinterpret_cast<const uint4*>(p);
      if (F32) q.hi = reinterpret_cast<const uint4*>(p)[1];
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
      q.lo = make_uint4(w[0], w[1], w[2], w[3]);
      if (F32) q.hi = make_uint4(w[4], w[5], w[6], w[7]);
    }
  };
  auto put = [&](const Vector& q, int k) {
    if (in_place && q.bits == 0xFFu) return;
    const int r = row_of(k), g = k - r * groups;
    char* p = dst0 + (int64_t)(r0 + r) * a.out_ld * eb + g * 8 * eb;
    uint32_t w[8] = {q.lo.x, q.lo.y, q.lo.z, q.lo.w};
    if (F32) w[4] = q.hi.x, w[5] = q.hi.y, w[6] = q.hi.z, w[7] = q.hi.w;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool ban = !(q.bits >> e & 1);
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
  };

  // ---- the tokens the rules concern ----------------------------------------
  if (live > 0 && t < kListThreads) {
    for (int i = t; i < kSlice / 4; i += kListThreads) {
      reinterpret_cast<int4*>(s.count)[i] = make_int4(0, 0, 0, 0);
      if (a.bias_ld > 0) reinterpret_cast<float4*>(s.bias)[i] = make_float4(0, 0, 0, 0);
      reinterpret_cast<uint32_t*>(s.known)[i] = 0;
    }
    if (t == 0) s.n = s.n_path = 0;
    list_barrier();
    auto list = [&](int x, int* n) { s.listed[atomicAdd(n, 1)] = (uint16_t)x; };
    for (int i0 = t; i0 < a.history_ld; i0 += 4 * kListThreads) {
      int x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kListThreads;
        x[u] = i < a.history_ld ? a.history[b * a.history_ld + i] - v0 : -1;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (x[u] >= 0 && x[u] < len && atomicAdd(&s.count[x[u]], 1) == 0) s.known[x[u]] = 1, list(x[u], &s.n);
    }
    const int np = a.mask ? n : min(n, r1 - 1);
    for (int j = t; j < np; j += kListThreads) {
      const int x = a.tokens[(int64_t)b * (a.R - 1) + j] - v0;
      if (x >= 0 && x < len) {
        const int q = atomicAdd(&s.n_path, 1);
        if (q < kNodes) s.node[q] = j + 1, s.token[q] = (uint16_t)x;
      }
    }
    list_barrier();
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
  } else {
    // ---- every logit: copied, or -inf --------------------------------------
    // A vector is always on its way: the next is asked for before the one at hand
    // is written.
    const int first = live > 0 ? kListThreads : 0, step = kRuleThreads - first;
    Vector now;
    fetch(now, t - first);
#pragma unroll 1
    for (int k = t - first; k < total; k += step) {
      Vector next;
      fetch(next, k + step);
      put(now, k);
      now = next;
    }
  }
  if (live <= 0) return;
  __syncthreads();

  // ---- the listed tokens again ---------------------------------------------
  const bool kept = s.n_path <= kNodes;
  const int nodes = kept ? s.n_path : a.mask ? n : min(n, r1 - 1);
  auto token_of = [&](int q) { return kept ? (int)s.token[q] : a.tokens[(int64_t)b * (a.R - 1) + q] - v0; };
  auto on_path = [&](int r, int q) {
    const int node = kept ? s.node[q] : q + 1;
    if (!a.mask) return node <= r0 + r;
    return (bool)(a.mask[((int64_t)b * a.R + r0 + r) * a.mask_ld + (node >> 5)] >> (node & 31) & 1);
  };
  // a row's logit of a listed token; banned ones stay as they are
  auto at = [&](int64_t ld, int r, int x) { return (int64_t)(r0 + r) * ld + x; };
  auto banned = [&](int r, int x) {
    const int v = v0 + x;
    return a.allowed && !(a.allowed[((int64_t)b * a.R + r0 + r) * a.allowed_ld + (v >> 5)] >> (v & 31) & 1);
  };
  auto logit = [&](int r, int x) {
    return F32 ? reinterpret_cast<const float*>(src0)[at(a.ld, r, x)]
               : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src0)[at(a.ld, r, x)]);
  };
  auto patch = [&](int r, int x, int c, float l) {
    if (c > 0) l = (l > 0.0f ? l / rep : l * rep) - (freq * (float)c + pres);
    if (a.bias_ld > 0) l += s.bias[x];
    if (F32)
      reinterpret_cast<float*>(dst0)[at(a.out_ld, r, x)] = l;
    else
      reinterpret_cast<__nv_bfloat16*>(dst0)[at(a.out_ld, r, x)] = __float2bfloat16_rn(l);
  };
  const int listed = s.n;
  for (int k0 = t; k0 < live * listed; k0 += 4 * kRuleThreads) {
    float l[4];
    bool off[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * kRuleThreads, r = k / listed;
      off[u] = k >= live * listed;
      if (off[u]) continue;
      const int x = s.listed[k - r * listed];
      l[u] = logit(r, x), off[u] = banned(r, x);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (off[u]) continue;
      const int k = k0 + u * kRuleThreads, r = k / listed, x = s.listed[k - r * listed];
      int c = s.count[x];
      for (int q = 0; q < nodes; ++q) c += token_of(q) == x && on_path(r, q);
      patch(r, x, c, l[u]);
    }
  }
  for (int k = t; k < live * nodes; k += kRuleThreads) {  // tokens that only the path has, each once
    const int r = k / nodes, q = k - r * nodes, x = token_of(q);
    if (x < 0 || x >= len || s.known[x] || !on_path(r, q)) continue;
    int c = 0, before = 0;
    for (int p = 0; p < nodes; ++p)
      if (token_of(p) == x && on_path(r, p)) ++c, before += p < q;
    if (!before && !banned(r, x)) patch(r, x, c, logit(r, x));
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
  if (a->V > 65535 * (int64_t)kSlice || a->R > 1 << 22) return SV_ERR_UNSUPPORTED;
  // Rows share a CTA's lists where there are CTAs enough without it; a small
  // call gives each row its own, so that rows do not wait for one another.
  const int64_t slices = (a->V + kSlice - 1) / kSlice, wanted = 2 * (int64_t)h->num_sms;
  int parts = (int)((wanted + slices * a->B - 1) / (slices * a->B));
  parts = parts < 1 ? 1 : parts > a->R ? a->R : parts;
  // a CTA counts rows x listed tokens and rows x drafted tokens in 32 bits
  const int most = (1 << 30) / (a->R > kSlice ? a->R : kSlice);
  int per = (a->R + parts - 1) / parts;
  per = per > most ? most : per;
  const dim3 grid((unsigned)a->B, (unsigned)slices, (unsigned)((a->R + per - 1) / per)), block(kRuleThreads);
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
