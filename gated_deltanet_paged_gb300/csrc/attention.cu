// attention.cu -- softmax attention of new tokens over a paged key / value
// cache.  The simplest right kernel: one warp per (token, query head) walks
// the visible keys four at a time with a running maximum and sum in fp32.
#include <math.h>

#include "attention_common.cuh"

namespace {

using gdn::PagedTokens;
using gdn::SeqRange;

constexpr int kWarps = 4;
constexpr int kKeys = 4;
constexpr float kLog2e = gdn::kLog2e;

struct SimpleArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* o;
  float* lse;
  const __nv_bfloat16* k_cache;
  const __nv_bfloat16* v_cache;
  int64_t page_stride, slot_stride, head_stride;
  PagedTokens paged;
  int32_t Hq, group;
  float scale, softcap;
  const float* slopes;
  const int32_t* full_lens;
  int32_t window;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attention_simple_kernel(const SimpleArgs a) {
  constexpr int kE = D / 32;  // elements per lane
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x;
  const int h = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (h >= a.Hq) return;
  int b = t;
  if (a.paged.cu_seqlens) {
    b = 0;
    for (int step = 1 << 30; step; step >>= 1)
      if (b + step < a.paged.num_seqs && a.paged.cu_seqlens[b + step] <= t) b += step;
  }
  const SeqRange s = gdn::seq_range(a.paged, b);
  if (s.refused && lane == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_TABLE, b);
  const int i = t - s.first_token;
  if (i < 0 || i >= s.new_tokens) return;
  const int pos = s.len - s.new_tokens + i;
  const int lo = a.window >= 0 ? max(0, pos - a.window) : 0;
  const int hi = max(pos + 1, a.full_lens ? min(a.full_lens[b], s.len) : 0);
  float q[kE], acc[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    q[e] = __bfloat162float(a.q[t * a.q_stride + static_cast<int64_t>(h) * D + lane * kE + e]) * a.scale;
    acc[e] = 0.f;
  }
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f;
  const int64_t head = (h / a.group) * a.head_stride + lane * kE;
  for (int j0 = lo; j0 < hi; j0 += kKeys) {
    float x[kKeys], v[kKeys][kE];
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      const int j = j0 + u;
      x[u] = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) v[u][e] = 0.f;
      if (j >= hi) continue;
      const int page = a.paged.pages[s.entry + j / a.paged.page_size];
      if (page < 0 || page >= a.paged.num_pages) {
        if (lane == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_ID, b);
        continue;
      }
      const int64_t at = page * a.page_stride + (j % a.paged.page_size) * a.slot_stride + head;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        x[u] += q[e] * __bfloat162float(a.k_cache[at + e]);
        v[u][e] = __bfloat162float(a.v_cache[at + e]);
      }
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
#pragma unroll
      for (int w = 16; w; w >>= 1) x[u] += __shfl_xor_sync(0xFFFFFFFFu, x[u], w);
      if (a.softcap > 0.f) x[u] = a.softcap * tanhf(x[u] / a.softcap);
      x[u] -= slope * fabsf(static_cast<float>(pos - (j0 + u)));
      x[u] = j0 + u < hi ? x[u] * kLog2e : -INFINITY;
      top = fmaxf(top, x[u]);
    }
    const float r = exp2f(m - top);
    l *= r;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] *= r;
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      const float p = exp2f(x[u] - top);
      l += p;
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[e] += p * v[u][e];
    }
    m = top;
  }
  const int64_t out = static_cast<int64_t>(t) * a.Hq + h;
#pragma unroll
  for (int e = 0; e < kE; ++e) a.o[out * D + lane * kE + e] = __float2bfloat16(acc[e] / l);
  if (a.lse && lane == 0) a.lse[out] = (m + log2f(l)) / kLog2e;
}

int attend(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* o, float* lse, const int32_t* cu_seqlens,
           int32_t total_tokens, int32_t Hq, const gdn_kv_cache* cache, const gdn_page_table* table, float scale,
           const gdn_attention_options* options, const void* workspace, size_t workspace_bytes, size_t need,
           int32_t* err_word, void* stream) {
  int rc = gdn_host::check_paged(cache, table, cu_seqlens, total_tokens);
  if (rc != GDN_OK) return rc;
  const int32_t D = cache->head_dim, Hkv = cache->num_heads;
  if (Hq < 1 || Hq % Hkv != 0) return GDN_ERR_INVALID_ARGUMENT;
  if ((D != 64 && D != 128) || Hq / Hkv > 128) return GDN_ERR_UNSUPPORTED;
  if (options && !isfinite(options->softcap)) return GDN_ERR_INVALID_ARGUMENT;
  if (options && options->window >= 0 && options->full_lens) return GDN_ERR_UNSUPPORTED;
  if (table->num_seqs == 0 || total_tokens == 0) return GDN_OK;
  if (gdn_host::bad_tokens(q, q_token_stride, Hq, D) || !o || !gdn_host::aligned16(o) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return GDN_ERR_INVALID_ARGUMENT;
  if (!workspace || !gdn_host::aligned16(workspace) || workspace_bytes < need) return GDN_ERR_INVALID_ARGUMENT;
  rc = gdn_host::check_device(nullptr);
  if (rc != GDN_OK) return rc;
  SimpleArgs a = {};
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_token_stride;
  a.o = reinterpret_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.k_cache = reinterpret_cast<const __nv_bfloat16*>(cache->k);
  a.v_cache = reinterpret_cast<const __nv_bfloat16*>(cache->v);
  a.page_stride = cache->page_stride;
  a.slot_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.paged = gdn_host::paged_tokens(cache, table, cu_seqlens, total_tokens, err_word);
  a.Hq = Hq;
  a.group = Hq / Hkv;
  a.scale = scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(D));
  a.softcap = options ? options->softcap : 0.f;
  a.slopes = options ? options->slopes : nullptr;
  a.full_lens = options ? options->full_lens : nullptr;
  a.window = options ? options->window : -1;
  const dim3 grid(total_tokens, (Hq + kWarps - 1) / kWarps), block(kWarps * 32);
  return D == 64 ? gdn_host::launch_pdl(attention_simple_kernel<64>, grid, block, 0, static_cast<cudaStream_t>(stream), a)
                 : gdn_host::launch_pdl(attention_simple_kernel<128>, grid, block, 0, static_cast<cudaStream_t>(stream), a);
}

}  // namespace

extern "C" size_t gdn_attention_workspace_bytes(int32_t num_seqs, int32_t total_tokens, int32_t Hq, int32_t Hkv,
                                                int32_t D) {
  return num_seqs < 0 || total_tokens < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128) ? 0 : 16;
}

extern "C" int gdn_attention_paged(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* o, float* lse,
                                   const int32_t* cu_seqlens, int32_t total_tokens, int32_t Hq,
                                   const gdn_kv_cache* cache, const gdn_page_table* table, float scale,
                                   const gdn_attention_options* options, void* workspace, size_t workspace_bytes,
                                   int32_t* err_word, void* stream) {
  return attend(q, q_token_stride, o, lse, cu_seqlens, total_tokens, Hq, cache, table, scale, options, workspace,
                workspace_bytes, 16, err_word, stream);
}
