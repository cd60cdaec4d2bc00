// attention8.cu -- paged attention over the 8-bit cache, a simple form: a warp takes one
// (token, query head) and goes through its keys with a running maximum and sum.
#include "cache8.cuh"

namespace {

using gdn::AttnArgs;

struct Args8 {
  AttnArgs a;
  gdn::Cache8 cache;
  int32_t D;
};

template <int D>
__global__ void __launch_bounds__(128) simple_attention8_kernel(const Args8 d) {
  constexpr int E = D / 32;
  const AttnArgs& a = d.a;
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int t = static_cast<int>(id / a.Hq), h = static_cast<int>(id % a.Hq), head = h / a.group;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.paged.num_seqs; b += 128)
      if (gdn::seq_range(a.paged, b).refused) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_TABLE, b);
  if (t >= a.paged.total_tokens) return;
  gdn::SeqRange s = {};
  int b = t;
  if (a.paged.cu_seqlens) {
    for (b = 0; b < a.paged.num_seqs; ++b)
      if (a.paged.cu_seqlens[b] <= t && t < a.paged.cu_seqlens[b + 1]) break;
    if (b == a.paged.num_seqs) return;
  }
  s = gdn::seq_range(a.paged, b);
  if (!s.new_tokens) return;
  const int pos = s.len - s.new_tokens + t - s.first_token;
  const int full = a.full_lens ? min(a.full_lens[b], s.len) : 0;
  const int lo = gdn::key_lo(a, pos), hi = max(pos + 1, full);
  const float slope = a.slopes ? a.slopes[h] * gdn::kLog2e : 0.f;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  for (int i = 0; i < E; ++i) q[i] = __bfloat162float(a.q[t * a.q_stride + static_cast<int64_t>(h) * D + lane * E + i]), o[i] = 0.f;
  for (int j = lo; j < hi; ++j) {
    const int e = j / a.paged.page_size, slot = j % a.paged.page_size, page = a.paged.pages[s.entry + e];
    float k[E] = {}, v[E] = {};
    if (page >= 0 && page < a.paged.num_pages) {
      const int64_t at = page * d.cache.page_stride + slot * d.cache.token_stride + head * d.cache.head_stride + lane * E;
      const int64_t sc = page * d.cache.scale_page + slot / gdn::kGroup * d.cache.scale_group + head * d.cache.scale_head;
      const float ks = gdn::scale_of(d.cache.scales[0][sc]), vs = gdn::scale_of(d.cache.scales[1][sc]);
      for (int i = 0; i < E; ++i) {
        k[i] = gdn::half2_to_float2(gdn::e4m3_to_half2(d.cache.codes[0][at + i])).x * ks;
        v[i] = gdn::half2_to_float2(gdn::e4m3_to_half2(d.cache.codes[1][at + i])).x * vs;
      }
    } else if (lane == 0) {
      gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_ID, b);
    }
    float x = 0.f;
    for (int i = 0; i < E; ++i) x = fmaf(q[i], k[i], x);
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    x = a.cap_log2 > 0.f ? gdn::capped(x, a) : x * a.scale_log2;
    if (a.slopes) x -= slope * static_cast<float>(abs(pos - j));
    const float top = fmaxf(m, x), r = m == -INFINITY ? 0.f : gdn::exp2_approx(m - top), w = gdn::exp2_approx(x - top);
    m = top;
    l = l * r + w;
    for (int i = 0; i < E; ++i) o[i] = o[i] * r + w * v[i];
  }
  const int64_t row = static_cast<int64_t>(t) * a.Hq + h;
  for (int i = 0; i < E; ++i) a.o[row * D + lane * E + i] = __float2bfloat16(o[i] / l);
  if (a.lse && lane == 0) a.lse[row] = (m + log2f(l)) / gdn::kLog2e;
}

int attend(const gdn_bf16* q, int64_t q_stride, gdn_bf16* o, float* lse, const int32_t* cu, int32_t T, int32_t Hq,
           const gdn_kv_cache_fp8* cache, const gdn_page_table* table, float scale, const gdn_attention_options* options,
           void* workspace, size_t workspace_bytes, size_t need, int32_t* err_word, void* stream) {
  gdn_kv_cache shell;
  int rc = gdn_host::check_paged8(cache, table, cu, T, &shell);
  if (rc != GDN_OK) return rc;
  Args8 d = {};
  rc = gdn_host::attention_args(&d.a, q, q_stride, o, lse, cu, T, Hq, &shell, table, scale, options, workspace, workspace_bytes, need, err_word, 128);
  if (rc != GDN_OK || table->num_seqs == 0 || T == 0) return rc;
  rc = gdn_host::check_device(nullptr);
  if (rc != GDN_OK) return rc;
  d.cache = gdn_host::cache8(cache);
  const int64_t blocks = (static_cast<int64_t>(T) * Hq + 3) / 4;
  const dim3 grid(static_cast<unsigned>(blocks));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cache->head_dim == 64 ? gdn_host::launch_pdl(simple_attention8_kernel<64>, grid, dim3(128), 0, s, d)
                               : gdn_host::launch_pdl(simple_attention8_kernel<128>, grid, dim3(128), 0, s, d);
}

}  // namespace

extern "C" int gdn_attention_paged_fp8(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* o, float* lse,
                                       const int32_t* cu_seqlens, int32_t total_tokens, int32_t Hq,
                                       const gdn_kv_cache_fp8* cache, const gdn_page_table* table, float scale,
                                       const gdn_attention_options* options, void* workspace, size_t workspace_bytes, int32_t* err_word, void* stream) {
  return attend(q, q_token_stride, o, lse, cu_seqlens, total_tokens, Hq, cache, table, scale, options, workspace, workspace_bytes,
                cache && table ? gdn_attention_workspace_bytes(table->num_seqs, total_tokens, Hq, cache->num_heads, cache->head_dim, table->num_entries, cache->page_size) : 0, err_word, stream);
}
