// attention8.cu -- softmax attention of a chunk of new tokens over the 8-bit cache.
//
// The kernel is that of attention.cu, but for the way of keys and values into shared
// memory: tiles of codes come by TMA into two tiles of their own, and the four epilogue
// warps turn them into bf16 (exactly: a code has 4 significant bits and its scale is a
// power of two) in the layout that the copies have there.  The products, the softmax and
// the outputs are bit for bit those over a 16-bit cache that holds the same values, but
// under a cap without slopes: such scores have a way of their own here, in which references
// move at other times.
//
// Bound: shared memory, then the tensor cores.  Per block of 128 keys and 256 rows at
// heads of 128 the products read 196 KB and the conversion moves 131 KB (codes in and
// out of it, bf16 back): 2,560 cycles at 128 bytes a cycle, where a 16-bit cache's copies
// make it 2,048 and the products take as long.  Measured: 3,500.
//
// Measured at 32 query heads on 8 key heads of 128: 4 prompts of 8,192 1.72 to 1.75 ms,
// 1,250 TFLOP/s, by way of a bf16 copy 1.31 to 1.36 in short runs and 1.40 to 1.48 in long
// ones; 64 mixed sequences, 16 heads, a cap of 30 and a window, 3.2 ms with scores that
// often pass the cap's polynomial and 2.8 without, by way of a copy 2.9 and 2.4.
#include "attention_chunk.cuh"

namespace {

template <int D, Scores kScores>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attention8_kernel(const __grid_constant__ ChunkArgs d, const __grid_constant__ CUtensorMap q_map,
                            const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                            const __grid_constant__ gdn::Cache8 codes) {
  chunk_attention<D, kScores, true, true>(d, q_map, k_map, v_map, codes);
}

template <int D, Scores kScores>
int launch(ChunkArgs d, int32_t total_tokens, const gdn_kv_cache_fp8* cache, void* workspace, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  CUtensorMap k_map, v_map;
  int rc;
  if ((rc = gdn_host::encode_codes_map(&k_map, cache->k, cache, d.a.box_shift)) != GDN_OK) return rc;
  if ((rc = gdn_host::encode_codes_map(&v_map, cache->v, cache, d.a.box_shift)) != GDN_OK) return rc;
  const auto kernel = chunk_attention8_kernel<D, kScores>;
  return launch_chunk<D, true>(kernel, d, total_tokens, done, workspace, sms, stream,
                         [&](dim3 grid, dim3 block, int smem, const CUtensorMap& q_map) {
                           return gdn_host::launch_pdl(kernel, grid, block, smem, stream, d, q_map, k_map, v_map, gdn_host::cache8(cache));
                         });
}

// Under a cap, over a bf16 copy: the scores as over the codes.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attention8_copied_kernel(const __grid_constant__ ChunkArgs d, const __grid_constant__ CUtensorMap q_map,
                                   const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  chunk_attention<D, kCapped, false, true>(d, q_map, k_map, v_map, gdn::Cache8{});
}

template <int D>
int launch_copied(ChunkArgs d, int32_t total_tokens, const gdn_kv_cache* cache, void* workspace, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  CUtensorMap k_map, v_map;
  int rc;
  if ((rc = gdn_host::encode_cache_map(&k_map, cache->k, cache, d.a.box_shift)) != GDN_OK) return rc;
  if ((rc = gdn_host::encode_cache_map(&v_map, cache->v, cache, d.a.box_shift)) != GDN_OK) return rc;
  const auto kernel = chunk_attention8_copied_kernel<D>;
  return launch_chunk<D, false>(kernel, d, total_tokens, done, workspace, sms, stream,
                                [&](dim3 grid, dim3 block, int smem, const CUtensorMap& q_map) {
                                  return gdn_host::launch_pdl(kernel, grid, block, smem, stream, d, q_map, k_map, v_map);
                                });
}

// A bf16 copy of what the batch sees, behind the workspace proper: the pages' numbers, then
// keys and values.  Written once and read by many rows it takes less time than the
// conversion of every block for every 256 rows.  At 32 query heads on 8, converted /
// copied: 2,048 rows per sequence (tokens times query heads per key head) 512 tokens over
// 8,000 80.6 / 77.3 us, over 131,072 799 / 744, 64 x 512 326 / 277; 8,192 rows 248 / 207; but
// 1,024 rows 49 / 55, 408 / 455, 133 / 127.  8 x 512 over 4,000: 250 / 245, under a cap 384 /
// 358; heads of 64 195 / 190, under a cap 322 / 327; 16 query heads on 4 of 64 108 / 112, under
// a cap 173 / 181 (with 4,096 rows 205 / 193 and 339 / 337).  Not for more than kCopyMost bytes.
// The host knows no more than the batch's averages, and the limit stands for sequences of
// one kind: where a few have most rows and the others most keys the copy may take longer
// (8,192 new tokens beside 15 single ones over 100,000, 16 query heads on 4: 0.79 / 1.43 ms;
// 4,096 beside 7 over 16,000, 32 on 8: 0.25 / 0.30; but 32,768 beside 60 over 16,000: 7.1 /
// 6.7).
constexpr int64_t kCopyRows = 2048;
constexpr size_t kCopyMost = size_t(4) << 30;
struct Copy {
  size_t base, pages, kv, total;  // offsets, and bytes; total 0: none
};
Copy copy_of(size_t base, int64_t num_seqs, int64_t total_tokens, int64_t Hq, int64_t Hkv, int64_t D, int64_t entries,
             int64_t page_size) {
  Copy c = {};
  if (total_tokens * (Hq / Hkv) < kCopyRows * num_seqs || entries < 1) return c;
  const auto rounded = [](size_t x) { return (x + 255) / 256 * 256; };
  c.base = rounded(base);
  c.pages = rounded(4 * static_cast<size_t>(entries));
  const double one = 2.0 * static_cast<double>(entries) * page_size * Hkv * D;  // bytes of keys
  if (2 * one > static_cast<double>(kCopyMost)) return Copy{};
  c.kv = static_cast<size_t>(one);
  c.total = c.base + c.pages + 2 * c.kv;
  return c;
}

}  // namespace

extern "C" int gdn_attention_paged_fp8(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* o, float* lse,
                                       const int32_t* cu_seqlens, int32_t total_tokens, int32_t Hq,
                                       const gdn_kv_cache_fp8* cache, const gdn_page_table* table, float scale,
                                       const gdn_attention_options* options, void* workspace, size_t workspace_bytes,
                                       int32_t* err_word, void* stream) {
  gdn_kv_cache shell;
  int rc = gdn_host::check_paged8(cache, table, cu_seqlens, total_tokens, &shell);
  if (rc != GDN_OK) return rc;
  ChunkArgs d = {};
  d.whole = whole_items(table->num_seqs, table->num_entries, cache->page_size);
  rc = gdn_host::attention_args(&d.a, q, q_token_stride, o, lse, cu_seqlens, total_tokens, Hq, &shell, table, scale,
                                options, workspace, workspace_bytes, workspace_bytes_of(cache->head_dim, d.whole),
                                err_word, kKeys);
  if (rc != GDN_OK || table->num_seqs == 0 || total_tokens == 0) return rc;
  int sms = 0;
  rc = gdn_host::check_device(&sms);
  if (rc != GDN_OK) return rc;
  const Copy copy = copy_of(workspace_bytes_of(cache->head_dim, d.whole), table->num_seqs, total_tokens, Hq, cache->num_heads,
                            cache->head_dim, table->num_entries, cache->page_size);
  const bool capped = d.a.cap_log2 > 0.f && !d.a.slopes;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  if (copy.total && workspace_bytes >= copy.total && (reinterpret_cast<uintptr_t>(ws) & 31u) == 0) {
    int32_t* const pages = reinterpret_cast<int32_t*>(ws + copy.base);
    gdn_bf16* const k = reinterpret_cast<gdn_bf16*>(ws + copy.base + copy.pages);
    gdn_bf16* const v = k + copy.kv / 2;
    rc = gdn_host::expand8(cache, d.a.paged, d.a.window, k, v, pages, sms, static_cast<cudaStream_t>(stream));
    if (rc != GDN_OK) return rc;
    const int64_t D = cache->head_dim, head = D * cache->page_size;
    const gdn_kv_cache whole = {k, v, table->num_entries, cache->page_size, cache->num_heads, cache->head_dim,
                                head * cache->num_heads, D, head};
    if (capped) {
      d.tile_tokens = kRows / d.a.group;
      d.a.paged.pages = pages;
      d.a.paged.num_pages = table->num_entries;
      const cudaStream_t on = static_cast<cudaStream_t>(stream);
      return D == 64 ? launch_copied<64>(d, total_tokens, &whole, workspace, sms, on)
                     : launch_copied<128>(d, total_tokens, &whole, workspace, sms, on);
    }
    gdn_page_table entries = *table;
    entries.page_indices = pages;
    return gdn_attention_paged(q, q_token_stride, o, lse, cu_seqlens, total_tokens, Hq, &whole, &entries, scale, options,
                               workspace, copy.base, err_word, stream);
  }
  d.tile_tokens = kRows / d.a.group;
  return by_scores(d.a, cache->head_dim, [&](auto dim, auto scores) {
    return launch<decltype(dim)::value, decltype(scores)::value>(d, total_tokens, cache, workspace, sms,
                                                                static_cast<cudaStream_t>(stream));
  });
}

extern "C" size_t gdn_attention_fp8_workspace_bytes(int32_t num_seqs, int32_t total_tokens, int32_t Hq, int32_t Hkv,
                                                    int32_t D, int32_t num_entries, int32_t page_size) {
  const size_t base = gdn_attention_workspace_bytes(num_seqs, total_tokens, Hq, Hkv, D, num_entries, page_size);
  if (num_seqs < 1 || num_entries < 1 || page_size < 1 || total_tokens < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 ||
      (D != 64 && D != 128))
    return base;
  const Copy copy = copy_of(base, num_seqs, total_tokens, Hq, Hkv, D, num_entries, page_size);
  return copy.total > base ? copy.total : base;
}
