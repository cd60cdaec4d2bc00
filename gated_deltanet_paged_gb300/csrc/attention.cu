// attention.cu -- softmax attention of a chunk of new tokens over a paged key /
// value cache, on the tcgen05 tensor cores.
//
// Mathematics: o = sum_j p_j v_j / sum_j p_j with p_j = 2^(x_j - m), x_j the
// score in units of log2 and m a running reference: m follows the maximum only
// when that has grown by more than 2^8, so that the accumulator is rescaled in
// few blocks (any m gives the same quotient; the weights stay below 256).
// Partial results (m, l, o) of disjoint key ranges join exactly.
//
// Bound: the tensor cores (4 D flops per visible pair and query head); for
// short chunks over long caches HBM.
//   - Rows of a product are (token, query head of the group) pairs: one key /
//     value head serves all its query heads at once, a chunk of few tokens still
//     fills rows, and K and V are read once per 128 rows rather than once per head.
//   - A CTA works on two tiles of 128 rows against the same 128-key blocks: while
//     the tensor core multiplies for one tile, a warpgroup takes the softmax of
//     the other.  S and O of both tiles fill the 512 columns of TMEM (D = 128); the
//     weights go back over the first half of their S as the A operand of P V.
//   - Warp roles: two softmax warpgroups (one row per thread, its 128 scores in
//     registers), two warps that issue the products, one that copies keys page by
//     page by TMA and one that copies values and clears those that no row may see,
//     and an epilogue warpgroup.
//   - The batch is one line of (sequence, token tile, key head) items, as long as
//     their key ranges, and each CTA takes an equal piece of it, cutting items
//     where the piece ends (as the decode kernel does); the line's prefix sums
//     have closed forms, so that every CTA finds its piece from the page table
//     itself.  A join kernel adds up the cut items.  Where items are few, each gets
//     CTAs to itself instead; where sequences are short, none is cut.
//
// Measured at 32 query heads on 8 key heads of 128 (4 D flops per visible pair): 4
// prompts of 8,192 1.32 to 1.36 ms in short runs, 1,620 to 1,660 TFLOP/s, and 1.55 ms
// (1,420) in long ones under the power limit, where a library matrix product falls
// from 1,852 to 1,725; the tensor pipe is active for 80% of the cycles, and what is
// left are the turns of the two tiles and the items' ends.  512 tokens over 131,072
// 610 us, 1,810 TFLOP/s; 16 over 131,072 95 us, 5.6 TB/s.  Heads of 64 1.08 ms (1,020
// TFLOP/s), a distance bias 1.69 ms (1,300), a cap of 30 1.86 ms (1,180): there the
// softmax takes longer than the products, at 0.5 instructions per cycle; four warps
// per scheduler instead of two, half a row each, issue no more.  Windows of 128 /
// 1,024 / 4,096 222 / 478 / 1,072 us: an item of one or two blocks is mostly its own
// fixed cost.  The shortest calls, 9 us, are launch and one block's latency.
#include "attention_chunk.cuh"

namespace {

template <int D, Scores kScores>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attention_kernel(const __grid_constant__ ChunkArgs d, const __grid_constant__ CUtensorMap q_map,
                           const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  chunk_attention<D, kScores, false, false>(d, q_map, k_map, v_map, gdn::Cache8{});
}

template <int D, Scores kScores>
int launch(ChunkArgs d, int32_t total_tokens, const gdn_kv_cache* cache, void* workspace, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  CUtensorMap k_map, v_map;
  int rc;
  if ((rc = gdn_host::encode_cache_map(&k_map, cache->k, cache, d.a.box_shift)) != GDN_OK) return rc;
  if ((rc = gdn_host::encode_cache_map(&v_map, cache->v, cache, d.a.box_shift)) != GDN_OK) return rc;
  const auto kernel = chunk_attention_kernel<D, kScores>;
  return launch_chunk<D, false>(kernel, d, total_tokens, done, workspace, sms, stream,
                         [&](dim3 grid, dim3 block, int smem, const CUtensorMap& q_map) {
                           return gdn_host::launch_pdl(kernel, grid, block, smem, stream, d, q_map, k_map, v_map);
                         });
}

}  // namespace

extern "C" size_t gdn_attention_workspace_bytes(int32_t num_seqs, int32_t total_tokens, int32_t Hq, int32_t Hkv,
                                                int32_t D, int32_t num_entries, int32_t page_size) {
  if (num_seqs < 0 || num_entries < 0 || page_size < 1 || total_tokens < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
  return workspace_bytes_of(D, whole_items(num_seqs, num_entries, page_size));
}

extern "C" int gdn_attention_paged(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* o, float* lse,
                                   const int32_t* cu_seqlens, int32_t total_tokens, int32_t Hq,
                                   const gdn_kv_cache* cache, const gdn_page_table* table, float scale,
                                   const gdn_attention_options* options, void* workspace, size_t workspace_bytes,
                                   int32_t* err_word, void* stream) {
  ChunkArgs d = {};
  d.whole = cache && table && whole_items(table->num_seqs, table->num_entries, cache->page_size);
  const size_t need = cache ? workspace_bytes_of(cache->head_dim, d.whole) : 0;
  int rc = gdn_host::attention_args(&d.a, q, q_token_stride, o, lse, cu_seqlens, total_tokens, Hq, cache, table, scale,
                                    options, workspace, workspace_bytes, need, err_word, kKeys);
  if (rc != GDN_OK || table->num_seqs == 0 || total_tokens == 0) return rc;
  int sms = 0;
  rc = gdn_host::check_device(&sms);
  if (rc != GDN_OK) return rc;
  d.tile_tokens = kRows / d.a.group;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return by_scores(d.a, cache->head_dim, [&](auto dim, auto scores) {
    return launch<decltype(dim)::value, decltype(scores)::value>(d, total_tokens, cache, workspace, sms, s);
  });
}
