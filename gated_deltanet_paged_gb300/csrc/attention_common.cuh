// attention_common.cuh -- page-table reading shared by the attention layer's
// kernels (rope.cu, attention.cu, attention_decode.cu) and their host checks.
#pragma once

#include "common.cuh"

namespace gdn {

// Device copy of gdn_page_table / gdn_kv_cache and the token ranges.
struct PagedTokens {
  const int32_t* cu_seqlens;  // nullptr: one new token per sequence
  const int32_t* pages;
  const int32_t* indptr;
  const int32_t* last_len;
  int32_t num_seqs;
  int32_t num_entries;
  int32_t num_pages;
  int32_t page_size;
  int32_t total_tokens;
  int32_t* err_word;
};

struct SeqRange {
  int32_t first_token;  // row of its first new token in q, k, v
  int32_t new_tokens;   // 0: nothing to do (none, or the sequence is refused)
  int32_t len;          // tokens with the new ones
  int32_t entry;        // its first entry of the page table
  bool refused;
};

// The range of sequence b, checked: a sequence that fails a check has no new
// tokens here, so no kernel reads or writes anything for it.
__device__ __forceinline__ SeqRange seq_range(const PagedTokens& p, int b) {
  SeqRange s;
  const int32_t t0 = p.cu_seqlens ? p.cu_seqlens[b] : b;
  const int32_t t1 = p.cu_seqlens ? p.cu_seqlens[b + 1] : b + 1;
  const int32_t i0 = p.indptr[b], i1 = p.indptr[b + 1];
  const int32_t lpl = p.last_len[b];
  const int64_t n = static_cast<int64_t>(t1) - t0;
  const int64_t pages = static_cast<int64_t>(i1) - i0;
  const int64_t len = (pages - 1) * p.page_size + lpl;
  s.first_token = t0;
  s.entry = i0;
  s.len = static_cast<int32_t>(len);
  s.new_tokens = static_cast<int32_t>(n);
  s.refused = n != 0 && (n < 0 || t0 < 0 || t1 > p.total_tokens || i0 < 0 || i1 > p.num_entries || pages < 1 ||
                         lpl < 1 || lpl > p.page_size || n > len || len > 0x3FFFFFFF);
  if (s.refused || n == 0) s.new_tokens = 0;
  return s;
}

}  // namespace gdn

namespace gdn_host {

// Checks of a page table and a cache that need no device data.
inline int check_paged(const gdn_kv_cache* c, const gdn_page_table* t, const int32_t* cu_seqlens, int32_t total_tokens) {
  if (!c || !t || !c->k || !c->v || !t->page_indices || !t->page_indptr || !t->last_page_len)
    return GDN_ERR_INVALID_ARGUMENT;
  if (t->num_seqs < 0 || t->num_entries < 0 || total_tokens < 0 || c->num_pages < 1 || c->page_size < 1 ||
      c->num_heads < 1 || c->head_dim < 8 || c->head_dim % 8 != 0)
    return GDN_ERR_INVALID_ARGUMENT;
  if (!cu_seqlens && total_tokens != t->num_seqs) return GDN_ERR_INVALID_ARGUMENT;
  if (!aligned16(c->k) || !aligned16(c->v)) return GDN_ERR_INVALID_ARGUMENT;
  if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0 || c->page_stride % 8 != 0 ||
      c->token_stride % 8 != 0 || c->head_stride % 8 != 0)
    return GDN_ERR_INVALID_ARGUMENT;
  // An axis of one entry may have any stride; the others advance by a head at least.
  if ((c->num_pages > 1 && c->page_stride < c->head_dim) || (c->page_size > 1 && c->token_stride < c->head_dim) ||
      (c->num_heads > 1 && c->head_stride < c->head_dim))
    return GDN_ERR_INVALID_ARGUMENT;
  return GDN_OK;
}

// A [T, H, D] tensor with dense heads: 16-byte aligned, token stride a multiple of 8 elements.
inline bool bad_tokens(const void* p, int64_t stride, int64_t H, int64_t D) {
  return !p || !aligned16(p) || stride < H * D || stride % 8 != 0;
}

inline gdn::PagedTokens paged_tokens(const gdn_kv_cache* c, const gdn_page_table* t, const int32_t* cu_seqlens,
                                     int32_t total_tokens, int32_t* err_word) {
  gdn::PagedTokens p;
  p.cu_seqlens = cu_seqlens;
  p.pages = t->page_indices;
  p.indptr = t->page_indptr;
  p.last_len = t->last_page_len;
  p.num_seqs = t->num_seqs;
  p.num_entries = t->num_entries;
  p.num_pages = c->num_pages;
  p.page_size = c->page_size;
  p.total_tokens = total_tokens;
  p.err_word = err_word;
  return p;
}

}  // namespace gdn_host
