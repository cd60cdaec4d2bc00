// attention_common.cuh -- page-table reading shared by the attention layer's
// kernels (rope.cu, attention.cu, attention_decode.cu) and their host checks.
#pragma once

#include <math.h>

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

constexpr float kLog2e = 1.4426950408889634f;

// What both attention kernels take.  Scores are kept in units of log2, so that
// every exponential is one exp2.
struct AttnArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* o;
  float* lse;  // nullptr: not wanted
  PagedTokens paged;
  int32_t Hq, Hkv, group;
  float scale_log2;           // scale * log2(e)
  float cap_log2;             // cap * log2(e), 0: no cap
  float cap_unit;             // scale / cap: the tanh's argument is u = score * cap_unit
  float cap_poly[5];          // log2(e) * scale * tanh(u) / u as a polynomial in score^2 ...
  float cap_near;             // ... for scores up to this
  const float* slopes;        // [Hq] or nullptr
  const int32_t* full_lens;   // [num_seqs] or nullptr
  int32_t window;             // < 0: none
  int32_t box_shift;          // log2 of the tokens per copy of a page
  uint32_t wait_ns;           // limit of the waits
  int32_t debug_stall;        // test hook (gdn_debug_set_wait_stall): a wait that runs out
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bounded wait of a whole warp: its lanes go on, or give up, together (a lane that
// gave up alone would leave the others at the next instruction that takes all 32).
// In line: with a function call in the chunk kernel its register split cannot be
// allocated.
// It gives up after limit_ns, or when *abort is set (nullptr: never).
__device__ __forceinline__ bool warp_wait_more(uint64_t* bar, uint32_t parity, const volatile int* abort, uint32_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    const bool there = mbar_try_wait_suspend(bar, parity);
    if (__all_sync(0xFFFFFFFFu, there)) return true;
    const bool out = (abort && *abort != 0) || globaltimer_ns() - t0 > limit_ns;
    if (__any_sync(0xFFFFFFFFu, out)) return false;
  }
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort, uint32_t limit_ns) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  return warp_wait_more(bar, parity, abort, limit_ns);
}

// The same of one lane, which alone goes on or takes a vote after it.
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, const volatile int* abort, uint32_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_suspend(bar, parity))
    if (*abort || globaltimer_ns() - t0 > limit_ns) return false;
  return true;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * tanh(u), u = s * scale / cap, in units of log2.
//   |u| <= 0.75: s * scale * log2(e) * (tanh(u) / u), the quotient as a polynomial in
//     u^2 (kCapPoly).  Its error is relative to the score, 5.7e-7, so that a cap
//     far above the scores leaves them as they are.
//   else: cap * (1 - 2 / (e^(2 u) + 1)), off by about 2^-23 of the cap, which is 2^-22
//     of the result there, and exact at the ends (e^(2 u) overflows to infinity or
//     vanishes).
// The hardware tanh is off by 2^-11 of the cap, a weight error of 1 percent under
// one of 30.
constexpr float kCapNear = 0.75f;
// tanh(u) / u for |u| <= 0.75 as a polynomial in u^2, fitted by least squares on
// Chebyshev nodes reweighted towards the minimax error (5.7e-07 relative).
constexpr double kCapPoly[5] = {0.9999994349237419, -0.3332825153150915, 0.1325898321214035, -0.05005630243018433, 0.0129296321851392};

// |s| <= cap_near, two scores on the FMA pipe alone: six operations a pair, where the
// exponential form takes three trips a score through the special function unit.
// (Seven, with u^2 instead of s^2 as the variable: 4 x 8,192 tokens 1.97 ms, 1.87 so.)
struct CapPoly {
  float2 c[5];
  __device__ __forceinline__ explicit CapPoly(const AttnArgs& a) {
#pragma unroll
    for (int i = 0; i < 5; ++i) c[i] = make_float2(a.cap_poly[i], a.cap_poly[i]);
  }
};
__device__ __forceinline__ float2 near_quotient(float2 s, const CapPoly& p) {
  const float2 t = __fmul2_rn(s, s);
  float2 h = __ffma2_rn(p.c[4], t, p.c[3]);
  h = __ffma2_rn(h, t, p.c[2]);
  h = __ffma2_rn(h, t, p.c[1]);
  return __ffma2_rn(h, t, p.c[0]);
}
__device__ __forceinline__ float2 capped_near(float2 s, const CapPoly& p) { return __fmul2_rn(s, near_quotient(s, p)); }
// ... and less a reference, at no further cost.
__device__ __forceinline__ float2 capped_near(float2 s, const CapPoly& p, float2 minus) {
  return __ffma2_rn(s, near_quotient(s, p), minus);
}
// The same for one score, rounding by rounding: a score has the same bits whichever
// of these functions took it, so that what decides between them shows nowhere.
__device__ __forceinline__ float capped_near(float s, const AttnArgs& a) {
  const float t = __fmul_rn(s, s);
  float h = fmaf(a.cap_poly[4], t, a.cap_poly[3]);
  h = fmaf(h, t, a.cap_poly[2]);
  h = fmaf(h, t, a.cap_poly[1]);
  h = fmaf(h, t, a.cap_poly[0]);
  return __fmul_rn(s, h);
}
// Any score.
__device__ __forceinline__ float capped(float s, const AttnArgs& a) {
  const float u = s * a.cap_unit, t = u * u;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(exp2_approx(u * (2.f * kLog2e)) + 1.f));
  float x = fmaf(-2.f * a.cap_log2, r, a.cap_log2);
  constexpr float c0 = kCapPoly[0], c1 = kCapPoly[1], c2 = kCapPoly[2], c3 = kCapPoly[3], c4 = kCapPoly[4];
  const float h = fmaf(fmaf(fmaf(fmaf(c4, t, c3), t, c2), t, c1), t, c0);
  if (fabsf(u) <= kCapNear) x = s * a.scale_log2 * h;
  if (fabsf(s) <= a.cap_near) x = capped_near(s, a);
  return x;
}

// A line of `total` units in equal pieces for `eff` CTAs: piece c is [start(c),
// start(c + 1)).  Any monotone boundaries do, so a product in floats replaces the
// 64-bit division, in steps of 2^shift units (doubles took 3,400 cycles here, with
// every thread of the CTA at the few FP64 units): this runs at the head of every
// CTA, where time counts in small calls.  No piece is empty: eff is chosen so
// that a piece is some steps long at least.
template <int kShift>
struct Shares {
  int64_t total;
  float per;  // steps
  int eff, shift;
  __device__ __forceinline__ Shares(int64_t units, int64_t most, int grid) {
    total = units;
    eff = static_cast<int>(most < 1 ? 1 : most < grid ? most : grid);
    shift = units >> (kShift + 31) ? kShift + 14 : kShift;  // steps in 32 bits
    per = __fdividef(static_cast<float>(static_cast<int>(units >> shift)), static_cast<float>(eff));
  }
  __device__ __forceinline__ int64_t start(int c) const {
    return c >= eff ? total : min(static_cast<int64_t>(static_cast<int>(per * static_cast<float>(c))) << shift, total);
  }
  // The piece that holds unit x.
  __device__ __forceinline__ int owner(int64_t x) const {
    int c = min(static_cast<int>(__fdividef(static_cast<float>(static_cast<int>(x >> shift)), per)), eff - 1);
    while (c + 1 < eff && start(c + 1) <= x) ++c;
    while (start(c) > x) --c;
    return c;
  }
};
// floor(x / d) for 0 <= x < d * most, without a 64-bit division.
__device__ __forceinline__ int small_quotient(int64_t x, int d, int most) {
  int c = min(static_cast<int>(__fdividef(static_cast<float>(x), static_cast<float>(d))), most - 1);
  while (static_cast<int64_t>(c + 1) * d <= x) ++c;
  while (static_cast<int64_t>(c) * d > x) --c;
  return c;
}

// Keys that a token at `pos` sees: [lo, hi).
__device__ __forceinline__ int key_lo(const AttnArgs& a, int pos) { return a.window >= 0 ? max(0, pos - a.window) : 0; }

// Copies of one K or V tile after the other by a warp: lane i has box i of every
// tile.  Where its rows lie follows from tile to tile without a division, and
// their page is asked for a tile ahead.  (The instructions of these warps are
// rarely in the cache: with a lookup per tile the products waited for keys.)  A
// tile of more than 32 boxes, from pages of an odd or once even size, is looked
// up on the spot.
template <int D, int kKeys>
struct TileCopies {
  const AttnArgs& a;
  const CUtensorMap* map;
  int lane, boxes, box_rows, step_entries, step_slots;
  int lo, hi, head, seq;
  const int32_t* pages;
  int key0, entry, slot, page;

  __device__ __forceinline__ TileCopies(const AttnArgs& args, const CUtensorMap* m, int l) : a(args), map(m), lane(l) {
    boxes = kKeys >> a.box_shift;
    box_rows = 1 << a.box_shift;
    step_entries = kKeys / a.paged.page_size;
    step_slots = kKeys % a.paged.page_size;
  }
  __device__ __forceinline__ bool visible(int k) const { return k + box_rows > lo && k < hi; }
  __device__ __forceinline__ int page_of(int e) const {
    int p = pages[e];
    if (p < 0 || p >= a.paged.num_pages) {
      record_error(a.paged.err_word, GDN_DEVERR_PAGE_ID, seq);
      p = a.paged.num_pages;  // outside the map: zeros
    }
    return p;
  }
  __device__ __forceinline__ void look_ahead() {
    if (boxes <= 32 && lane < boxes && visible(key0 + lane * box_rows)) page = page_of(entry);
  }
  // From tile `first` on, for keys [from, to) of a head; table_entry: the first of the sequence.
  __device__ __forceinline__ void begin(int from, int to, int kv_head, int b, int table_entry, int first) {
    lo = from, hi = to, head = kv_head, seq = b;
    pages = a.paged.pages + table_entry;
    key0 = first;
    const int key = key0 + lane * box_rows;
    entry = key / a.paged.page_size;
    slot = key - entry * a.paged.page_size;
    look_ahead();
  }
  // Bytes of the boxes that hold a visible key; the others are not copied.
  __device__ __forceinline__ int bytes() const {
    const int first = max(0, lo - key0) >> a.box_shift;
    const int last = (min(kKeys, hi - key0) + box_rows - 1) >> a.box_shift;
    return (last - first) * box_rows * D * 2;
  }
  __device__ __forceinline__ void box(uint8_t* dst, uint64_t* bar, int i, int o, int p) const {
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      tma_load_4d(dst + c * (kKeys * 128) + i * box_rows * 128, map, bar, c * 64, head, o, p);
  }
  // The current tile; then on to the next of `more`.
  __device__ __forceinline__ void copy(uint8_t* dst, uint64_t* bar, bool more) {
    if (boxes <= 32) {
      if (lane < boxes && visible(key0 + lane * box_rows)) box(dst, bar, lane, slot, page);
    } else {
#pragma unroll 1
      for (int i = lane; i < boxes; i += 32) {
        const int k = key0 + i * box_rows;
        if (!visible(k)) continue;
        const int e = k / a.paged.page_size;
        box(dst, bar, i, k - e * a.paged.page_size, page_of(e));
      }
    }
    __syncwarp();
    key0 += kKeys;
    entry += step_entries;
    slot += step_slots;
    if (slot >= a.paged.page_size) slot -= a.paged.page_size, ++entry;
    if (more) look_ahead();
  }
};

}  // namespace gdn

namespace gdn_host {

// Checks of a page table and a cache that need no device data.
inline int check_paged(const gdn_kv_cache* c, const gdn_page_table* t, const int32_t* cu_seqlens, int32_t total_tokens) {
  if (!c || !t || !c->k || !c->v || !t->page_indptr) return GDN_ERR_INVALID_ARGUMENT;
  // An array without entries may be NULL, as an empty tensor's pointer is.
  if ((!t->page_indices && t->num_entries != 0) || (!t->last_page_len && t->num_seqs != 0)) return GDN_ERR_INVALID_ARGUMENT;
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

// Argument checks of the two attention calls, and their common arguments.
// tile_keys: keys per tile, a power of two; a copy moves the largest power of two
// of tokens that divides both a page and a tile.
inline int attention_args(gdn::AttnArgs* a, const gdn_bf16* q, int64_t q_stride, gdn_bf16* o, float* lse,
                          const int32_t* cu_seqlens, int32_t total_tokens, int32_t Hq, const gdn_kv_cache* cache,
                          const gdn_page_table* table, float scale, const gdn_attention_options* options,
                          const void* workspace, size_t workspace_bytes, size_t need, int32_t* err_word,
                          int tile_keys) {
  const int rc = check_paged(cache, table, cu_seqlens, total_tokens);
  if (rc != GDN_OK) return rc;
  const int32_t D = cache->head_dim, Hkv = cache->num_heads;
  if (Hq < 1 || Hq % Hkv != 0) return GDN_ERR_INVALID_ARGUMENT;
  if ((D != 64 && D != 128) || Hq / Hkv > 128) return GDN_ERR_UNSUPPORTED;
  const float cap = options ? options->softcap : 0.f;
  if (!(fabsf(cap) <= 3.0e38f) || scale != scale) return GDN_ERR_INVALID_ARGUMENT;
  if (options && options->window >= 0 && options->full_lens) return GDN_ERR_UNSUPPORTED;
  if (table->num_seqs == 0 || total_tokens == 0) return GDN_OK;
  if (bad_tokens(q, q_stride, Hq, D) || !o || !aligned16(o) || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return GDN_ERR_INVALID_ARGUMENT;
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return GDN_ERR_INVALID_ARGUMENT;
  *a = gdn::AttnArgs{};
  a->q = reinterpret_cast<const __nv_bfloat16*>(q);
  a->q_stride = q_stride;
  a->o = reinterpret_cast<__nv_bfloat16*>(o);
  a->lse = lse;
  a->paged = paged_tokens(cache, table, cu_seqlens, total_tokens, err_word);
  a->Hq = Hq;
  a->Hkv = Hkv;
  a->group = Hq / Hkv;
  const float s = scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(D));
  if (!(s <= 3.0e38f) || (cap > 0.f && !(2.f * s / cap * gdn::kLog2e <= 3.0e38f))) return GDN_ERR_INVALID_ARGUMENT;
  a->scale_log2 = s * gdn::kLog2e;
  if (cap > 0.f) {
    a->cap_log2 = cap * gdn::kLog2e;
    a->cap_unit = s / cap;
    // The polynomial in the score has the powers of cap_unit in its coefficients.
    // Those that leave the normal numbers (scale / cap below about 4e-5) are left out,
    // and it is used up to where they would weigh 2^-24 of the whole.
    constexpr double kUpTo[5] = {4e-4, 0.025, 0.1, 0.2, (1.0 - 1e-6) * gdn::kCapNear};
    const double k = static_cast<double>(s) / cap;
    double c[5], power = s * 1.4426950408889634;
    bool fits = true;
    for (int i = 0; i < 5; ++i, power *= k * k) {
      c[i] = gdn::kCapPoly[i] * power;
      fits = fits && fabs(c[i]) < 1e38;
    }
    int top = 4;
    while (top > 0 && fabs(c[top]) < 1.2e-38) --top;
    for (int i = 0; i <= top && fits; ++i) a->cap_poly[i] = static_cast<float>(c[i]);
    // Scores whose squares are finite.
    a->cap_near = fits ? static_cast<float>(fmin(kUpTo[top] / k, 1e19)) : -1.f;
  }
  a->slopes = options ? options->slopes : nullptr;
  a->full_lens = options ? options->full_lens : nullptr;
  // No sequence has 2^30 tokens, so that a larger window hides nothing; the kernels
  // add to distances in 32 bits.
  a->window = options && options->window < (1 << 30) ? options->window : -1;
  a->debug_stall = debug_wait_stall();
  a->wait_ns = a->debug_stall ? 1000000u : 2000000000u;
  while ((1 << a->box_shift) < tile_keys && cache->page_size % (2 << a->box_shift) == 0) ++a->box_shift;
  return GDN_OK;
}

// The longest sequence that a table can hold has every entry that the others do
// not need, where each has a page.  Beside sequences without any it can be longer
// (the calls are right all the same).
inline int64_t longest_sequence(int32_t num_seqs, int32_t num_entries, int32_t page_size) {
  return (static_cast<int64_t>(num_entries) - num_seqs + 1) * page_size;
}

// Tensor map of one cache array, {D, heads, slots, pages}, with boxes of 64
// dimensions of one head of 2^box_shift slots.  An axis of one entry may carry any
// stride; the map wants a multiple of 16 bytes.
inline int encode_cache_map(CUtensorMap* map, const gdn_bf16* base, const gdn_kv_cache* c, int box_shift) {
  const int64_t dims[4] = {c->head_dim, c->num_heads, c->page_size, c->num_pages};
  const int64_t strides[3] = {2 * (c->num_heads > 1 ? c->head_stride : c->head_dim),
                              2 * (c->page_size > 1 ? c->token_stride : c->head_dim),
                              2 * (c->num_pages > 1 ? c->page_stride : c->head_dim)};
  return encode_map_4d(map, base, dims, strides, 1, 1 << box_shift);
}

}  // namespace gdn_host
