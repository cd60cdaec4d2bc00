// rope.cu -- rotary positions, and the append of keys and values to a paged
// cache with the rotation applied on the way.
//
// Mathematics.  Pair i of a head's rotated dimensions at position p turns by
// the angle 2 pi p f_i / 2^64 with f_i a whole number: the product modulo 2^64
// is three integer multiplies, its top 32 bits are the angle in 2^-32 turns,
// and sincospif of that half-turn count is the whole evaluation -- no range
// reduction, and no position at which the angle loses bits (a 32-bit float
// product p * theta is off by 0.016 radians at p = 262,144).
//
// Bound: HBM, 4 bytes moved per element (2 read, 2 written); every element is
// touched once.  A warp owns one token (or a slice of its heads): its lanes
// first evaluate the token's sines and cosines once, into shared memory, and
// then stream heads, each lane moving the two 16-byte pieces that hold its
// eight pairs.  Evaluating them per head instead would cost ~10 instructions
// per element moved, above the memory time.
//
// Measured: 65,536 tokens of 40 heads of 128 (1.34 GB moved) 196 us, 6.8 TB/s, the
// rate of a plain copy; an append of 8 ragged prompts (402 MB) 65 us, 6.2 TB/s; one
// token each of 256 sequences 4.7 us, 4 tokens 2.2 us, which are launch and latency.
#include <math.h>

#include "rotate.cuh"

namespace {

using gdn::kMaxPairs;
using gdn::PagedTokens;
using gdn::Piece;
using gdn::SeqRange;
using gdn_host::bad_rotation;
using gdn_host::bf;

constexpr int kWarps = 4;

// One kernel serves both calls: the heads of a token are Hq rotated query
// heads (src q, dst q_out), then Hkv rotated keys and Hkv copied values, both
// written to the token's cache slot.
struct RotateArgs {
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  int64_t q_stride, q_out_stride, k_stride, v_stride;         // per token
  int64_t page_stride, slot_stride, head_stride;              // cache
  const int32_t* positions;                                   // gdn_rope; nullptr: from the page table
  const int64_t* freq;                                        // nullptr: nothing is rotated
  PagedTokens paged;
  int32_t T, Hq, Hkv, D;
  int32_t half;         // rotated pairs (rotary_dim / 2; 0 without frequencies)
  int32_t units;        // lanes' pieces per head: D / (2 W)
  int32_t slices;       // warps per token
  int32_t interleaved;
  float sign;           // -1: inverse
  float amplitude;
};

constexpr int kBatch = 4;  // heads in flight per lane

template <int W>
__global__ void __launch_bounds__(kWarps * 32) rotate_kernel(const RotateArgs a) {
  __shared__ float2 cs_all[kWarps][kMaxPairs];
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int t = static_cast<int>(id / a.slices), slice = static_cast<int>(id % a.slices);
  if (t >= a.T) return;

  const int heads = a.Hq + 2 * a.Hkv;
  const int total = heads * a.units;
  const int stride = a.slices * 32;
  const int rotated = a.half / W;  // units that rotate; the rest are copied
  // Where unit `unit` of a head keeps its two pieces.
  auto offsets = [&](int unit, int* first, int* second) {
    if (unit < rotated && !a.interleaved) {
      *first = unit * W;
      *second = a.half + *first;
    } else {
      *first = unit * 2 * W;  // rotated units end at 2 * half, so copied ones follow on
      *second = *first + W;
    }
  };
  Piece<W> pa[kBatch], pb[kBatch];
  auto load = [&](int u0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int u = u0 + j * stride;
      if (u >= total) continue;
      const int h = u / a.units;
      int first, second;
      offsets(u - h * a.units, &first, &second);
      const __nv_bfloat16* src;
      if (h < a.Hq)
        src = a.q + t * a.q_stride + static_cast<int64_t>(h) * a.D;
      else if (h < a.Hq + a.Hkv)
        src = a.k + t * a.k_stride + static_cast<int64_t>(h - a.Hq) * a.D;
      else
        src = a.v + t * a.v_stride + static_cast<int64_t>(h - a.Hq - a.Hkv) * a.D;
      pa[j] = gdn::load_piece<W>(src + first);
      pb[j] = gdn::load_piece<W>(src + second);
    }
  };
  // The first heads and the frequencies are asked for before the position: finding
  // that takes up to four loads that wait for one another.
  int u0 = slice * 32 + lane;
  load(u0);
  int64_t freq[kMaxPairs / 32];
#pragma unroll
  for (int i = 0; i < kMaxPairs / 32; ++i)
    if (lane + 32 * i < a.half) freq[i] = a.freq[lane + 32 * i];

  int position;
  int64_t slot = -1;  // element offset of the token's cache slot
  if (a.positions) {
    position = a.positions[t];
  } else {
    const int b = a.paged.cu_seqlens ? gdn::find_sequence(a.paged.cu_seqlens, a.paged.num_seqs, t) : t;
    const SeqRange s = gdn::seq_range(a.paged, b);
    const int i = t - s.first_token;
    if (s.refused) {
      if (lane == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_TABLE, b);
      return;
    }
    if (i < 0 || i >= s.new_tokens) return;  // a token of no sequence
    position = s.len - s.new_tokens + i;
    const int page = a.paged.pages[s.entry + position / a.paged.page_size];
    if (page < 0 || page >= a.paged.num_pages) {
      if (lane == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_ID, b);
    } else {
      slot = page * a.page_stride + (position % a.paged.page_size) * a.slot_stride;
    }
  }

  float2* cs = cs_all[warp];
#pragma unroll
  for (int i = 0; i < kMaxPairs / 32; ++i) {
    if (lane + 32 * i >= a.half) break;
    cs[lane + 32 * i] = gdn::pair_turn(position, freq[i], a.amplitude, a.sign);
  }
  __syncwarp();

  while (u0 < total) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int u = u0 + j * stride;
      if (u >= total) continue;
      const int h = u / a.units, unit = u - h * a.units;
      int first, second;
      offsets(unit, &first, &second);
      __nv_bfloat16* dst;
      bool turns = unit < rotated;
      if (h < a.Hq) {
        dst = a.q_out + t * a.q_out_stride + static_cast<int64_t>(h) * a.D;
      } else {
        if (slot < 0) continue;
        const bool is_v = h >= a.Hq + a.Hkv;
        dst = (is_v ? a.v_cache : a.k_cache) + slot + (h - a.Hq - (is_v ? a.Hkv : 0)) * a.head_stride;
        turns = turns && !is_v;
      }
      if (turns) gdn::rotate<W>(pa[j], pb[j], cs + unit * W, a.interleaved != 0);
      gdn::store_piece<W>(dst + first, pa[j]);
      gdn::store_piece<W>(dst + second, pb[j]);
    }
    u0 += kBatch * stride;
    load(u0);
  }
}

int launch_rotate(RotateArgs a, cudaStream_t stream) {
  const int W = gdn_host::piece_width(a.half, a.D);
  a.units = a.D / (2 * W);
  const int64_t iterations = (static_cast<int64_t>(a.Hq + 2 * a.Hkv) * a.units + 31) / 32;
  // One warp per token where that fills the GPU (it evaluates the sines once
  // for all heads); with fewer tokens the heads are spread over more warps (40
  // heads of 128, 1 / 300 / 1,000 / 4,000 tokens: 2.5 / 4.3 / 6.6 / 14.7 us; with
  // one warp per token always 7.0 / 7.0 / 7.6 / 14.9, with four times as many
  // warps 2.5 / 3.7 / 7.0 / 16.2, with a quarter 2.7 / 4.5 / 8.8 / 17.4).
  const int64_t want = 152 * 16;
  int64_t slices = a.T >= want ? 1 : (want + a.T - 1) / a.T;
  if (slices > iterations) slices = iterations;
  a.slices = static_cast<int32_t>(slices);
  const int64_t blocks = (static_cast<int64_t>(a.T) * slices + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFF) return GDN_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kWarps * 32);
  switch (W) {
    case 8: return gdn_host::launch_pdl(rotate_kernel<8>, grid, block, 0, stream, a);
    case 4: return gdn_host::launch_pdl(rotate_kernel<4>, grid, block, 0, stream, a);
    case 2: return gdn_host::launch_pdl(rotate_kernel<2>, grid, block, 0, stream, a);
    default: return gdn_host::launch_pdl(rotate_kernel<1>, grid, block, 0, stream, a);
  }
}

}  // namespace

extern "C" int gdn_rope_frequencies(int32_t rotary_dim, double base, double factor, double original_len,
                                    double low_turns, double high_turns, int64_t* out) {
  if (!out || rotary_dim <= 0 || rotary_dim % 2 != 0 || !(base >= 1.0) || !isfinite(base) || !(factor >= 1.0) ||
      !isfinite(factor) || !isfinite(original_len))
    return GDN_ERR_INVALID_ARGUMENT;
  if (original_len > 0 && !(high_turns > low_turns)) return GDN_ERR_INVALID_ARGUMENT;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    double theta = pow(base, -2.0 * i / rotary_dim);
    double keep = 0.0;
    if (original_len > 0) {
      keep = (original_len * theta / kTwoPi - low_turns) / (high_turns - low_turns);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
    }
    theta = theta * keep + theta / factor * (1.0 - keep);
    // theta <= 1 radian per position, so the turns stay below 0.16 and fit.
    out[i] = static_cast<int64_t>(ldexp(theta / kTwoPi, 64));
  }
  return GDN_OK;
}

extern "C" int gdn_rope(const gdn_bf16* x, int64_t x_token_stride, gdn_bf16* y, int64_t y_token_stride,
                        const int32_t* positions, const int64_t* frequencies, int32_t total_tokens, int32_t H,
                        int32_t D, int32_t rotary_dim, int32_t interleaved, int32_t inverse, float amplitude,
                        void* stream) {
  if (total_tokens < 0 || H < 1 || D < 8 || D % 8 != 0 || !frequencies || bad_rotation(frequencies, rotary_dim, D, amplitude))
    return GDN_ERR_INVALID_ARGUMENT;
  if (total_tokens == 0) return GDN_OK;
  if (!positions || gdn_host::bad_tokens(x, x_token_stride, H, D) || gdn_host::bad_tokens(y, y_token_stride, H, D))
    return GDN_ERR_INVALID_ARGUMENT;
  if (x == y && x_token_stride != y_token_stride) return GDN_ERR_INVALID_ARGUMENT;
  const int rc = gdn_host::check_device(nullptr);
  if (rc != GDN_OK) return rc;
  RotateArgs a = {};
  a.q = bf(x);
  a.q_out = bf(y);
  a.q_stride = x_token_stride;
  a.q_out_stride = y_token_stride;
  a.positions = positions;
  a.freq = frequencies;
  a.T = total_tokens;
  a.Hq = H;
  a.D = D;
  a.half = rotary_dim / 2;
  a.interleaved = interleaved;
  a.sign = inverse ? -1.f : 1.f;
  a.amplitude = amplitude;
  return launch_rotate(a, static_cast<cudaStream_t>(stream));
}

extern "C" int gdn_kv_append_paged(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* q_out, const gdn_bf16* k,
                                   int64_t k_token_stride, const gdn_bf16* v, int64_t v_token_stride,
                                   const int32_t* cu_seqlens, int32_t total_tokens, int32_t Hq,
                                   const gdn_kv_cache* cache, const gdn_page_table* table,
                                   const int64_t* frequencies, int32_t rotary_dim, int32_t interleaved,
                                   float amplitude, int32_t* err_word, void* stream) {
  int rc = gdn_host::check_paged(cache, table, cu_seqlens, total_tokens);
  if (rc != GDN_OK) return rc;
  const int32_t D = cache->head_dim, Hkv = cache->num_heads;
  if (Hq < 0 || bad_rotation(frequencies, rotary_dim, D, amplitude)) return GDN_ERR_INVALID_ARGUMENT;
  if (table->num_seqs == 0 || total_tokens == 0) return GDN_OK;
  if ((Hq > 0) != (q != nullptr) || (Hq > 0) != (q_out != nullptr)) return GDN_ERR_INVALID_ARGUMENT;
  if (gdn_host::bad_tokens(k, k_token_stride, Hkv, D) || gdn_host::bad_tokens(v, v_token_stride, Hkv, D))
    return GDN_ERR_INVALID_ARGUMENT;
  if (Hq > 0 && (gdn_host::bad_tokens(q, q_token_stride, Hq, D) || !gdn_host::aligned16(q_out) ||
                 (q == q_out && q_token_stride != static_cast<int64_t>(Hq) * D)))
    return GDN_ERR_INVALID_ARGUMENT;
  rc = gdn_host::check_device(nullptr);
  if (rc != GDN_OK) return rc;
  RotateArgs a = {};
  a.q = bf(q);
  a.q_out = bf(q_out);
  a.k = bf(k);
  a.v = bf(v);
  a.k_cache = bf(cache->k);
  a.v_cache = bf(cache->v);
  a.q_stride = q_token_stride;
  a.q_out_stride = static_cast<int64_t>(Hq) * D;
  a.k_stride = k_token_stride;
  a.v_stride = v_token_stride;
  a.page_stride = cache->page_stride;
  a.slot_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.freq = frequencies;
  a.paged = gdn_host::paged_tokens(cache, table, cu_seqlens, total_tokens, err_word);
  a.T = total_tokens;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.half = rotary_dim / 2;
  a.interleaved = interleaved;
  a.sign = 1.f;
  a.amplitude = amplitude;
  return launch_rotate(a, static_cast<cudaStream_t>(stream));
}
