// cache8.cu -- the 8-bit cache of the attention layer: norms of queries and keys
// with the rotation in the same pass, the append that quantises keys and values as it
// writes them, and reading them back.
//
// Mathematics.  y = x / sqrt(mean(x^2) + eps) * (offset + weight) per head, then the
// rotation of rope.cu, all in fp32 with one rounding at the end: to bf16 for queries,
// to e4m3 for keys.  A group of 16 tokens of a head has the scale 2^e with the least e
// for which its largest value is at most 448 * 2^e; e4m3 is a floating format, so
// that a power of two costs no significant bits and rounding goes wrong by 2^-4 of a
// value at most (down to 2^-6 of the scale; by 2^-10 of the scale below).
//
// Bound: HBM, every element is touched once: 4 bytes a query element (2 in, 2 out), 3
// a key's or value's.
//   - norm and rotation alone: a warp takes a token (or a slice of its heads),
//     evaluates the token's sines and cosines once and streams heads, D / 16 lanes a
//     head, 16 elements a lane.  The sum of squares goes over those lanes by shuffles.
//   - append: a CTA takes a group of 16 tokens of a sequence, which is what has a scale
//     in common, so that nothing is shared between CTAs; a warp takes all 16 rows of
//     a head at a time in registers, from the load to the codes, and finds the largest
//     by one reduction.  The group's sines and cosines are evaluated once for all
//     heads.
#include "cache8.cuh"
#include "rotate.cuh"

namespace {

using gdn::Cache8;
using gdn::kGroup;
using gdn::PagedTokens;
using gdn::Piece;
using gdn::SeqRange;
using gdn_host::bf;

struct NormRope {
  const __nv_bfloat16* q_weight;  // nullptr: no norm
  const __nv_bfloat16* k_weight;
  float eps, offset, inv_dim;
  const int64_t* freq;  // nullptr: nothing is rotated
  int32_t half;         // rotated pairs
  int32_t interleaved;
  float amplitude;
};

// Where unit `unit` of a head keeps its two pieces of W elements.
template <int W>
__device__ __forceinline__ void offsets(const NormRope& n, int unit, int* first, int* second) {
  if (unit * W < n.half && !n.interleaved) {
    *first = unit * W;
    *second = n.half + *first;
  } else {
    *first = unit * 2 * W;  // rotated units end at 2 * half, so the others follow on
    *second = *first + W;
  }
}
// Sines and cosines of a token in the order in which lanes read them, two pairs of a
// unit beside those of the next one: lanes of a head read 16 bytes each, side by side.
template <int W>
__device__ __forceinline__ int cs_at(int pair, int units) {
  if constexpr (W == 1) return pair;
  const int unit = pair / W, i = pair % W;
  return ((i >> 1) * units + unit) * 2 + (i & 1);
}
template <int W>
struct CsOf {
  const float2* cs;
  int unit, units;
  __device__ __forceinline__ float2 operator()(int i) const {
    if constexpr (W == 1) return cs[unit];
    return cs[((i >> 1) * units + unit) * 2 + (i & 1)];
  }
};

// A lane's part of a head: U units, lane `at` of `lanes` has units at, at + lanes, ...
template <int W, int U>
struct Part {
  float x[U][W], y[U][W];
  __device__ __forceinline__ void unpack(const Piece<W> (&a)[U], const Piece<W> (&b)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < W; ++i) x[u][i] = gdn::get<W>(a[u], i), y[u][i] = gdn::get<W>(b[u], i);
  }
  // Over the root mean square of the head, times the weights.  Lanes of units past the
  // head hold zeros.
  __device__ __forceinline__ void norm(const NormRope& n, const Piece<W> (&wa)[U], const Piece<W> (&wb)[U], int lanes) {
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < W; ++i) s = fmaf(x[u][i], x[u][i], fmaf(y[u][i], y[u][i], s));
    for (int o = lanes >> 1; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const float r = rsqrtf(fmaf(s, n.inv_dim, n.eps));
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        x[u][i] *= r * (gdn::get<W>(wa[u], i) + n.offset);
        y[u][i] *= r * (gdn::get<W>(wb[u], i) + n.offset);
      }
  }
};

// ------------------------------------------------------------------ norm and rotation
constexpr int kWarps = 4;
constexpr int kBatch = 4;   // heads in flight per lane
constexpr int kMaxDim = 256;

struct NormArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  const int32_t* positions;
  NormRope n;
  int32_t T, Hq, Hkv, D;
  int32_t units;   // per head: D / (2 W)
  int32_t lanes;   // per head, a power of two
  int32_t slices;  // warps per token
};

template <int W>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_kernel(const NormArgs a) {
  constexpr int U = W == 1 ? 4 : W == 2 ? 2 : 1;  // D / (2 W) <= 32 U
  __shared__ float2 cs_all[kWarps][kMaxDim / 2];
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int t = static_cast<int>(id / a.slices), slice = static_cast<int>(id % a.slices);
  if (t >= a.T) return;
  const int heads = a.Hq + a.Hkv, per = 32 / a.lanes;  // heads at a time
  const int at = lane & (a.lanes - 1), stride = a.slices * per;
  int first[U], second[U];
  bool mine[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    offsets<W>(a.n, at + u * a.lanes, &first[u], &second[u]);
    mine[u] = at + u * a.lanes < a.units;
  }
  Piece<W> pa[kBatch][U], pb[kBatch][U];
  auto load = [&](int h0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = h0 + j * stride;
      const __nv_bfloat16* src = h < a.Hq ? a.q + t * a.q_stride + static_cast<int64_t>(h) * a.D
                                          : a.k + t * a.k_stride + static_cast<int64_t>(h - a.Hq) * a.D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        pa[j][u] = pb[j][u] = Piece<W>{};
        if (h >= heads || !mine[u]) continue;
        pa[j][u] = gdn::load_piece<W>(src + first[u]);
        pb[j][u] = gdn::load_piece<W>(src + second[u]);
      }
    }
  };
  int h0 = slice * per + lane / a.lanes;
  load(h0);
  Piece<W> qa[U], qb[U], ka[U], kb[U];  // weights
#pragma unroll
  for (int u = 0; u < U; ++u) {
    qa[u] = qb[u] = ka[u] = kb[u] = Piece<W>{};
    if (!mine[u]) continue;
    qa[u] = gdn::load_piece<W>(a.n.q_weight + first[u]);
    qb[u] = gdn::load_piece<W>(a.n.q_weight + second[u]);
    if (!a.Hkv) continue;
    ka[u] = gdn::load_piece<W>(a.n.k_weight + first[u]);
    kb[u] = gdn::load_piece<W>(a.n.k_weight + second[u]);
  }
  float2* cs = cs_all[warp];
  const int position = a.n.half ? a.positions[t] : 0;
#pragma unroll
  for (int i = 0; i < kMaxDim / 64; ++i) {
    const int pair = lane + 32 * i;
    if (pair < a.n.half) cs[cs_at<W>(pair, a.units)] = gdn::pair_turn(position, a.n.freq[pair], a.n.amplitude, 1.f);
  }
  __syncwarp();
  // All lanes go through as many steps: the norm's shuffles take the whole warp.
  for (int base = slice * per; base < heads; base += kBatch * stride, h0 += kBatch * stride) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = h0 + j * stride;
      const bool is_k = h >= a.Hq;
      Part<W, U> p;
      p.unpack(pa[j], pb[j]);
      Piece<W> wa[U], wb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) wa[u] = is_k ? ka[u] : qa[u], wb[u] = is_k ? kb[u] : qb[u];
      p.norm(a.n, wa, wb, a.lanes);
      if (h >= heads) continue;
      __nv_bfloat16* dst = is_k ? a.k_out + t * a.k_out_stride + static_cast<int64_t>(h - a.Hq) * a.D
                                : a.q_out + t * a.q_out_stride + static_cast<int64_t>(h) * a.D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int unit = at + u * a.lanes;
        if (!mine[u]) continue;
        if (unit * W < a.n.half) gdn::turn<W>(p.x[u], p.y[u], CsOf<W>{cs, unit, a.units}, a.n.interleaved != 0);
        gdn::store_piece<W>(dst + first[u], gdn::pack<W>(p.x[u]));
        gdn::store_piece<W>(dst + second[u], gdn::pack<W>(p.y[u]));
      }
    }
    load(h0 + kBatch * stride);
  }
}

// ------------------------------------------------------------------ groups of a batch
// Group `slot` of the batch's new tokens.  Sequence b has the slots from
// cu_seqlens[b] / 16 + 2 b on: n new tokens touch n / 16 + 2 groups at most, so that
// every sequence finds room for its own (most leave one or two slots empty).  Without
// cu_seqlens, slot b is the group of sequence b's token.
struct Group {
  int seq;
  int rows0, rows1;      // its new tokens are rows [rows0, rows1) of 16; rows before are earlier tokens
  int64_t token;         // new token of row 0 (of rows0 and above)
  int position;          // of row 0
  int page;              // -1: out of range
  int slot;              // of row 0 within the page
};
__device__ __forceinline__ int first_slot(const int32_t* cu, int b) { return (cu[b] >> 4) + 2 * b; }

// Taken by a whole warp; false: nothing there.
__device__ __forceinline__ bool find_group(const PagedTokens& p, int slot, Group* g) {
  int b = slot, local = 0;
  if (p.cu_seqlens) {
    // The last sequence that begins at or before the slot.
    const int lane = threadIdx.x & 31;
    int lo = 0, n = p.num_seqs;
    while (n > 1) {
      const int step = (n + 31) / 32;
      const int at = lo + lane * step;
      const bool below = at < lo + n && first_slot(p.cu_seqlens, at) <= slot;
      const int k = max(__popc(__ballot_sync(0xFFFFFFFFu, below)) - 1, 0);
      n = min(step, lo + n - (lo + k * step));
      lo += k * step;
    }
    b = lo;
    local = slot - first_slot(p.cu_seqlens, b);
    if (local < 0) return false;
  }
  const SeqRange s = gdn::seq_range(p, b);
  if (!s.new_tokens) return false;
  const int first = s.len - s.new_tokens;
  const int64_t at = (first / kGroup + static_cast<int64_t>(local)) * kGroup;
  if (at >= s.len) return false;
  g->seq = b;
  g->position = static_cast<int>(at);
  g->rows0 = max(0, first - g->position);
  g->rows1 = min(kGroup, s.len - g->position);
  g->token = static_cast<int64_t>(s.first_token) + g->position - first;
  const int entry = g->position / p.page_size;
  g->page = p.pages[s.entry + entry];
  g->slot = g->position - entry * p.page_size;
  if (g->page < 0 || g->page >= p.num_pages) g->page = -1;
  return true;
}
// Slots of a call.
int64_t group_slots(const int32_t* cu_seqlens, int32_t num_seqs, int32_t total_tokens) {
  return cu_seqlens ? total_tokens / kGroup + 2 * static_cast<int64_t>(num_seqs) : num_seqs;
}
// Refused sequences, reported by one block behind all groups: some have no slot.
__device__ __forceinline__ void report_refused(const PagedTokens& p) {
  for (int b = threadIdx.x; b < p.num_seqs; b += blockDim.x)
    if (gdn::seq_range(p, b).refused) gdn::record_error(p.err_word, GDN_DEVERR_PAGE_TABLE, b);
}

// ----------------------------------------------------------------------------- append
constexpr int kAppendWarps = 8;

struct AppendArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  int64_t q_stride, k_stride, v_stride;
  Cache8 cache;
  PagedTokens paged;
  NormRope n;
  int32_t Hq, Hkv;
  int32_t groups;  // slots; block `groups` reports refused sequences
};

template <int W>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[W], float inv) {
  if constexpr (W == 1) {
    *p = static_cast<uint8_t>(gdn::to_e4m3(x[0] * inv, 0.f));
  } else {
    uint32_t r[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) r[i] = gdn::to_e4m3(x[2 * i] * inv, x[2 * i + 1] * inv);
    if constexpr (W == 2) *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(r[0]);
    if constexpr (W == 4) *reinterpret_cast<uint32_t*>(p) = r[0] | r[1] << 16;
    if constexpr (W == 8) *reinterpret_cast<uint2*>(p) = make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
  }
}

template <int D, int W>
__global__ void __launch_bounds__(kAppendWarps * 32) append8_kernel(const AppendArgs a) {
  constexpr int kUnits = D / (2 * W);
  constexpr int kLanes = kUnits < 32 ? kUnits : 32;  // per head
  constexpr int U = kUnits / kLanes;
  constexpr int kPer = 32 / kLanes;                  // heads or rows at a time
  constexpr int kSteps = kGroup / kPer;
  __shared__ alignas(16) float2 cs[kGroup][D / 2];
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  if (blockIdx.x == a.groups) {
    if (blockIdx.y == 0) report_refused(a.paged);
    return;
  }
  Group g;
  if (!find_group(a.paged, blockIdx.x, &g)) return;  // all threads alike
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, at = lane % kLanes;
  const int worker = blockIdx.y * kAppendWarps + warp, workers = gridDim.y * kAppendWarps;
  if (a.n.half) {
    for (int r = g.rows0 + warp; r < g.rows1; r += kAppendWarps)
      for (int pair = lane; pair < a.n.half; pair += 32)
        cs[r][cs_at<W>(pair, kUnits)] = gdn::pair_turn(g.position + r, a.n.freq[pair], a.n.amplitude, 1.f);
    __syncthreads();
  }
  int first[U], second[U];
#pragma unroll
  for (int u = 0; u < U; ++u) offsets<W>(a.n, at + u * kLanes, &first[u], &second[u]);
  const bool normed = a.n.q_weight != nullptr;
  auto weights = [&](const __nv_bfloat16* w, Piece<W> (&wa)[U], Piece<W> (&wb)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      wa[u] = wb[u] = Piece<W>{};
      if (!normed) continue;
      wa[u] = gdn::load_piece<W>(w + first[u]);
      wb[u] = gdn::load_piece<W>(w + second[u]);
    }
  };
  auto turned = [&](Part<W, U>& p, int row) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = at + u * kLanes;
      if (unit * W < a.n.half) gdn::turn<W>(p.x[u], p.y[u], CsOf<W>{cs[row], unit, kUnits}, a.n.interleaved != 0);
    }
  };

  // Queries: kPer heads of a row at a time.
  if (a.Hq) {
    Piece<W> wa[U], wb[U];
    weights(a.n.q_weight, wa, wb);
    const int per_row = (a.Hq + kPer - 1) / kPer, jobs = (g.rows1 - g.rows0) * per_row;
    for (int j0 = worker; j0 < jobs; j0 += kSteps * workers) {
      Piece<W> pa[kSteps][U], pb[kSteps][U];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int j = j0 + i * workers, row = g.rows0 + j / per_row, h = j % per_row * kPer + lane / kLanes;
        const __nv_bfloat16* src = a.q + (g.token + row) * a.q_stride + static_cast<int64_t>(h) * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          pa[i][u] = pb[i][u] = Piece<W>{};
          if (j >= jobs || h >= a.Hq) continue;
          pa[i][u] = gdn::load_piece<W>(src + first[u]);
          pb[i][u] = gdn::load_piece<W>(src + second[u]);
        }
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int j = j0 + i * workers, row = g.rows0 + j / per_row, h = j % per_row * kPer + lane / kLanes;
        if (j >= jobs) break;
        Part<W, U> p;
        p.unpack(pa[i], pb[i]);
        if (normed) p.norm(a.n, wa, wb, kLanes);
        turned(p, row);
        if (h >= a.Hq) continue;
        __nv_bfloat16* dst = a.q_out + ((g.token + row) * a.Hq + h) * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          gdn::store_piece<W>(dst + first[u], gdn::pack<W>(p.x[u]));
          gdn::store_piece<W>(dst + second[u], gdn::pack<W>(p.y[u]));
        }
      }
    }
  }

  if (g.page < 0) {
    if (worker == 0 && lane == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_ID, g.seq);
    return;
  }
  // Keys and values: all rows of a head at a time.
  Piece<W> wa[U], wb[U];
  weights(a.n.k_weight, wa, wb);
  for (int item = worker; item < 2 * a.Hkv; item += workers) {
    const bool is_k = item < a.Hkv;
    const int h = is_k ? item : item - a.Hkv;
    const __nv_bfloat16* src = (is_k ? a.k : a.v) + static_cast<int64_t>(h) * D;
    const int64_t stride = is_k ? a.k_stride : a.v_stride;
    uint8_t* codes = a.cache.codes[is_k ? 0 : 1] + g.page * a.cache.page_stride + g.slot * a.cache.token_stride +
                     h * a.cache.head_stride;
    uint8_t* scale = a.cache.scales[is_k ? 0 : 1] + g.page * a.cache.scale_page +
                     g.slot / kGroup * a.cache.scale_group + h * a.cache.scale_head;
    const uint32_t before = g.rows0 > 0 ? *scale : 0u;  // earlier tokens' scale
    Piece<W> pa[kSteps][U], pb[kSteps][U];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = i * kPer + lane / kLanes;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        pa[i][u] = pb[i][u] = Piece<W>{};
        if (row < g.rows0 || row >= g.rows1) continue;
        pa[i][u] = gdn::load_piece<W>(src + (g.token + row) * stride + first[u]);
        pb[i][u] = gdn::load_piece<W>(src + (g.token + row) * stride + second[u]);
      }
    }
    Part<W, U> p[kSteps];
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = i * kPer + lane / kLanes;
      const bool there = row >= g.rows0 && row < g.rows1;
      p[i].unpack(pa[i], pb[i]);
      if (is_k) {
        if (normed) p[i].norm(a.n, wa, wb, kLanes);
        if (there) turned(p[i], row);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < W; ++k) most = fmaxf(most, fmaxf(fabsf(p[i].x[u][k]), fabsf(p[i].y[u][k])));
    }
    // Numbers that are not negative compare as their bits do.  448 = 1.75 * 2^8.
    const uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
    const int least = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    const uint32_t byte = max(static_cast<uint32_t>(min(max(least, gdn::kScaleLeast), gdn::kScaleMost)), before);
    const float inv = __uint_as_float((254u - min(byte, 253u)) << 23);
    __syncwarp();  // every lane has read the scale
    if (lane == 0) *scale = static_cast<uint8_t>(byte);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = i * kPer + lane / kLanes;
      if (row < g.rows0 || row >= g.rows1) continue;
      uint8_t* dst = codes + row * a.cache.token_stride;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        store_codes<W>(dst + first[u], p[i].x[u], inv);
        store_codes<W>(dst + second[u], p[i].y[u], inv);
      }
    }
    if (g.rows0 > 0 && byte > before) {
      // Earlier tokens' codes, rounded to the scale that has grown (by 2^-126 all of
      // them become zero, as by less).
      const float by = __uint_as_float(max(127 - static_cast<int>(byte - before), 1) << 23);
      for (int i = lane; i < g.rows0 * (D / 16); i += 32) {
        uint4* x = reinterpret_cast<uint4*>(codes + i / (D / 16) * a.cache.token_stride + i % (D / 16) * 16);
        uint4 four = *x;
        uint32_t* w = reinterpret_cast<uint32_t*>(&four);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t lo, hi;
          gdn::e4m3_to_half4(w[k], lo, hi);
          const float2 f = gdn::half2_to_float2(lo), f2 = gdn::half2_to_float2(hi);
          w[k] = gdn::to_e4m3(f.x * by, f.y * by) | gdn::to_e4m3(f2.x * by, f2.y * by) << 16;
        }
        *x = four;
      }
    }
  }
}

// ------------------------------------------------------------------------------- read
constexpr int kReadThreads = 256;
constexpr int kReadBatch = 4;

struct ReadArgs {
  Cache8 cache;
  PagedTokens paged;
  __nv_bfloat16* out[2];
  int32_t Hkv, D;
  int32_t groups;
};

// A CTA takes a group of 16 tokens, a thread 16 codes at a time: HBM-bound, 3 bytes
// an element.
__global__ void __launch_bounds__(kReadThreads) read8_kernel(const ReadArgs a) {
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  if (blockIdx.x == a.groups) {
    report_refused(a.paged);
    return;
  }
  Group g;
  if (!find_group(a.paged, blockIdx.x, &g)) return;
  if (g.page < 0 && threadIdx.x == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_ID, g.seq);
  const int chunks = a.D / 16, per_row = a.Hkv * chunks, one = (g.rows1 - g.rows0) * per_row;
  for (int j0 = threadIdx.x; j0 < 2 * one; j0 += kReadBatch * kReadThreads) {
    uint4 x[kReadBatch];
    float s[kReadBatch];
    __nv_bfloat16* dst[kReadBatch];
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      int j = j0 + i * kReadThreads;
      x[i] = make_uint4(0, 0, 0, 0);
      s[i] = 0.f;
      dst[i] = nullptr;
      if (j >= 2 * one) continue;
      const int kv = j >= one ? 1 : 0;
      j -= kv * one;
      const int row = g.rows0 + j / per_row, in_row = j % per_row, h = in_row / chunks, c = in_row % chunks;
      dst[i] = a.out[kv] + (g.token + row) * a.Hkv * a.D + in_row * 16;
      if (g.page < 0) continue;
      x[i] = *reinterpret_cast<const uint4*>(a.cache.codes[kv] + g.page * a.cache.page_stride +
                                             (g.slot + row) * a.cache.token_stride + h * a.cache.head_stride + c * 16);
      s[i] = gdn::scale_of(a.cache.scales[kv][g.page * a.cache.scale_page + g.slot / kGroup * a.cache.scale_group +
                                              h * a.cache.scale_head]);
    }
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      if (!dst[i]) continue;
      const float2 scale = make_float2(s[i], s[i]);
      const uint2 y0 = gdn::e4m3_to_bf16(x[i].x, scale), y1 = gdn::e4m3_to_bf16(x[i].y, scale);
      const uint2 y2 = gdn::e4m3_to_bf16(x[i].z, scale), y3 = gdn::e4m3_to_bf16(x[i].w, scale);
      reinterpret_cast<uint4*>(dst[i])[0] = make_uint4(y0.x, y0.y, y1.x, y1.y);
      reinterpret_cast<uint4*>(dst[i])[1] = make_uint4(y2.x, y2.y, y3.x, y3.y);
    }
  }
}

// ------------------------------------------------------------------------------- host
bool bad_norm(const gdn_qk_norm* n, bool q, bool k) {
  return !(n->eps > 0.f) || !isfinite(n->eps) || !isfinite(n->weight_offset) ||
         (q && (!n->q_weight || !gdn_host::aligned16(n->q_weight))) ||
         (k && (!n->k_weight || !gdn_host::aligned16(n->k_weight)));
}

NormRope norm_rope(const gdn_qk_norm* n, const int64_t* frequencies, int32_t rotary_dim, int32_t interleaved,
                   float amplitude, int32_t D) {
  NormRope r = {};
  if (n) {
    r.q_weight = bf(n->q_weight);
    r.k_weight = bf(n->k_weight);
    r.eps = n->eps;
    r.offset = n->weight_offset;
  }
  r.inv_dim = 1.f / static_cast<float>(D);
  r.freq = frequencies;
  r.half = rotary_dim / 2;
  r.interleaved = interleaved;
  r.amplitude = amplitude;
  return r;
}

template <int D>
int launch_append(const AppendArgs& a, dim3 grid, cudaStream_t stream) {
  const dim3 block(kAppendWarps * 32);
  switch (gdn_host::piece_width(a.n.half, D)) {
    case 8: return gdn_host::launch_pdl(append8_kernel<D, 8>, grid, block, 0, stream, a);
    case 4: return gdn_host::launch_pdl(append8_kernel<D, 4>, grid, block, 0, stream, a);
    case 2: return gdn_host::launch_pdl(append8_kernel<D, 2>, grid, block, 0, stream, a);
    default: return gdn_host::launch_pdl(append8_kernel<D, 1>, grid, block, 0, stream, a);
  }
}

}  // namespace

extern "C" int gdn_qk_norm_rope(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* q_out, int64_t q_out_token_stride,
                                const gdn_bf16* k, int64_t k_token_stride, gdn_bf16* k_out, int64_t k_out_token_stride,
                                const gdn_qk_norm* norm, const int32_t* positions, const int64_t* frequencies,
                                int32_t total_tokens, int32_t Hq, int32_t Hkv, int32_t D, int32_t rotary_dim,
                                int32_t interleaved, float amplitude, void* stream) {
  if (total_tokens < 0 || Hq < 1 || Hkv < 0 || D < 8 || D % 8 != 0 || !norm ||
      gdn_host::bad_rotation(frequencies, rotary_dim, D, amplitude) || bad_norm(norm, true, Hkv > 0))
    return GDN_ERR_INVALID_ARGUMENT;
  if (D > kMaxDim) return GDN_ERR_UNSUPPORTED;
  if ((Hkv > 0) != (k != nullptr && k_out != nullptr) && total_tokens > 0) return GDN_ERR_INVALID_ARGUMENT;
  if (total_tokens == 0) return GDN_OK;
  const auto bad = [&](const gdn_bf16* x, int64_t xs, const gdn_bf16* y, int64_t ys, int32_t H) {
    return gdn_host::bad_tokens(x, xs, H, D) || gdn_host::bad_tokens(y, ys, H, D) || (x == y && xs != ys);
  };
  if (bad(q, q_token_stride, q_out, q_out_token_stride, Hq) ||
      (Hkv > 0 && bad(k, k_token_stride, k_out, k_out_token_stride, Hkv)) || (frequencies && !positions))
    return GDN_ERR_INVALID_ARGUMENT;
  const int rc = gdn_host::check_device(nullptr);
  if (rc != GDN_OK) return rc;
  NormArgs a = {};
  a.q = bf(q);
  a.k = bf(k);
  a.q_out = bf(q_out);
  a.k_out = bf(k_out);
  a.q_stride = q_token_stride;
  a.k_stride = k_token_stride;
  a.q_out_stride = q_out_token_stride;
  a.k_out_stride = k_out_token_stride;
  a.positions = positions;
  a.n = norm_rope(norm, frequencies, rotary_dim, interleaved, amplitude, D);
  a.T = total_tokens;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  const int W = gdn_host::piece_width(a.n.half, D);
  a.units = D / (2 * W);
  a.lanes = 1;
  while (a.lanes < a.units && a.lanes < 32) a.lanes <<= 1;
  const int64_t steps = (static_cast<int64_t>(Hq) + Hkv + 32 / a.lanes - 1) / (32 / a.lanes);
  // One warp per token where that fills the GPU, as in rope.cu.
  const int64_t want = 152 * 16;
  int64_t slices = total_tokens >= want ? 1 : (want + total_tokens - 1) / total_tokens;
  if (slices > steps) slices = steps;
  a.slices = static_cast<int32_t>(slices);
  const int64_t blocks = (total_tokens * slices + kWarps - 1) / kWarps;
  if (blocks > 0x7FFFFFFF) return GDN_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kWarps * 32);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (W) {
    case 8: return gdn_host::launch_pdl(norm_rope_kernel<8>, grid, block, 0, s, a);
    case 4: return gdn_host::launch_pdl(norm_rope_kernel<4>, grid, block, 0, s, a);
    case 2: return gdn_host::launch_pdl(norm_rope_kernel<2>, grid, block, 0, s, a);
    default: return gdn_host::launch_pdl(norm_rope_kernel<1>, grid, block, 0, s, a);
  }
}

extern "C" int gdn_kv_append_paged_fp8(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* q_out, const gdn_bf16* k,
                                       int64_t k_token_stride, const gdn_bf16* v, int64_t v_token_stride,
                                       const int32_t* cu_seqlens, int32_t total_tokens, int32_t Hq,
                                       const gdn_kv_cache_fp8* cache, const gdn_page_table* table,
                                       const gdn_qk_norm* norm, const int64_t* frequencies, int32_t rotary_dim,
                                       int32_t interleaved, float amplitude, int32_t* err_word, void* stream) {
  gdn_kv_cache shell;
  int rc = gdn_host::check_paged8(cache, table, cu_seqlens, total_tokens, &shell);
  if (rc != GDN_OK) return rc;
  const int32_t D = cache->head_dim, Hkv = cache->num_heads;
  if (Hq < 0 || gdn_host::bad_rotation(frequencies, rotary_dim, D, amplitude)) return GDN_ERR_INVALID_ARGUMENT;
  if (norm && bad_norm(norm, true, true)) return GDN_ERR_INVALID_ARGUMENT;
  if (table->num_seqs == 0 || total_tokens == 0) return GDN_OK;
  if ((Hq > 0) != (q != nullptr) || (Hq > 0) != (q_out != nullptr)) return GDN_ERR_INVALID_ARGUMENT;
  if (gdn_host::bad_tokens(k, k_token_stride, Hkv, D) || gdn_host::bad_tokens(v, v_token_stride, Hkv, D))
    return GDN_ERR_INVALID_ARGUMENT;
  if (Hq > 0 && (gdn_host::bad_tokens(q, q_token_stride, Hq, D) || !gdn_host::aligned16(q_out) ||
                 (q == q_out && q_token_stride != static_cast<int64_t>(Hq) * D)))
    return GDN_ERR_INVALID_ARGUMENT;
  int sms = 0;
  rc = gdn_host::check_device(&sms);
  if (rc != GDN_OK) return rc;
  AppendArgs a = {};
  a.q = bf(q);
  a.k = bf(k);
  a.v = bf(v);
  a.q_out = bf(q_out);
  a.q_stride = q_token_stride;
  a.k_stride = k_token_stride;
  a.v_stride = v_token_stride;
  a.cache = gdn_host::cache8(cache);
  a.paged = gdn_host::paged_tokens(&shell, table, cu_seqlens, total_tokens, err_word);
  a.n = norm_rope(norm, frequencies, rotary_dim, interleaved, amplitude, D);
  a.Hq = Hq;
  a.Hkv = Hkv;
  const int64_t groups = group_slots(cu_seqlens, table->num_seqs, total_tokens);
  if (groups > 0x7FFFFFFE) return GDN_ERR_UNSUPPORTED;
  a.groups = static_cast<int32_t>(groups);
  // Few groups share their heads out among CTAs.
  const int64_t most = (2 * static_cast<int64_t>(Hkv) + (Hq + 3) / 4 + kAppendWarps - 1) / kAppendWarps;
  int64_t slices = 2 * sms / (groups + 1);
  slices = slices < 1 ? 1 : slices > most ? most : slices;
  if (slices > 65535) slices = 65535;
  const dim3 grid(static_cast<unsigned>(groups) + 1, static_cast<unsigned>(slices));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return D == 64 ? launch_append<64>(a, grid, s) : launch_append<128>(a, grid, s);
}

extern "C" int gdn_kv_read_paged_fp8(const gdn_kv_cache_fp8* cache, const gdn_page_table* table,
                                     const int32_t* cu_seqlens, int32_t total_tokens, gdn_bf16* k_out, gdn_bf16* v_out,
                                     int32_t* err_word, void* stream) {
  gdn_kv_cache shell;
  int rc = gdn_host::check_paged8(cache, table, cu_seqlens, total_tokens, &shell);
  if (rc != GDN_OK) return rc;
  if (table->num_seqs == 0 || total_tokens == 0) return GDN_OK;
  if (!k_out || !v_out || !gdn_host::aligned16(k_out) || !gdn_host::aligned16(v_out)) return GDN_ERR_INVALID_ARGUMENT;
  rc = gdn_host::check_device(nullptr);
  if (rc != GDN_OK) return rc;
  ReadArgs a = {};
  a.cache = gdn_host::cache8(cache);
  a.paged = gdn_host::paged_tokens(&shell, table, cu_seqlens, total_tokens, err_word);
  a.out[0] = bf(k_out);
  a.out[1] = bf(v_out);
  a.Hkv = cache->num_heads;
  a.D = cache->head_dim;
  const int64_t groups = group_slots(cu_seqlens, table->num_seqs, total_tokens);
  if (groups > 0x7FFFFFFE) return GDN_ERR_UNSUPPORTED;
  a.groups = static_cast<int32_t>(groups);
  return gdn_host::launch_pdl(read8_kernel, dim3(static_cast<unsigned>(groups) + 1), dim3(kReadThreads), 0,
                              static_cast<cudaStream_t>(stream), a);
}
