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
//     heads.  Where sequences have a token or two, a head's lanes take its rows one after
//     the other, and a warp several heads.
//   - reading back: a thread takes 16 codes of a head in one row after the other.
//
// Measured: norm and rotation of 65,536 tokens of 40 heads of 128 (1.34 GB) 216 us, 6.2
// TB/s, of 4 tokens 2.2; append of 8 ragged prompts, 32 + 8 heads (408 MB) 80 us, 5.1 TB/s,
// with 16 warps per SM at 122 registers (rows read twice instead of held take fewer
// registers and 88 to 97 us); of one token for each of 256 sequences 5.6 us, of which most
// is latency (with all rows of a head to a warp 9.0); 4 x 16,384 tokens of 8 heads read
// back (403 MB) 62.6 us, 6.4 TB/s.
#include <type_traits>

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
  float eps, offset, two_over_dim;
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
// Cosines, then sines of a token in the order in which lanes read them: four pairs of a
// unit beside those of the next one, so that the lanes of a head read 16 bytes each, side
// by side.
template <int W>
__device__ __forceinline__ int cs_at(int pair, int units) {
  constexpr int Q = W < 4 ? W : 4;
  const int unit = pair / W, i = pair % W;
  return ((i / Q) * units + unit) * Q + i % Q;
}
// What a unit's pairs take from shared memory: cosines and sines, or the weights of the
// first and of the second elements; two arrays, half_dim apart.
template <int W>
struct Two {
  float c[W], s[W];
  __device__ __forceinline__ void read(const float* cs, int half_dim, int unit, int units) {
    constexpr int Q = W < 4 ? W : 4;
#pragma unroll
    for (int i = 0; i < W; i += Q) {
      const float* at = cs + ((i / Q) * units + unit) * Q;
      if constexpr (Q == 4) {
        const float4 x = *reinterpret_cast<const float4*>(at), y = *reinterpret_cast<const float4*>(at + half_dim);
        c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
        s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
      } else {
#pragma unroll
        for (int k = 0; k < Q; ++k) c[i + k] = at[k], s[i + k] = at[half_dim + k];
      }
    }
  }
};

// W pairs of a head in fp32, the first elements of the pairs and the second ones; of what
// is not rotated, any two halves.
template <int W>
struct Pairs {
  float e[W], o[W];
  template <bool kInterleaved>
  __device__ __forceinline__ void unpack(const Piece<W>& a, const Piece<W>& b) {
    if constexpr (kInterleaved) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        e[i] = 2 * i < W ? gdn::get<W>(a, (2 * i) % W) : gdn::get<W>(b, (2 * i) % W);
        o[i] = 2 * i + 1 < W ? gdn::get<W>(a, (2 * i + 1) % W) : gdn::get<W>(b, (2 * i + 1) % W);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) e[i] = gdn::get<W>(a, i), o[i] = gdn::get<W>(b, i);
    }
  }
  // In the order of the head's elements.
  template <bool kInterleaved>
  __device__ __forceinline__ void ordered(float (&x)[W], float (&y)[W]) const {
    if constexpr (kInterleaved) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (2 * i < W) x[(2 * i) % W] = e[i]; else y[(2 * i) % W] = e[i];
        if (2 * i + 1 < W) x[(2 * i + 1) % W] = o[i]; else y[(2 * i + 1) % W] = o[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = e[i], y[i] = o[i];
    }
  }
  __device__ __forceinline__ float squares() const {
    if constexpr (W == 1) return fmaf(e[0], e[0], o[0] * o[0]);
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i + 1 < W; i += 2) {
      t = __ffma2_rn(make_float2(e[i], e[i + 1]), make_float2(e[i], e[i + 1]), t);
      t = __ffma2_rn(make_float2(o[i], o[i + 1]), make_float2(o[i], o[i + 1]), t);
    }
    return t.x + t.y;
  }
  __device__ __forceinline__ void scale(float r, const Two<W>& w) {
    if constexpr (W == 1) {
      e[0] *= w.c[0] * r;
      o[0] *= w.s[0] * r;
    }
    const float2 r2 = make_float2(r, r);
#pragma unroll
    for (int i = 0; i + 1 < W; i += 2) {
      const float2 x = __fmul2_rn(make_float2(e[i], e[i + 1]), __fmul2_rn(make_float2(w.c[i], w.c[i + 1]), r2));
      const float2 y = __fmul2_rn(make_float2(o[i], o[i + 1]), __fmul2_rn(make_float2(w.s[i], w.s[i + 1]), r2));
      e[i] = x.x, e[i + 1] = x.y, o[i] = y.x, o[i + 1] = y.y;
    }
  }
  __device__ __forceinline__ void turn(const Two<W>& t) {
    if constexpr (W == 1) {
      const float a = e[0], b = o[0];
      e[0] = fmaf(a, t.c[0], -b * t.s[0]);
      o[0] = fmaf(a, t.s[0], b * t.c[0]);
    }
#pragma unroll
    for (int i = 0; i + 1 < W; i += 2) {
      const float2 a = make_float2(e[i], e[i + 1]), b = make_float2(o[i], o[i + 1]);
      const float2 c = make_float2(t.c[i], t.c[i + 1]), s = make_float2(t.s[i], t.s[i + 1]);
      const float2 x = __ffma2_rn(a, c, __fmul2_rn(b, make_float2(-s.x, -s.y))), y = __ffma2_rn(a, s, __fmul2_rn(b, c));
      e[i] = x.x, e[i + 1] = x.y, o[i] = y.x, o[i + 1] = y.y;
    }
  }
};

// A kind's weights to shared memory by a block, offset included.
template <int W, bool kInterleaved>
__device__ __forceinline__ void weights_to(const NormRope& n, const __nv_bfloat16* w, float* to, int half_dim, int units) {
  for (int i = threadIdx.x; i < units * W; i += blockDim.x) {
    const int unit = i / W, k = i % W;
    int first, second;
    offsets<W>(n, unit, &first, &second);
    to[cs_at<W>(i, units)] = __bfloat162float(w[kInterleaved ? first + 2 * k : first + k]) + n.offset;
    to[half_dim + cs_at<W>(i, units)] = __bfloat162float(w[kInterleaved ? first + 2 * k + 1 : second + k]) + n.offset;
  }
}
// Over the root mean square of the head, of which `lanes` lanes have units at, at + lanes,
// ..., times the weights.  Lanes of units past the head hold zeros.
template <int W, int U>
__device__ __forceinline__ void norm(Pairs<W> (&p)[U], const NormRope& n, const float* weights, int half_dim, int at, int units,
                                     int lanes) {
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) s += p[u].squares();
  s *= 0.5f;  // 256 squares of 2^120 are more than a float
  for (int o = lanes >> 1; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const float r = rsqrtf(fmaf(s, n.two_over_dim, n.eps));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (at + u * lanes >= units) continue;
    Two<W> w;
    w.read(weights, half_dim, at + u * lanes, units);
    p[u].scale(r, w);
  }
}

// ------------------------------------------------------------------ norm and rotation
constexpr int kWarps = 4;
constexpr int kBatch = 4;   // heads in flight per lane
constexpr int kMaxDim = 256;

// One kind of heads, queries or keys.
struct NormHeads {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  const __nv_bfloat16* weight;
  int64_t x_stride, y_stride;
  int32_t H;
  int32_t steps;  // of as many heads as a warp takes at a time
};
struct NormArgs {
  NormHeads kind[2];
  const int32_t* positions;
  NormRope n;
  int32_t T, D;
  int32_t units;   // per head: D / (2 W)
  int32_t lanes;   // per head, a power of two
  int32_t slices;  // warps per token
};

template <int W, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32, 5) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  constexpr int U = W == 1 ? 4 : W == 2 ? 2 : 1;  // D / (2 W) <= 32 U
  // Weights and sines wait in shared memory: in registers they leave room for fewer warps,
  // and HBM is fed by the loads of many (65,536 tokens of 40 heads 216 us, in registers 236,
  // and in 80 of them, some spilled, 251).
  __shared__ alignas(16) float cs_all[kWarps][kMaxDim];
  __shared__ alignas(16) float weights[2][kMaxDim];
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned id = blockIdx.x * kWarps + warp, token = id / a.slices;
  const int t = static_cast<int>(min(token, static_cast<unsigned>(a.T))), slice = static_cast<int>(id - token * a.slices);
  const int per = 32 / a.lanes, at = lane & (a.lanes - 1), sub = lane / a.lanes;  // `per` heads at a time
  const int q_steps = a.kind[0].steps, steps = t < a.T ? q_steps + a.kind[1].steps : 0;
  int first[U], second[U];
  bool mine[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    offsets<W>(a.n, at + u * a.lanes, &first[u], &second[u]);
    mine[u] = at + u * a.lanes < a.units;
  }
  Piece<W> pa[kBatch][U], pb[kBatch][U];
  auto load = [&](int j, int step) {
    const NormHeads& k = a.kind[step >= q_steps ? 1 : 0];
    const int h = (step >= q_steps ? step - q_steps : step) * per + sub;
    const __nv_bfloat16* src = k.x + t * k.x_stride + h * a.D;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      pa[j][u] = pb[j][u] = Piece<W>{};
      if (step >= steps || h >= k.H || !mine[u]) continue;
      pa[j][u] = gdn::load_piece<W>(src + first[u]);
      pb[j][u] = gdn::load_piece<W>(src + second[u]);
    }
  };
#pragma unroll
  for (int j = 0; j < kBatch; ++j) load(j, slice + j * a.slices);
  weights_to<W, kInterleaved>(a.n, a.kind[0].weight, weights[0], kMaxDim / 2, a.units);
  if (a.kind[1].H) weights_to<W, kInterleaved>(a.n, a.kind[1].weight, weights[1], kMaxDim / 2, a.units);
  float* cs = cs_all[warp];
  if (a.n.half && steps) {
    const int position = a.positions[t];
#pragma unroll 1
    for (int pair = lane; pair < a.n.half; pair += 32) {
      const float2 x = gdn::pair_turn(position, a.n.freq[pair], a.n.amplitude, 1.f);
      const int to = cs_at<W>(pair, a.units);
      cs[to] = x.x;
      cs[kMaxDim / 2 + to] = x.y;
    }
  }
  __syncthreads();
  for (int s0 = slice; s0 < steps; s0 += kBatch * a.slices) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int step = s0 + j * a.slices;
      if (step >= steps) break;
      const bool is_k = step >= q_steps;
      const NormHeads& k = a.kind[is_k ? 1 : 0];
      Pairs<W> p[U];
#pragma unroll
      for (int u = 0; u < U; ++u) p[u].template unpack<kInterleaved>(pa[j][u], pb[j][u]);
      load(j, step + kBatch * a.slices);
      norm<W, U>(p, a.n, weights[is_k ? 1 : 0], kMaxDim / 2, at, a.units, a.lanes);
      const int h = (is_k ? step - q_steps : step) * per + sub;
      __nv_bfloat16* dst = k.y + t * k.y_stride + h * a.D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h >= k.H || !mine[u]) continue;
        if ((at + u * a.lanes) * W < a.n.half) {
          Two<W> turn;
          turn.read(cs, kMaxDim / 2, at + u * a.lanes, a.units);
          p[u].turn(turn);
        }
        float x[W], y[W];
        p[u].template ordered<kInterleaved>(x, y);
        gdn::store_piece<W>(dst + first[u], gdn::pack<W>(x));
        gdn::store_piece<W>(dst + second[u], gdn::pack<W>(y));
      }
    }
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
// Warps of a CTA.
template <bool kWide>
constexpr int kAppendWarps = kWide ? 8 : 4;

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

// The group's scale and codes in one head, of a warp (kWide) or of the lanes of a head.
struct Slot {
  uint8_t* codes;  // of row 0
  uint8_t* scale;
  uint32_t before;  // scale of the earlier tokens, 0: there are none
};
// The scale byte for a largest value (its bits; numbers that are not negative compare as
// those do): the least e with it <= 448 * 2^e, 448 = 1.75 * 2^8, and no less than before.
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits, uint32_t before) {
  const int least = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(static_cast<uint32_t>(min(max(least, gdn::kScaleLeast), gdn::kScaleMost)), before);
}
// Earlier tokens' codes, rounded to the scale that has grown (by 2^-126 all of them become
// zero, as by less); a lane takes every `lanes`-th 16 of them.
template <int D>
__device__ __forceinline__ void round_again(const Slot& s, int64_t token_stride, int rows, uint32_t byte, int lane, int lanes) {
  const float by = __uint_as_float(max(127 - static_cast<int>(byte - s.before), 1) << 23);
#pragma unroll 1
  for (int i = lane; i < rows * (D / 16); i += lanes) {
    uint4* x = reinterpret_cast<uint4*>(s.codes + i / (D / 16) * token_stride + i % (D / 16) * 16);
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

// kWide: a warp takes all rows of a group's head at a time.  Otherwise, where groups have
// a new token or two, the lanes of a head take its rows one after the other, and a
// warp as many heads as it has lanes for; rows behind the first are read twice.
template <int D, int W, bool kInterleaved, bool kWide>
__global__ void __launch_bounds__(kAppendWarps<kWide> * 32, kWide ? 2 : 4) append8_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kWarpsOf = kAppendWarps<kWide>;
  constexpr int kUnits = D / (2 * W);
  constexpr int kLanes = kUnits < 32 ? kUnits : 32;  // per head
  constexpr int U = kUnits / kLanes;
  constexpr int kPer = 32 / kLanes;                  // heads or rows at a time
  constexpr int kSteps = kGroup / kPer;
  __shared__ alignas(16) float cs[kGroup][D];
  __shared__ alignas(16) float q_weights[D], k_weights[D];
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  if (blockIdx.x == a.groups) {
    if (blockIdx.y == 0) report_refused(a.paged);
    return;
  }
  Group g;
  if (!find_group(a.paged, blockIdx.x, &g)) return;  // all threads alike
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, at = lane % kLanes, sub = lane / kLanes;
  const int worker = blockIdx.y * kWarpsOf + warp, workers = gridDim.y * kWarpsOf;
  const bool normed = a.n.q_weight != nullptr;
  int first[U], second[U];
#pragma unroll
  for (int u = 0; u < U; ++u) offsets<W>(a.n, at + u * kLanes, &first[u], &second[u]);
  auto load = [&](const __nv_bfloat16* src, bool there, Piece<W> (&pa)[U], Piece<W> (&pb)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      pa[u] = pb[u] = Piece<W>{};
      if (!there) continue;
      pa[u] = gdn::load_piece<W>(src + first[u]);
      pb[u] = gdn::load_piece<W>(src + second[u]);
    }
  };
  // Unpacked, over its norm, rotated for the group's row.
  auto take = [&](const Piece<W> (&pa)[U], const Piece<W> (&pb)[U], const float* w, bool computed, int row,
                  Pairs<W> (&p)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) p[u].template unpack<kInterleaved>(pa[u], pb[u]);
    if (!computed) return;
    if (normed) norm<W, U>(p, a.n, w, D / 2, at, kUnits, kLanes);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = at + u * kLanes;
      if (unit * W >= a.n.half) continue;
      Two<W> t;
      t.read(cs[row], D / 2, unit, kUnits);
      p[u].turn(t);
    }
  };

  // Queries: kPer heads of a row at a time.  The first are asked for before the sines.
  const int per_row = (a.Hq + kPer - 1) / kPer, jobs = (g.rows1 - g.rows0) * per_row;
  constexpr int kAhead = 4;
  Piece<W> pa[kAhead][U], pb[kAhead][U];
  auto load_query = [&](int i, int j) {
    const int row = g.rows0 + j / max(per_row, 1), h = j % max(per_row, 1) * kPer + sub;
    load(a.q + (g.token + row) * a.q_stride + static_cast<int64_t>(h) * D, j < jobs && h < a.Hq, pa[i], pb[i]);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load_query(i, worker + i * workers);
  if (a.n.half) {
    for (int r = g.rows0 + warp; r < g.rows1; r += kWarpsOf)
      for (int pair = lane; pair < a.n.half; pair += 32) {
        const float2 x = gdn::pair_turn(g.position + r, a.n.freq[pair], a.n.amplitude, 1.f);
        cs[r][cs_at<W>(pair, kUnits)] = x.x;
        cs[r][D / 2 + cs_at<W>(pair, kUnits)] = x.y;
      }
  }
  if (normed) {
    weights_to<W, kInterleaved>(a.n, a.n.q_weight, q_weights, D / 2, kUnits);
    weights_to<W, kInterleaved>(a.n, a.n.k_weight, k_weights, D / 2, kUnits);
  }
  __syncthreads();
  for (int j0 = worker; j0 < jobs; j0 += kAhead * workers) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = j0 + i * workers, row = g.rows0 + j / per_row, h = j % per_row * kPer + sub;
      if (j >= jobs) break;
      Pairs<W> p[U];
      take(pa[i], pb[i], q_weights, true, row, p);
      if (kWide || j + kAhead * workers < jobs) load_query(i, j + kAhead * workers);  // groups of a token have few
      if (h >= a.Hq) continue;
      __nv_bfloat16* dst = a.q_out + ((g.token + row) * a.Hq + h) * D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[W], y[W];
        p[u].template ordered<kInterleaved>(x, y);
        gdn::store_piece<W>(dst + first[u], gdn::pack<W>(x));
        gdn::store_piece<W>(dst + second[u], gdn::pack<W>(y));
      }
    }
  }

  if (g.page < 0) {
    if (worker == 0 && lane == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_ID, g.seq);
    return;
  }
  // Keys, then values: item h, or Hkv + h.
  auto slot_of = [&](int kv, int h) {
    Slot s;
    s.codes = a.cache.codes[kv] + g.page * a.cache.page_stride + g.slot * a.cache.token_stride + h * a.cache.head_stride;
    s.scale = a.cache.scales[kv] + g.page * a.cache.scale_page + g.slot / kGroup * a.cache.scale_group + h * a.cache.scale_head;
    s.before = g.rows0 > 0 ? *s.scale : 0u;
    return s;
  };
  auto most_of = [&](const Pairs<W> (&p)[U], float most) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < W; ++k) most = gdn::max3_abs(most, p[u].e[k], p[u].o[k]);
    return most;
  };
  auto store = [&](const Slot& s, int row, const Pairs<W> (&p)[U], float inv) {
    uint8_t* dst = s.codes + row * a.cache.token_stride;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[W], y[W];
      p[u].template ordered<kInterleaved>(x, y);
      store_codes<W>(dst + first[u], x, inv);
      store_codes<W>(dst + second[u], y, inv);
    }
  };
  const auto inverse = [](uint32_t byte) { return __uint_as_float((254u - min(byte, 253u)) << 23); };
  if constexpr (kWide) {
    for (int item = worker; item < 2 * a.Hkv; item += workers) {
      const bool is_k = item < a.Hkv;
      const int h = is_k ? item : item - a.Hkv;
      const __nv_bfloat16* src = (is_k ? a.k : a.v) + static_cast<int64_t>(h) * D;
      const int64_t stride = is_k ? a.k_stride : a.v_stride;
      const Slot slot = slot_of(is_k ? 0 : 1, h);
      Piece<W> xa[kSteps][U], xb[kSteps][U];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int row = i * kPer + sub;
        load(src + (g.token + row) * stride, row >= g.rows0 && row < g.rows1, xa[i], xb[i]);
      }
      Pairs<W> p[kSteps][U];
      float most = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int row = i * kPer + sub;
        take(xa[i], xb[i], k_weights, is_k, min(max(row, g.rows0), g.rows1 - 1), p[i]);
        most = most_of(p[i], most);
      }
      const uint32_t byte = scale_byte(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most)), slot.before);
      const float inv = inverse(byte);
      __syncwarp();  // every lane has read the scale
      if (lane == 0) *slot.scale = static_cast<uint8_t>(byte);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int row = i * kPer + sub;
        if (row >= g.rows0 && row < g.rows1) store(slot, row, p[i], inv);
      }
      if (g.rows0 > 0 && byte > slot.before) round_again<D>(slot, a.cache.token_stride, g.rows0, byte, lane, 32);
    }
  } else {
    for (int item0 = worker * kPer; item0 < 2 * a.Hkv; item0 += workers * kPer) {
      const int item = min(item0 + sub, 2 * a.Hkv - 1);
      const bool there = item0 + sub < 2 * a.Hkv, is_k = item < a.Hkv;
      const int h = is_k ? item : item - a.Hkv;
      const __nv_bfloat16* src = (is_k ? a.k : a.v) + g.token * (is_k ? a.k_stride : a.v_stride) + static_cast<int64_t>(h) * D;
      const int64_t stride = is_k ? a.k_stride : a.v_stride;
      const Slot slot = slot_of(is_k ? 0 : 1, h);
      Pairs<W> p[U];
      // Keys and values may stand side by side in a warp, which takes the norm together.
      auto row_of = [&](int row) {
        Piece<W> xa[U], xb[U];
        load(src + row * stride, true, xa, xb);
        Pairs<W> raw[U];
        take(xa, xb, k_weights, false, row, raw);
        take(xa, xb, k_weights, true, row, p);
        if (is_k) return;
#pragma unroll
        for (int u = 0; u < U; ++u) p[u] = raw[u];
      };
      float most = 0.f;
#pragma unroll 1
      for (int row = g.rows1 - 1; row >= g.rows0; --row) {
        row_of(row);
        most = most_of(p, most);
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      const uint32_t byte = scale_byte(__float_as_uint(most), slot.before);
      const float inv = inverse(byte);
      __syncwarp();  // every lane has read the scale
      if (there && at == 0) *slot.scale = static_cast<uint8_t>(byte);
#pragma unroll 1
      for (int row = g.rows0; row < g.rows1; ++row) {
        if (row > g.rows0) row_of(row);  // the first row's was taken last
        if (there) store(slot, row, p, inv);
      }
      if (there && g.rows0 > 0 && byte > slot.before) round_again<D>(slot, a.cache.token_stride, g.rows0, byte, at, kLanes);
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
  int32_t aligned32;  // of both outputs
};

// A CTA takes a group of 16 tokens, a thread 16 codes of a head in one row after the other:
// HBM-bound, 3 bytes an element.
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
  const int chunks = a.D / 16, per_row = a.Hkv * chunks;  // 16 codes each
  // Where a row's chunks are fewer than threads, rows stand side by side.
  const int beside = max(1, kReadThreads / (2 * per_row));
  const int row0 = g.rows0 + (beside > 1 ? static_cast<int>(threadIdx.x) / (2 * per_row) : 0);
  if (row0 >= g.rows0 + beside) return;
  for (int j = beside > 1 ? static_cast<int>(threadIdx.x) % (2 * per_row) : threadIdx.x; j < 2 * per_row; j += kReadThreads) {
    const int kv = j >= per_row ? 1 : 0, in_row = j - kv * per_row, h = in_row / chunks, c = in_row % chunks;
    const uint8_t* src = nullptr;
    float f = 0.f;
    if (g.page >= 0) {
      src = a.cache.codes[kv] + g.page * a.cache.page_stride + g.slot * a.cache.token_stride + h * a.cache.head_stride + c * 16;
      f = gdn::scale_of(a.cache.scales[kv][g.page * a.cache.scale_page + g.slot / kGroup * a.cache.scale_group +
                                           h * a.cache.scale_head]);
    }
    const float2 scale = make_float2(f, f);
    __nv_bfloat16* const dst = a.out[kv] + g.token * a.Hkv * a.D + in_row * 16;
    for (int r0 = row0; r0 < g.rows1; r0 += kReadBatch * beside) {
      uint4 x[kReadBatch];
#pragma unroll
      for (int i = 0; i < kReadBatch; ++i) {
        const int row = r0 + i * beside;
        x[i] = make_uint4(0, 0, 0, 0);
        if (src && row < g.rows1) x[i] = *reinterpret_cast<const uint4*>(src + row * a.cache.token_stride);
      }
#pragma unroll
      for (int i = 0; i < kReadBatch; ++i) {
        const int row = r0 + i * beside;
        if (row >= g.rows1) continue;
        const uint2 y0 = gdn::e4m3_to_bf16(x[i].x, scale), y1 = gdn::e4m3_to_bf16(x[i].y, scale);
        const uint2 y2 = gdn::e4m3_to_bf16(x[i].z, scale), y3 = gdn::e4m3_to_bf16(x[i].w, scale);
        const uint32_t y[8] = {y0.x, y0.y, y1.x, y1.y, y2.x, y2.y, y3.x, y3.y};
        gdn::store32(dst + static_cast<int64_t>(row) * a.Hkv * a.D, y, a.aligned32 != 0);
      }
    }
  }
}

// ----------------------------------------------------------------------------- expand
// What the new tokens of a batch may see, out of the 8-bit cache into bf16 pages [table
// entry, Hkv, page_size, D] of their own, so that many rows read it as it is.  The batch is
// one line of groups of 16 tokens, and each CTA takes an equal piece.  HBM-bound, 3 bytes
// an element.
constexpr int kExpandThreads = 256;

struct ExpandArgs {
  Cache8 cache;
  PagedTokens paged;
  __nv_bfloat16* out[2];
  int32_t* pages;  // receives 0, 1, 2, ...: the table entries' pages among `out`
  int32_t Hkv, D, window;
};

struct Needed {
  SeqRange s;
  int first;   // group
  int groups;
};
__device__ __forceinline__ Needed needed(const ExpandArgs& a, int b) {
  Needed n;
  n.s = gdn::seq_range(a.paged, b);
  const int position = n.s.len - n.s.new_tokens;
  n.first = a.window >= 0 ? max(0, position - a.window) / kGroup : 0;
  n.groups = n.s.new_tokens ? (n.s.len + kGroup - 1) / kGroup - n.first : 0;
  return n;
}

__global__ void __launch_bounds__(kExpandThreads) expand8_kernel(const __grid_constant__ ExpandArgs a) {
  __shared__ int64_t scan[kExpandThreads / 32];
  __shared__ int begin[2];  // sequence, group
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kExpandThreads + tid; i < a.paged.num_entries;
       i += static_cast<int64_t>(gridDim.x) * kExpandThreads)
    a.pages[i] = static_cast<int32_t>(i);
  const int per = (a.paged.num_seqs + kExpandThreads - 1) / kExpandThreads;
  const int b0 = min(tid * per, a.paged.num_seqs), b1 = min(b0 + per, a.paged.num_seqs);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += needed(a, b).groups;
  int64_t before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) scan[warp] = before;
  __syncthreads();
  before -= mine;
  int64_t total = 0;
  for (int i = 0; i < kExpandThreads / 32; ++i) {
    if (i < warp) before += scan[i];
    total += scan[i];
  }
  const int64_t start = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;
  if (start < end && before <= start && start < before + mine) {
    int b = b0;
    int64_t rest = start - before;
    for (int n; rest >= (n = needed(a, b).groups); ++b) rest -= n;
    begin[0] = b;
    begin[1] = static_cast<int>(rest);
  }
  __syncthreads();
  if (start >= end) return;
  int b = begin[0], group = begin[1];
  Needed n = needed(a, b);
  const int chunks = a.D / 16, per_row = a.Hkv * chunks;  // 16 codes each
  for (int64_t at = start; at < end; ++at, ++group) {
    while (group >= n.groups) {
      n = needed(a, ++b);
      group = 0;
    }
    const int position = (n.first + group) * kGroup, rows = min(kGroup, n.s.len - position);
    const int in_table = position / a.paged.page_size, slot = position - in_table * a.paged.page_size;
    const int64_t entry = static_cast<int64_t>(n.s.entry) + in_table;
    const int page = a.paged.pages[entry];
    const bool there = page >= 0 && page < a.paged.num_pages;
    if (!there && tid == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_ID, b);
    // 16 rows of a chunk by neighbours: a row's 16 codes are 32 bytes of a run of rows.
    for (int j0 = tid; j0 < 2 * per_row * kGroup; j0 += kReadBatch * kExpandThreads) {
      uint4 x[kReadBatch];
      float f[kReadBatch];
#pragma unroll
      for (int i = 0; i < kReadBatch; ++i) {
        const int j = j0 + i * kExpandThreads;
        const int c = j % chunks, row = j / chunks % kGroup, head = j / (chunks * kGroup), kv = head >= a.Hkv ? 1 : 0;
        const int h = head - kv * a.Hkv;
        x[i] = make_uint4(0, 0, 0, 0);
        f[i] = 0.f;
        if (!there || j >= 2 * per_row * kGroup || row >= rows) continue;
        x[i] = *reinterpret_cast<const uint4*>(a.cache.codes[kv] + page * a.cache.page_stride +
                                               (slot + row) * a.cache.token_stride + h * a.cache.head_stride + c * 16);
        f[i] = gdn::scale_of(a.cache.scales[kv][page * a.cache.scale_page + slot / kGroup * a.cache.scale_group +
                                                h * a.cache.scale_head]);
      }
#pragma unroll
      for (int i = 0; i < kReadBatch; ++i) {
        const int j = j0 + i * kExpandThreads;
        const int c = j % chunks, row = j / chunks % kGroup, head = j / (chunks * kGroup), kv = head >= a.Hkv ? 1 : 0;
        const int h = head - kv * a.Hkv;
        if (j >= 2 * per_row * kGroup || row >= rows) continue;
        const float2 scale = make_float2(f[i], f[i]);
        const uint2 y0 = gdn::e4m3_to_bf16(x[i].x, scale), y1 = gdn::e4m3_to_bf16(x[i].y, scale);
        const uint2 y2 = gdn::e4m3_to_bf16(x[i].z, scale), y3 = gdn::e4m3_to_bf16(x[i].w, scale);
        const uint32_t y[8] = {y0.x, y0.y, y1.x, y1.y, y2.x, y2.y, y3.x, y3.y};
        gdn::store32(a.out[kv] + ((entry * a.Hkv + h) * a.paged.page_size + slot + row) * a.D + c * 16, y, true);
      }
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
  r.two_over_dim = 2.f / static_cast<float>(D);
  r.freq = frequencies;
  r.half = rotary_dim / 2;
  r.interleaved = interleaved;
  r.amplitude = amplitude;
  return r;
}

// Calls run with the widest piece, and whether pairs are interleaved.
template <typename Run>
int by_pairs(int32_t half, int32_t D, bool interleaved, const Run& run) {
  const auto of = [&](auto width) {
    return interleaved && half ? run(width, std::true_type()) : run(width, std::false_type());
  };
  switch (gdn_host::piece_width(half, D)) {
    case 8: return of(std::integral_constant<int, 8>());
    case 4: return of(std::integral_constant<int, 4>());
    case 2: return of(std::integral_constant<int, 2>());
    default: return of(std::integral_constant<int, 1>());
  }
}

template <int D, bool kWide>
int launch_append(const AppendArgs& a, dim3 grid, cudaStream_t stream) {
  return by_pairs(a.n.half, D, a.n.interleaved != 0, [&](auto width, auto interleaved) {
    return gdn_host::launch_pdl(append8_kernel<D, decltype(width)::value, decltype(interleaved)::value, kWide>, grid,
                                dim3(kAppendWarps<kWide> * 32), 0, stream, a);
  });
}

}  // namespace

int gdn_host::expand8(const gdn_kv_cache_fp8* cache, const PagedTokens& paged, int32_t window, gdn_bf16* k, gdn_bf16* v,
                      int32_t* pages, int sms, cudaStream_t stream) {
  ExpandArgs a = {};
  a.cache = cache8(cache);
  a.paged = paged;
  a.out[0] = bf(k);
  a.out[1] = bf(v);
  a.pages = pages;
  a.Hkv = cache->num_heads;
  a.D = cache->head_dim;
  a.window = window;
  return launch_pdl(expand8_kernel, dim3(static_cast<unsigned>(6 * sms)), dim3(kExpandThreads), 0, stream, a);
}

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
  a.positions = positions;
  a.n = norm_rope(norm, frequencies, rotary_dim, interleaved, amplitude, D);
  a.T = total_tokens;
  a.D = D;
  const int W = gdn_host::piece_width(a.n.half, D);
  a.units = D / (2 * W);
  a.lanes = 1;
  while (a.lanes < a.units && a.lanes < 32) a.lanes <<= 1;
  const int per = 32 / a.lanes;
  a.kind[0] = NormHeads{bf(q), bf(q_out), bf(norm->q_weight), q_token_stride, q_out_token_stride, Hq, (Hq + per - 1) / per};
  a.kind[1] = NormHeads{bf(k), bf(k_out), bf(norm->k_weight), k_token_stride, k_out_token_stride, Hkv, (Hkv + per - 1) / per};
  const int64_t steps = static_cast<int64_t>(a.kind[0].steps) + a.kind[1].steps;
  // One warp per token where that fills the GPU, as in rope.cu.
  const int64_t want = 152 * 16;
  int64_t slices = total_tokens >= want ? 1 : (want + total_tokens - 1) / total_tokens;
  if (slices > steps) slices = steps;
  a.slices = static_cast<int32_t>(slices);
  const dim3 grid(static_cast<unsigned>((total_tokens * slices + kWarps - 1) / kWarps)), block(kWarps * 32);
  return by_pairs(a.n.half, D, interleaved != 0, [&](auto width, auto pairs) {
    return gdn_host::launch_pdl(norm_rope_kernel<decltype(width)::value, decltype(pairs)::value>, grid, block, 0,
                                static_cast<cudaStream_t>(stream), a);
  });
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
  // Sequences of a new token or two, as in decoding.
  const bool wide = total_tokens > 2 * static_cast<int64_t>(table->num_seqs);
  // Few groups share their heads out among CTAs.
  const int64_t most = wide ? (2 * static_cast<int64_t>(Hkv) + Hq / 4) / kAppendWarps<true> + 1
                            : (2 * static_cast<int64_t>(Hkv) + Hq / 4) / kAppendWarps<false> + 1;
  int64_t slices = 4 * sms / (groups + 1);
  slices = slices < 1 ? 1 : slices > most ? most : slices;
  if (slices > 65535) slices = 65535;
  const dim3 grid(static_cast<unsigned>(groups) + 1, static_cast<unsigned>(slices));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (wide) return D == 64 ? launch_append<64, true>(a, grid, s) : launch_append<128, true>(a, grid, s);
  return D == 64 ? launch_append<64, false>(a, grid, s) : launch_append<128, false>(a, grid, s);
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
  a.aligned32 = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31u) == 0;
  const int64_t groups = group_slots(cu_seqlens, table->num_seqs, total_tokens);
  if (groups > 0x7FFFFFFE) return GDN_ERR_UNSUPPORTED;
  a.groups = static_cast<int32_t>(groups);
  return gdn_host::launch_pdl(read8_kernel, dim3(static_cast<unsigned>(groups) + 1), dim3(kReadThreads), 0,
                              static_cast<cudaStream_t>(stream), a);
}
