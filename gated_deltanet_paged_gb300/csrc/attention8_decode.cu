// attention8_decode.cu -- paged attention of one new token per sequence over the 8-bit
// cache.
//
// Mathematics, as over the 16-bit cache, with k_j = 2^a c_j and v_j = 2^b d_j (codes c, d
// of a group of 16 tokens with the scales 2^a and 2^b): the keys' scale multiplies the
// group's scores, and the values' goes into the weights.  The products take fp16, which
// holds every code exactly:
//   - q is taken to the range of fp16 by a power of two per head: its largest element
//     lies in [2^14, 2^15), so that elements down to 2^-28 of that keep all 8 bits and
//     smaller ones are off by 2^-39 of it;
//   - weights and sum have references of their own.  w_j = 2^(x_j + b_j - r + 7), r a
//     maximum of x + b that moves when one is more than 8 above it: at most 2^15, and 11
//     bits are kept down to 2^-21 of the largest (2^-31 of it is the last step), so that
//     neither many small weights nor scales far apart are lost; l = sum_j 2^(x_j - m) is
//     taken in fp32, m moving in the same way.  At the end of a segment o = sum w_j d_j
//     goes over to the reference m: o 2^(r - m - 7), and (m, l, o) joins as ever.
//
// Bound: HBM, 2 D bytes per (key, head) and 1/8 for scales.  The copies, shares and joins
// are those of attention_decode.cu; a block is 16,384 / D keys, so as many bytes are on
// their way.  Twice as many keys per second have to be multiplied, though, and every
// code converted (two per instruction), so the work per key is cut:
//   - keys are the 16 rows of the products and up to 8 query heads the columns, S = K
//     q^T, O^T = V^T P^T: half the products, scores and accumulators of the form with
//     the heads as rows, which has as many for 8 heads as for 16;
//   - four consumer warps, each with registers for two groups of keys at a time (256
//     sequences 576 us, with the heads as rows 750; eight warps with half the
//     registers, some of them spilled, 680);
//   - K: the products may take the dimensions in any order, as long as q does too: a lane
//     reads 16 consecutive codes of a key, which are four steps' operands;
//   - V: a 16 x 16 block of bytes is transposed as it is read (ldmatrix on bytes): a lane
//     gets four consecutive keys of a dimension.  The rows of S are dealt out to keys so
//     that a transposed tile of weights (movmatrix) has those of the same four.
//
// Measured: 256 sequences of up to 32,768 tokens, 4 key heads of 128 (4 GB) 575 us, 6.86
// TB/s; 61 of up to 9,000, heads of 64, 17.0 us; 2 short ones 5.0 us (launch and latency).
#include "attention_decode.cuh"
#include "cache8.cuh"

namespace {

template <int D>
constexpr int kBlock = kTileBytes / D;  // keys

struct Decode8Args {
  DecodeArgs d;
  gdn::Cache8 cache;
};

constexpr int kConsumers = 4;
constexpr int kThreads = threads_of(kConsumers);

// NT: query heads in tiles of 8.
template <int D, int NT>
struct Smem8 : Smem<kConsumers, NT * D / 16, NT> {
  static constexpr int kGroups = kBlock<D> / gdn::kGroup;
  float scale[kStages][2][kGroups];  // the keys' scales, and the exponents of the values'
};

// Two 16 x 16 blocks of bytes, transposed: lane 4 g + t gets bytes 4 t .. 4 t + 3 of column
// g (r[0]) and g + 8 (r[1]) of the first, whose rows are at the addresses of lanes 0 to
// 15; r[2], r[3] of the second.
__device__ __forceinline__ void ldmatrix2_bytes_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four bytes' two rows, transposed as an 8 x 8 tile of 16-bit numbers.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

constexpr float kShift = 7.f;  // weights are 2^7 where their reference is set
constexpr float kOver = 8.f;   // ... and 2^15 where it moves at last

// The end of an item's segment in the consumer warps: m, l (of this lane's keys) and o of
// query heads 8 n + 2 t and + 1, dimensions 16 c + g and + 8, become the CTA's, a result
// or a part of one.  false: a wait ran out.
template <int D, int NT>
__device__ __forceinline__ bool end_segment(const DecodeArgs& d, Smem8<D, NT>& sh, const Walk& w,
                                            const gdn::Shares<0>& shares, float (&m)[NT][2], float (&l)[NT][2],
                                            const float (&o)[NT][D / 16][4]) {
  const AttnArgs& a = d.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], x);
  consumers_sync<kConsumers>();  // the last item's results have been read
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
      sh.join_o[warp][n * (D / 16) + c][lane] = make_float4(o[n][c][0], o[n][c][1], o[n][c][2], o[n][c][3]);
    sh.join_ml[warp][n][lane] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
  }
  if (tid == 0) sh.stop = *static_cast<volatile int*>(&sh.abort);  // one reading for all warps
  consumers_sync<kConsumers>();
  if (sh.stop) {
    if (tid == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_TIMEOUT, 0);
    return false;
  }
  const bool starts = w.blk0 == 0, ends = w.blk1 == w.it.blocks;
  // One segment of a CTA at most starts an item that it does not end, and one at
  // most continues one: two slots per CTA.
  const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (starts ? 1 : 0);
  const int64_t row0 = static_cast<int64_t>(w.b) * a.Hq + w.head * a.group;
  // A tile of 16 dimensions of 8 heads per warp and turn.
#pragma unroll
  for (int at = warp; at < NT * D / 16; at += kConsumers) {
    const int n = at / (D / 16), c = at % (D / 16);
    float f[kConsumers][2], top[2], sum[2] = {0.f, 0.f};
    float4 ml[kConsumers];
    top[0] = top[1] = -INFINITY;
#pragma unroll
    for (int v = 0; v < kConsumers; ++v) {
      ml[v] = sh.join_ml[v][n][lane];
      top[0] = fmaxf(top[0], ml[v].x);
      top[1] = fmaxf(top[1], ml[v].y);
    }
#pragma unroll
    for (int v = 0; v < kConsumers; ++v) {
      f[v][0] = ml[v].x == -INFINITY ? 0.f : gdn::exp2_approx(ml[v].x - top[0]);
      f[v][1] = ml[v].y == -INFINITY ? 0.f : gdn::exp2_approx(ml[v].y - top[1]);
      sum[0] = fmaf(ml[v].z, f[v][0], sum[0]);
      sum[1] = fmaf(ml[v].w, f[v][1], sum[1]);
    }
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kConsumers; ++v) {
      const float4 y = sh.join_o[v][at][lane];
      x[0] = fmaf(y.x, f[v][0], x[0]);
      x[1] = fmaf(y.y, f[v][1], x[1]);
      x[2] = fmaf(y.z, f[v][0], x[2]);
      x[3] = fmaf(y.w, f[v][1], x[3]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * n + 2 * t + i;
      if (r >= a.group) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int dim = 16 * c + 8 * k + g;
        if (starts && ends)
          a.o[(row0 + r) * D + dim] = __float2bfloat16(x[2 * k + i] / sum[i]);
        else
          d.part_o[(slot * kRows + r) * D + dim] = x[2 * k + i];
      }
      if (c != 0 || g != 0) continue;
      if (!(starts && ends))
        d.part_ml[slot * kRows + r] = make_float2(top[i], sum[i]);
      else if (a.lse)
        a.lse[row0 + r] = (top[i] + log2f(sum[i])) / gdn::kLog2e;
    }
  }
  if (tid == 0 && starts && !ends)
    d.cuts[blockIdx.x] = make_int4(w.b, w.head, shares.owner(w.item0 + w.it.cost - 1), 0);
  return true;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2)
    decode_attention8_kernel(const __grid_constant__ Decode8Args d8, const __grid_constant__ CUtensorMap k_map,
                             const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ uint8_t raw[];
  Smem8<D, NT>& sh = *reinterpret_cast<Smem8<D, NT>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const DecodeArgs& d = d8.d;
  const AttnArgs& a = d.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  if (tid == kConsumers * 32) {
    gdn::prefetch_tensormap(&k_map);
    gdn::prefetch_tensormap(&v_map);
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      gdn::mbar_init(&sh.full[i], 2);
      gdn::mbar_init(&sh.empty[i], kConsumers);
    }
    gdn::mbar_init(&sh.never, 1);
    sh.abort = 0;
    gdn::fence_mbar_init();
  }
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();

  Walk w;
  gdn::Shares<0> shares(0, 1, 1);
  if (!take_share<kBlock<D>, kItemCost8>(d, sh, w, shares)) return;

  if (warp >= kConsumers) {
    // ------------------------------------------------ keys, or values
    const int kv = warp - kConsumers;
    gdn::TileCopies<D, kBlock<D>, 1> tiles(a, kv ? &v_map : &k_map, lane);
    gdn::ScaleCopies<kBlock<D>> scales(a, d8.cache, kv, lane);
    int n = 0;  // blocks issued
    bool ok = true;
    while (ok && next_segment<kBlock<D>, kItemCost8>(d, w)) {
      const int first = (w.it.first + w.blk0) * kBlock<D>;
      tiles.begin(w.it.lo, w.it.hi, w.head, w.b, w.it.s.entry, first);
      scales.begin(w.it.lo, w.it.hi, w.head, w.it.s.entry, first);
      for (int blk = w.blk0; blk < w.blk1; ++blk, ++n) {
        const int stage = n % kStages;
        if (n >= kStages) ok = warp_wait(&sh.empty[stage], ((n / kStages) - 1) & 1, &sh.abort, a.wait_ns);
        if (!ok) break;
        if (lane < Smem8<D, NT>::kGroups)
          sh.scale[stage][kv][lane] = kv ? static_cast<float>(static_cast<int>(scales.byte) - 127) : gdn::scale_of(scales.byte);
        __syncwarp();
        if (lane == 0) gdn::mbar_arrive_expect_tx(&sh.full[stage], tiles.bytes());
        __syncwarp();
        tiles.copy(sh.kv[stage][kv], &sh.full[stage], blk + 1 < w.blk1);
        scales.next(blk + 1 < w.blk1);
      }
    }
    if (!ok) sh.abort = 1;
    // Leave no copy in flight behind, whoever gave up: the stages that were issued
    // complete by themselves (bounded waits, as everywhere).
#pragma unroll 1
    for (int i = max(0, n - kStages); i < n; ++i)
      ok = wait_more(&sh.full[i % kStages], (i / kStages) & 1, nullptr, 2000000000u) && ok;
    if (!ok && lane == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_TIMEOUT, 0);
    return;
  }

  // ------------------------------------------------------------ consumers
  const int g = lane >> 2, t = lane & 3;  // fragment row and column pair
  constexpr int kSub = kBlock<D> / (16 * kConsumers);  // 16-key groups of this warp
  int n = 0;
  while (next_segment<kBlock<D>, kItemCost8>(d, w)) {
    // Queries as B fragments, heads past the group are zero: of head 8 v + g, step 4 c + i
    // takes dimensions 64 c + 16 t + 4 i to + 3.
    uint32_t q[NT][D / 16][2];
    float unit[NT][2], slope[NT][2];  // of heads 8 v + 2 t, + 1: what products are multiplied by
    {
      const __nv_bfloat16* base = a.q + static_cast<int64_t>(w.b) * a.q_stride + static_cast<int64_t>(w.head * a.group) * D;
#pragma unroll
      for (int v = 0; v < NT; ++v) {
        const int r = 8 * v + g;
        uint32_t x[D / 8];
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint4 y = make_uint4(0, 0, 0, 0);
          if (r < a.group) y = *reinterpret_cast<const uint4*>(base + r * D + (k >> 1) * 64 + t * 16 + (k & 1) * 8);
          x[4 * k] = y.x, x[4 * k + 1] = y.y, x[4 * k + 2] = y.z, x[4 * k + 3] = y.w;
        }
        uint32_t most = 0;  // numbers that are not negative compare as their bits do
#pragma unroll
        for (int k = 0; k < D / 8; ++k) most = __vmaxu2(most, x[k] & 0x7FFF7FFFu);
        most = max(most >> 16, most & 0xFFFFu);
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        // 2^(14 - e) for the largest in [2^e, 2^(e + 1)).
        const int e = min(max(static_cast<int>(most >> 7) - 127, -106), 127);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const float2 f = gdn::unpack_bf162(x[k]);
          q[v][k >> 1][k & 1] = gdn::pack_half2(f.x * up, f.y * up);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int of = __shfl_sync(0xFFFFFFFFu, e, 4 * (2 * t + i)), head = 8 * v + 2 * t + i;
          unit[v][i] = __uint_as_float(static_cast<uint32_t>(127 - 14 + of) << 23);
          slope[v][i] = a.slopes && head < a.group ? a.slopes[w.head * a.group + head] * gdn::kLog2e : 0.f;
        }
      }
    }
    float o[NT][D / 16][4], m[NT][2], mv[NT][2], l[NT][2];
#pragma unroll
    for (int v = 0; v < NT; ++v) {
      m[v][0] = m[v][1] = mv[v][0] = mv[v][1] = -INFINITY;
      l[v][0] = l[v][1] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[v][c][0] = o[v][c][1] = o[v][c][2] = o[v][c][3] = 0.f;
    }

    for (int blk = w.blk0; blk < w.blk1; ++blk, ++n) {
      const int stage = n % kStages;
      if (!warp_wait(a.debug_stall ? &sh.never : &sh.full[stage], a.debug_stall ? 0 : (n / kStages) & 1, &sh.abort,
                     a.wait_ns)) {
        sh.abort = 1;
        break;
      }
      const int row0 = warp * 16 * kSub;
      const int key0 = (w.it.first + blk) * kBlock<D> + row0;  // this warp's keys
      const int lo = w.it.lo - key0, hi = w.it.hi - key0;
      if (hi > 0 && lo < 16 * kSub) {
        const uint32_t kt = gdn::smem_u32(sh.kv[stage][0]), vt = gdn::smem_u32(sh.kv[stage][1]);
        // Row r of a group's product is key 4 (r % 8 / 2) + r % 2 + 2 (r / 8): transposed, a lane
        // has the weights of keys 4 t to 4 t + 3.
        const int key = 4 * (g >> 1) + (g & 1);
        float s[kSub][NT][4] = {};
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 x = gdn::lds128(kt + gdn::chunk_at<D>(row0 + 16 * u + key, 4 * c + t));
            const uint4 y = gdn::lds128(kt + gdn::chunk_at<D>(row0 + 16 * u + key + 2, 4 * c + t));
            const uint32_t upper[4] = {x.x, x.y, x.z, x.w}, lower[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t k[4];
              gdn::e4m3_to_half4(upper[i], k[0], k[2]);
              gdn::e4m3_to_half4(lower[i], k[1], k[3]);
#pragma unroll
              for (int v = 0; v < NT; ++v) mma_16816(s[u][v], k, q[v][4 * c + i][0], q[v][4 * c + i][1]);
            }
          }
        const bool edge = lo > 0 || hi < 16 * kSub;
        float ve[kSub];  // exponents of the values' scales
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          const float ks = sh.scale[stage][0][warp * kSub + u];
          ve[u] = sh.scale[stage][1][warp * kSub + u];
          // One factor after the other: 2^119 times a large query's is no float, where the
          // score may be zero.
#pragma unroll
          for (int v = 0; v < NT; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][v][i] = s[u][v][i] * unit[v][i & 1] * ks;
        }
        if (a.cap_log2 > 0.f) {
          float most = 0.f;
#pragma unroll
          for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int v = 0; v < NT; ++v)
              most = gdn::max3_abs(gdn::max3_abs(most, s[u][v][0], s[u][v][1]), s[u][v][2], s[u][v][3]);
          const bool near = __all_sync(0xFFFFFFFFu, most <= a.cap_near);
#pragma unroll
          for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int v = 0; v < NT; ++v)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[u][v][i] = near ? gdn::capped_near(s[u][v][i], a) : gdn::capped(s[u][v][i], a);
        } else {
#pragma unroll
          for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int v = 0; v < NT; ++v)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[u][v][i] *= a.scale_log2;
        }
        bool grow = false;
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = 16 * u + key + (i & 2);
            const bool hidden = edge && (at < lo || at >= hi);
            const float back = static_cast<float>(w.it.s.len - 1 - (key0 + at));
#pragma unroll
            for (int v = 0; v < NT; ++v) {
              float x = s[u][v][i];
              if (a.slopes) x = fmaf(-slope[v][i & 1], back, x);
              if (hidden) x = -INFINITY;
              s[u][v][i] = x;
              grow = grow || x > m[v][i & 1] + kOver || x + ve[u] > mv[v][i & 1] + kOver;
            }
          }
        if (__any_sync(0xFFFFFFFFu, grow)) {
          // The references move to the largest so far.
#pragma unroll
          for (int v = 0; v < NT; ++v)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float top = m[v][i], top_v = mv[v][i];
#pragma unroll
              for (int u = 0; u < kSub; ++u) {
                top = gdn::max3(top, s[u][v][i], s[u][v][i + 2]);
                top_v = gdn::max3(top_v, s[u][v][i] + ve[u], s[u][v][i + 2] + ve[u]);
              }
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                top_v = fmaxf(top_v, __shfl_xor_sync(0xFFFFFFFFu, top_v, x));
              }
              l[v][i] *= top > m[v][i] ? gdn::exp2_approx(m[v][i] - top) : 1.f;
              const float r = top_v > mv[v][i] ? gdn::exp2_approx(mv[v][i] - top_v) : 1.f;
              m[v][i] = top;
              mv[v][i] = top_v;
#pragma unroll
              for (int c = 0; c < D / 16; ++c) o[v][c][i] *= r, o[v][c][i + 2] *= r;
            }
        }
        uint32_t p[kSub][NT][2];
#pragma unroll
        for (int v = 0; v < NT; ++v) {
          // A head that has seen nothing yet has no reference: weights 2^-inf = 0.
          float ref[2], ref_v[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ref[i] = m[v][i] == -INFINITY ? 0.f : m[v][i];
            ref_v[i] = mv[v][i] == -INFINITY ? 0.f : mv[v][i] - kShift;
          }
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] = gdn::exp2_approx(s[u][v][i] + (ve[u] - ref_v[i & 1]));
              l[v][i & 1] += gdn::exp2_approx(s[u][v][i] - ref[i & 1]);
            }
            p[u][v][0] = transposed(gdn::pack_half2(x[0], x[1]));
            p[u][v][1] = transposed(gdn::pack_half2(x[2], x[3]));
          }
        }
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          // Codes of keys outside [lo, hi) are cleared: 0 * NaN would reach the sum.
          uint32_t keep = 0xFFFFFFFFu;
          if (edge) {
            keep = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at = 16 * u + 4 * t + i;
              if (at >= lo && at < hi) keep |= 0xFFu << (8 * i);
            }
          }
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint32_t x[4];
            ldmatrix2_bytes_trans(vt + gdn::chunk_at<D>(row0 + 16 * u + (lane & 15), 2 * k + (lane >> 4)), x);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t y[4];
              gdn::e4m3_to_half4(x[2 * i] & keep, y[0], y[2]);
              gdn::e4m3_to_half4(x[2 * i + 1] & keep, y[1], y[3]);
#pragma unroll
              for (int v = 0; v < NT; ++v) mma_16816(o[v][2 * k + i], y, p[u][v][0], p[u][v][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) gdn::mbar_arrive(&sh.empty[stage]);
    }
    // From the weights' reference to that of the sum.  The shift goes first: the rest is
    // the ratio of two sums with scales between them.
#pragma unroll
    for (int v = 0; v < NT; ++v)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f = mv[v][i] == -INFINITY ? 0.f : gdn::exp2_approx(mv[v][i] - m[v][i]);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          o[v][c][i] = o[v][c][i] * 0x1p-7f * f;
          o[v][c][i + 2] = o[v][c][i + 2] * 0x1p-7f * f;
        }
      }
    if (!end_segment<D, NT>(d, sh, w, shares, m, l, o)) return;
  }
}

template <int D, int NT>
int launch(const Decode8Args& base, const gdn_kv_cache_fp8* cache, const gdn_page_table* table, void* workspace, int sms,
           cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int smem = sizeof(Smem8<D, NT>) + 1024;
  int rc = gdn_host::func_attr_once(decode_attention8_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, done);
  if (rc != GDN_OK) return rc;
  Decode8Args d = base;
  CUtensorMap k_map, v_map;
  if ((rc = gdn_host::encode_codes_map(&k_map, cache->k, cache, d.d.a.box_shift)) != GDN_OK) return rc;
  if ((rc = gdn_host::encode_codes_map(&v_map, cache->v, cache, d.d.a.box_shift)) != GDN_OK) return rc;
  return launch_shared<D>(d.d, table, workspace, sms, stream, [&](int grid) {
    return gdn_host::launch_pdl(decode_attention8_kernel<D, NT>, dim3(grid), dim3(kThreads), smem, stream, d, k_map, v_map);
  });
}

}  // namespace

extern "C" int gdn_attention_decode_paged_fp8(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* o, float* lse,
                                              int32_t Hq, const gdn_kv_cache_fp8* cache, const gdn_page_table* table,
                                              float scale, const gdn_attention_options* options, void* workspace,
                                              size_t workspace_bytes, int32_t* err_word, void* stream) {
  // As over the 16-bit cache, more query heads per key head than this kernel's rows go to
  // the chunk kernel.
  if (cache && cache->num_heads >= 1 && Hq / cache->num_heads > kRows)
    return gdn_attention_paged_fp8(q, q_token_stride, o, lse, nullptr, table ? table->num_seqs : 0, Hq, cache, table, scale,
                                   options, workspace, workspace_bytes, err_word, stream);
  const int32_t n = table ? table->num_seqs : 0;
  gdn_kv_cache shell;
  int rc = gdn_host::check_paged8(cache, table, nullptr, n, &shell);
  if (rc != GDN_OK) return rc;
  Decode8Args d = {};
  d.d.whole = whole_items(n, table->num_entries, cache->page_size);
  const int32_t D = cache->head_dim;
  rc = gdn_host::attention_args(&d.d.a, q, q_token_stride, o, lse, nullptr, n, Hq, &shell, table, scale, options, workspace,
                                workspace_bytes, workspace_bytes_of(D, d.d.whole), err_word, D == 64 ? kBlock<64> : kBlock<128>);
  if (rc != GDN_OK || n == 0) return rc;
  int sms = 0;
  rc = gdn_host::check_device(&sms);
  if (rc != GDN_OK) return rc;
  d.cache = gdn_host::cache8(cache);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d.d.a.group <= 8)
    return D == 64 ? launch<64, 1>(d, cache, table, workspace, sms, s) : launch<128, 1>(d, cache, table, workspace, sms, s);
  return D == 64 ? launch<64, 2>(d, cache, table, workspace, sms, s) : launch<128, 2>(d, cache, table, workspace, sms, s);
}
