// attention8_decode.cu -- paged attention of one new token per sequence over the 8-bit
// cache.
//
// Mathematics, as over the 16-bit cache, with k_j = 2^a c_j and v_j = 2^b d_j (codes c, d
// of a group of 16 tokens with the scales 2^a and 2^b): the keys' scale multiplies the
// group's scores, and the values' goes into the weights.  The products take fp16, which
// holds every code exactly:
//   - q is taken to the range of fp16 by a power of two per row: its largest element
//     lies in [2^14, 2^15), so that elements down to 2^-28 of that keep all 8 bits and
//     smaller ones are off by 2^-39 of it;
//   - weights have two maxima.  w_j = 2^(x_j + b_j - r), r the running maximum of x + b
//     less 15, is at most 2^15 and keeps 11 bits down to 2^-29 of the largest, so that
//     neither many small weights nor scales far apart are lost; l = sum_j 2^(x_j - m)
//     is taken in fp32 with a maximum m of its own.  At the end of a segment o = sum w_j
//     d_j goes over to the reference m: o 2^(r - m), and (m, l, o) joins as ever.
//
// Bound: HBM, 2 D bytes per (key, head) and 1/8 for scales.  The copies, shares and joins
// are those of attention_decode.cu; a block is 16,384 / D keys, half of what a byte per
// element less would be there, so as many bytes are on their way.  What is new is done
// in registers: two codes become two fp16 numbers in one instruction.
//   - K: the products may take the dimensions in any order, as long as q does too: a lane
//     reads 16 consecutive codes of a key, which are four steps' operands.
//   - V: a 16 x 16 block of bytes is transposed as it is read (ldmatrix on bytes): a lane
//     gets four consecutive keys of a dimension.  The scores' columns are dealt out
//     to keys so that a lane has the weights of those four.
#include "attention_decode.cuh"
#include "cache8.cuh"

namespace {

template <int D>
constexpr int kBlock = kTileBytes / D;  // keys

struct Decode8Args {
  DecodeArgs d;
  gdn::Cache8 cache;
};

template <int D>
struct Smem8 : Smem<D> {
  static constexpr int kGroups = kBlock<D> / gdn::kGroup;
  float scale[kStages][2][kGroups];  // the keys' scales, and the exponents of the values'
};

// Scale bytes of one block after the other, a group's by a lane, asked for a block ahead.
template <int kBlockKeys>
struct ScaleCopies {
  const AttnArgs& a;
  const uint8_t* scales;
  int64_t page_stride, group_stride, head_stride;
  int lane, lo, hi, key, entry, slot;
  const int32_t* pages;
  int64_t head_at;
  uint32_t byte;

  __device__ __forceinline__ ScaleCopies(const Decode8Args& d, int kv, int l)
      : a(d.d.a), scales(d.cache.scales[kv]), page_stride(d.cache.scale_page), group_stride(d.cache.scale_group),
        head_stride(d.cache.scale_head), lane(l) {}
  __device__ __forceinline__ void look_ahead() {
    byte = 127;
    if (lane >= kBlockKeys / gdn::kGroup || key + gdn::kGroup <= lo || key >= hi) return;
    const int p = pages[entry];
    if (p >= 0 && p < a.paged.num_pages)  // else its codes are zeros, reported by the copies
      byte = scales[p * page_stride + (slot / gdn::kGroup) * group_stride + head_at];
  }
  __device__ __forceinline__ void begin(int from, int to, int head, int table_entry, int first) {
    lo = from, hi = to, head_at = head * head_stride;
    pages = a.paged.pages + table_entry;
    key = first + lane * gdn::kGroup;
    entry = key / a.paged.page_size;
    slot = key - entry * a.paged.page_size;
    look_ahead();
  }
  __device__ __forceinline__ void next(bool more) {
    key += kBlockKeys;
    entry += kBlockKeys / a.paged.page_size;
    slot += kBlockKeys % a.paged.page_size;
    if (slot >= a.paged.page_size) slot -= a.paged.page_size, ++entry;
    if (more) look_ahead();
  }
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
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte chunk c of key r of a tile: swizzled over 128 or 64 bytes.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(uint32_t r, uint32_t c) {
  if constexpr (D == 128) return gdn::swz(r, c);
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

constexpr float kShift = 15.f;  // weights are 2^15 at most

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    decode_attention8_kernel(const __grid_constant__ Decode8Args d8, const __grid_constant__ CUtensorMap k_map,
                             const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ uint8_t raw[];
  Smem8<D>& sh = *reinterpret_cast<Smem8<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
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
  if (!take_share<kBlock<D>>(d, sh, w, shares)) return;

  if (warp >= kConsumers) {
    // ------------------------------------------------ keys, or values
    const int kv = warp - kConsumers;
    gdn::TileCopies<D, kBlock<D>, 1> tiles(a, kv ? &v_map : &k_map, lane);
    ScaleCopies<kBlock<D>> scales(d8, kv, lane);
    int n = 0;  // blocks issued
    bool ok = true;
    while (ok && next_segment<kBlock<D>>(d, w)) {
      const int first = (w.it.first + w.blk0) * kBlock<D>;
      tiles.begin(w.it.lo, w.it.hi, w.head, w.b, w.it.s.entry, first);
      scales.begin(w.it.lo, w.it.hi, w.head, w.it.s.entry, first);
      for (int blk = w.blk0; blk < w.blk1; ++blk, ++n) {
        const int stage = n % kStages;
        if (n >= kStages) ok = warp_wait(&sh.empty[stage], ((n / kStages) - 1) & 1, &sh.abort, a.wait_ns);
        if (!ok) break;
        if (lane < Smem8<D>::kGroups)
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
  int n = 0;
  while (next_segment<kBlock<D>>(d, w)) {
    const int h0 = w.head * a.group;  // first query head of the rows
    const int rows = a.group;
    // Queries as A fragments, rows past the group are zero.  Step 4 c + i of the lanes with
    // column pair t takes dimensions 64 c + 16 t + 4 i to + 3.
    uint32_t q[D / 16][4];
    float unit[2];  // what a row's products are to be multiplied by
    {
      const __nv_bfloat16* base = a.q + static_cast<int64_t>(w.b) * a.q_stride + static_cast<int64_t>(h0) * D;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = g + 8 * i;
        uint32_t x[D / 8];
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint4 y = make_uint4(0, 0, 0, 0);
          if (r < rows) y = *reinterpret_cast<const uint4*>(base + r * D + (k >> 1) * 64 + t * 16 + (k & 1) * 8);
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
        unit[i] = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const float2 f = gdn::unpack_bf162(x[k]);
          q[k >> 1][i + 2 * (k & 1)] = gdn::pack_half2(f.x * up, f.y * up);
        }
      }
    }
    float slope[2] = {0.f, 0.f};
    if (a.slopes) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (g + 8 * i < rows) slope[i] = a.slopes[h0 + g + 8 * i] * gdn::kLog2e;
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, mv[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int blk = w.blk0; blk < w.blk1; ++blk, ++n) {
      const int stage = n % kStages;
      if (!warp_wait(a.debug_stall ? &sh.never : &sh.full[stage], a.debug_stall ? 0 : (n / kStages) & 1, &sh.abort,
                     a.wait_ns)) {
        sh.abort = 1;
        break;
      }
      constexpr int kSub = kBlock<D> / 64;  // 16-key groups of this warp
      const int row0 = warp * 16 * kSub;
      const int key0 = (w.it.first + blk) * kBlock<D> + row0;  // this warp's keys
      const int lo = w.it.lo - key0, hi = w.it.hi - key0;
      if (hi > 0 && lo < 16 * kSub) {
        const uint32_t kt = gdn::smem_u32(sh.kv[stage][0]), vt = gdn::smem_u32(sh.kv[stage][1]);
        // Column n of product j of a group is key 4 (n / 2) + n % 2 + 2 j: a lane has the scores of
        // keys 4 t to 4 t + 3.
        float s[2 * kSub][4] = {};
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t r = row0 + 16 * u + 4 * (g >> 1) + (g & 1) + 2 * j;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              const uint4 x = lds128(kt + chunk_at<D>(r, 4 * c + t));
              const uint32_t four[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t b0, b1;
                gdn::e4m3_to_half4(four[i], b0, b1);
                mma_16816(s[2 * u + j], q[4 * c + i], b0, b1);
              }
            }
          }
        const bool edge = lo > 0 || hi < 16 * kSub;
        float ks[kSub], ve[kSub];
#pragma unroll
        for (int u = 0; u < kSub; ++u) ks[u] = sh.scale[stage][0][warp * kSub + u], ve[u] = sh.scale[stage][1][warp * kSub + u];
#pragma unroll
        for (int j = 0; j < 2 * kSub; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[j][i] *= unit[i >> 1] * ks[j >> 1];
        if (a.cap_log2 > 0.f) {
          float most = 0.f;
#pragma unroll
          for (int j = 0; j < 2 * kSub; ++j) most = gdn::max3_abs(gdn::max3_abs(most, s[j][0], s[j][1]), s[j][2], s[j][3]);
          if (__all_sync(0xFFFFFFFFu, most <= a.cap_near)) {
#pragma unroll
            for (int j = 0; j < 2 * kSub; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[j][i] = gdn::capped_near(s[j][i], a);
          } else {
#pragma unroll
            for (int j = 0; j < 2 * kSub; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[j][i] = gdn::capped(s[j][i], a);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2 * kSub; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] *= a.scale_log2;
        }
        float top[2] = {m[0], m[1]}, top_v[2] = {mv[0], mv[1]};
#pragma unroll
        for (int j = 0; j < 2 * kSub; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = s[j][i];
            const int key = (j >> 1) * 16 + 4 * t + 2 * (j & 1) + (i & 1);
            if (a.slopes) x = fmaf(-slope[i >> 1], static_cast<float>(w.it.s.len - 1 - (key0 + key)), x);
            if (edge && (key < lo || key >= hi)) x = -INFINITY;
            s[j][i] = x;
            top[i >> 1] = fmaxf(top[i >> 1], x);
            top_v[i >> 1] = fmaxf(top_v[i >> 1], x + ve[j >> 1]);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
          top_v[i] = fmaxf(top_v[i], __shfl_xor_sync(0xFFFFFFFFu, top_v[i], 1));
          top_v[i] = fmaxf(top_v[i], __shfl_xor_sync(0xFFFFFFFFu, top_v[i], 2));
          l[i] *= top[i] > m[i] ? gdn::exp2_approx(m[i] - top[i]) : 1.f;
          m[i] = top[i];
        }
        // The accumulators are rescaled only in the blocks that raise a maximum.
        if (__any_sync(0xFFFFFFFFu, top_v[0] > mv[0] || top_v[1] > mv[1])) {
          float r[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            r[i] = top_v[i] > mv[i] ? gdn::exp2_approx(mv[i] - top_v[i]) : 1.f;
            mv[i] = top_v[i];
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= r[0], o[i][1] *= r[0];
            o[i][2] *= r[1], o[i][3] *= r[1];
          }
        }
        uint32_t p[kSub][4];
#pragma unroll
        for (int j = 0; j < 2 * kSub; ++j) {
          float v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // A row that has seen nothing yet keeps m = -inf; its weights are 0.
            const bool none = s[j][i] == -INFINITY;
            v[i] = none ? 0.f : gdn::exp2_approx(s[j][i] + (ve[j >> 1] - (mv[i >> 1] - kShift)));
            l[i >> 1] += none ? 0.f : gdn::exp2_approx(s[j][i] - m[i >> 1]);
          }
          p[j >> 1][2 * (j & 1)] = gdn::pack_half2(v[0], v[1]);
          p[j >> 1][2 * (j & 1) + 1] = gdn::pack_half2(v[2], v[3]);
        }
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          // Codes of keys outside [lo, hi) are cleared: 0 * NaN would reach the sum.
          uint32_t keep = 0xFFFFFFFFu;
          if (edge) {
            keep = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = 16 * u + 4 * t + i;
              if (key >= lo && key < hi) keep |= 0xFFu << (8 * i);
            }
          }
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint32_t x[4];
            ldmatrix2_bytes_trans(vt + chunk_at<D>(row0 + 16 * u + (lane & 15), 2 * k + (lane >> 4)), x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t b0, b1;
              gdn::e4m3_to_half4(x[i] & keep, b0, b1);
              mma_16816(o[4 * k + i], p[u], b0, b1);
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
    for (int i = 0; i < 2; ++i) {
      const float f = mv[i] == -INFINITY ? 0.f : gdn::exp2_approx(mv[i] - m[i]);
#pragma unroll
      for (int k = 0; k < D / 8; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c) o[k][2 * i + c] = o[k][2 * i + c] * 0x1p-15f * f;
    }
    if (!end_segment<D>(d, sh, w, shares, rows, m, l, o)) return;
  }
}

template <int D>
int launch(const Decode8Args& base, const gdn_kv_cache_fp8* cache, const gdn_page_table* table, void* workspace, int sms,
           cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int smem = sizeof(Smem8<D>) + 1024;
  int rc = gdn_host::func_attr_once(decode_attention8_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, done);
  if (rc != GDN_OK) return rc;
  Decode8Args d = base;
  CUtensorMap k_map, v_map;
  if ((rc = gdn_host::encode_codes_map(&k_map, cache->k, cache, d.d.a.box_shift)) != GDN_OK) return rc;
  if ((rc = gdn_host::encode_codes_map(&v_map, cache->v, cache, d.d.a.box_shift)) != GDN_OK) return rc;
  return launch_shared<D>(d.d, table, workspace, sms, stream, [&](int grid) {
    return gdn_host::launch_pdl(decode_attention8_kernel<D>, dim3(grid), dim3(kThreads), smem, stream, d, k_map, v_map);
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
  return D == 64 ? launch<64>(d, cache, table, workspace, sms, s) : launch<128>(d, cache, table, workspace, sms, s);
}
