// attention_decode.cu -- paged attention of one new token per sequence.
//
// Mathematics: o = sum_j p_j v_j / sum_j p_j with p_j = 2^(x_j - m), x_j the
// score in units of log2 and m a running maximum; partial results (m, l, o) of
// disjoint key ranges join exactly by 2^(m_i - m).
//
// Bound: HBM.  Every key and value is read once, 4 D bytes per (key, head), for
// 4 D G flops (G query heads per key head), far below the ridge.  What the
// kernel needs is bytes in flight and equal shares:
//   - the whole batch is one line of blocks of 8,192 / D keys, (sequence, head) after
//     (sequence, head), and each CTA takes an equal piece of it, cutting
//     (sequence, head) items wherever the piece ends.  Every CTA derives its
//     piece from the page table itself: no planning launch, no host
//     synchronisation.  A cut item leaves partial results in the workspace, and
//     a small second kernel joins them in a fixed order.
//   - two warps keep two blocks of K and V (32 KB each) in flight by TMA, page by
//     page; two CTAs per SM.
//   - four consumer warps take a quarter of a block's keys each and never wait for one
//     another inside an item: mma.sync with the G query heads as the 16 rows
//     (the matrix work is a tenth of the copy time), private (m, l, o), joined
//     through shared memory when the item ends.
//
// Measured: 256 sequences of up to 32,768 tokens, 4 key heads of 128 (8.5 GB) 1.17 to
// 1.20 ms, 7.1 to 7.3 TB/s; 4 of 65,600, 8 key heads (1.07 GB) 157 us, 6.8 TB/s (a plain
// copy: 6.7).  61 sequences of up to 9,000 (65 MB) 15.7 us, under a cap 16.8: launch, the
// shares and the join are 7 of them; 2 short sequences 5.3 us are launch and latency
// alone.
#include "attention_decode.cuh"

namespace {

// Keys per stage: 16 KB each of K and V.
template <int D>
constexpr int kBlock = kTileBytes / (2 * D);
constexpr int kConsumers = 4;
constexpr int kThreads = threads_of(kConsumers);

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The end of an item's segment in the consumer warps: m, l and o of their two rows each
// (g and g + 8, in the fragment layout of the products) become the CTA's, a result or
// a part of one.  false: a wait ran out.
template <int D>
__device__ __forceinline__ bool end_segment(const DecodeArgs& d, Smem<kConsumers, D / 8, 1>& sh, const Walk& w,
                                            const gdn::Shares<0>& shares, int rows, float (&m)[2], float (&l)[2],
                                            const float (&o)[D / 8][4]) {
  const AttnArgs& a = d.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int g = lane >> 2, t = lane & 3;
  const int h0 = w.head * a.group;
  // ---- join the four warps: each takes a quarter of the dimensions of all ----
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
    l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
  }
  consumers_sync<kConsumers>();  // the last item's results have been read
#pragma unroll
  for (int i = 0; i < D / 8; ++i) sh.join_o[warp][i][lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
  sh.join_ml[warp][0][lane] = make_float4(m[0], m[1], l[0], l[1]);
  if (tid == 0) sh.stop = *static_cast<volatile int*>(&sh.abort);  // one reading for all warps
  consumers_sync<kConsumers>();
  if (sh.stop) {
    if (tid == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_TIMEOUT, 0);
    return false;
  }
  float f[kConsumers][2];
  {
    float4 ml[kConsumers];
#pragma unroll
    for (int v = 0; v < kConsumers; ++v) ml[v] = sh.join_ml[v][0][lane];
    m[0] = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
    m[1] = fmaxf(fmaxf(ml[0].y, ml[1].y), fmaxf(ml[2].y, ml[3].y));
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int v = 0; v < kConsumers; ++v) {
      f[v][0] = ml[v].x == -INFINITY ? 0.f : gdn::exp2_approx(ml[v].x - m[0]);
      f[v][1] = ml[v].y == -INFINITY ? 0.f : gdn::exp2_approx(ml[v].y - m[1]);
      l[0] = fmaf(ml[v].z, f[v][0], l[0]);
      l[1] = fmaf(ml[v].w, f[v][1], l[1]);
    }
  }
  const bool starts = w.blk0 == 0, ends = w.blk1 == w.it.blocks;
  // One segment of a CTA at most starts an item that it does not end, and one at
  // most continues one: two slots per CTA.
  const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (starts ? 1 : 0);
  const int64_t row0 = static_cast<int64_t>(w.b) * a.Hq + h0;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    const int at = warp * (D / 32) + k;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < kConsumers; ++v) {
      const float4 y = sh.join_o[v][at][lane];
      x[0] = fmaf(y.x, f[v][0], x[0]);
      x[1] = fmaf(y.y, f[v][0], x[1]);
      x[2] = fmaf(y.z, f[v][1], x[2]);
      x[3] = fmaf(y.w, f[v][1], x[3]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      if (r >= rows) continue;
      if (starts && ends)
        reinterpret_cast<uint32_t*>(a.o + (row0 + r) * D)[at * 4 + t] =
            gdn::pack_bf162(x[2 * i] / l[i], x[2 * i + 1] / l[i]);
      else
        reinterpret_cast<float2*>(d.part_o + (slot * kRows + r) * D)[at * 4 + t] = make_float2(x[2 * i], x[2 * i + 1]);
    }
  }
  if (warp == 0 && t == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      if (r >= rows) continue;
      if (!(starts && ends))
        d.part_ml[slot * kRows + r] = make_float2(m[i], l[i]);
      else if (a.lse)
        a.lse[row0 + r] = (m[i] + log2f(l[i])) / gdn::kLog2e;
    }
  }
  if (tid == 0 && starts && !ends)
    d.cuts[blockIdx.x] = make_int4(w.b, w.head, shares.owner(w.item0 + w.it.cost - 1), 0);
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    decode_attention_kernel(const __grid_constant__ DecodeArgs d, const __grid_constant__ CUtensorMap k_map,
                            const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ uint8_t raw[];
  Smem<kConsumers, D / 8, 1>& sh = *reinterpret_cast<Smem<kConsumers, D / 8, 1>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
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
  if (!take_share<kBlock<D>, kItemCost16>(d, sh, w, shares)) return;

  if (warp >= kConsumers) {
    // ------------------------------------------------ keys, or values
    const int kv = warp - kConsumers;
    gdn::TileCopies<D, kBlock<D>> tiles(a, kv ? &v_map : &k_map, lane);
    int n = 0;  // blocks issued
    bool ok = true;
    while (ok && next_segment<kBlock<D>, kItemCost16>(d, w)) {
      tiles.begin(w.it.lo, w.it.hi, w.head, w.b, w.it.s.entry, (w.it.first + w.blk0) * kBlock<D>);
      for (int blk = w.blk0; blk < w.blk1; ++blk, ++n) {
        const int stage = n % kStages;
        if (n >= kStages) ok = warp_wait(&sh.empty[stage], ((n / kStages) - 1) & 1, &sh.abort, a.wait_ns);
        if (!ok) break;
        if (lane == 0) gdn::mbar_arrive_expect_tx(&sh.full[stage], tiles.bytes());
        __syncwarp();
        tiles.copy(sh.kv[stage][kv], &sh.full[stage], blk + 1 < w.blk1);
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
  while (next_segment<kBlock<D>, kItemCost16>(d, w)) {
    const int h0 = w.head * a.group;  // first query head of the rows
    const int rows = a.group;
    // Queries as A fragments; rows past the group are zero.
    uint32_t q[D / 16][4];
    {
      const __nv_bfloat16* base = a.q + static_cast<int64_t>(w.b) * a.q_stride + static_cast<int64_t>(h0) * D;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = g + (i & 1) * 8, c = k * 16 + 2 * t + (i >> 1) * 8;
          q[k][i] = r < rows ? *reinterpret_cast<const uint32_t*>(base + r * D + c) : 0u;
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
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

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
        float s[2 * kSub][4] = {};
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            uint32_t b[4];
            const uint32_t r = row0 + 16 * u + (lane >> 4) * 8 + (lane & 7), c = 2 * k + ((lane >> 3) & 1);
            ldmatrix4(kt + (c >> 3) * (kBlock<D> * 128) + gdn::swz(r, c & 7), b);
            mma_16816(s[2 * u], q[k], b[0], b[1]);
            mma_16816(s[2 * u + 1], q[k], b[2], b[3]);
          }
        const bool edge = lo > 0 || hi < 16 * kSub;
        float top[2] = {m[0], m[1]};
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
#pragma unroll
        for (int j = 0; j < 2 * kSub; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = s[j][i];
            const int key = j * 8 + 2 * t + (i & 1);
            if (a.slopes) x = fmaf(-slope[i >> 1], static_cast<float>(w.it.s.len - 1 - (key0 + key)), x);
            if (edge && (key < lo || key >= hi)) x = -INFINITY;
            s[j][i] = x;
            top[i >> 1] = fmaxf(top[i >> 1], x);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
        }
        // The accumulators are rescaled only in the blocks that raise a maximum.
        if (__any_sync(0xFFFFFFFFu, top[0] > m[0] || top[1] > m[1])) {
          float r[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            r[i] = top[i] > m[i] ? gdn::exp2_approx(m[i] - top[i]) : 1.f;
            m[i] = top[i];
            l[i] *= r[i];
          }
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= r[0], o[i][1] *= r[0];
            o[i][2] *= r[1], o[i][3] *= r[1];
          }
        }
        // Weights: fp32 into the sum, bf16 (as the values are) into the product.
        uint32_t p[kSub][4];
#pragma unroll
        for (int j = 0; j < 2 * kSub; ++j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // A row that has seen nothing yet keeps m = -inf; its weights are 0.
            s[j][i] = s[j][i] == -INFINITY ? 0.f : gdn::exp2_approx(s[j][i] - m[i >> 1]);
            l[i >> 1] += s[j][i];
          }
          p[j >> 1][2 * (j & 1)] = gdn::pack_bf162(s[j][0], s[j][1]);
          p[j >> 1][2 * (j & 1) + 1] = gdn::pack_bf162(s[j][2], s[j][3]);
        }
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          // Values of keys outside [lo, hi) are cleared: 0 * NaN would reach the sum.
          uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
          if (edge) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int key = 16 * u + 2 * t + 8 * i;
              keep[i] = ((key >= lo && key < hi) ? 0x0000FFFFu : 0u) | ((key + 1 >= lo && key + 1 < hi) ? 0xFFFF0000u : 0u);
            }
          }
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            const uint32_t r = row0 + 16 * u + ((lane >> 3) & 1) * 8 + (lane & 7), c = 2 * k + (lane >> 4);
            ldmatrix4_trans(vt + (c >> 3) * (kBlock<D> * 128) + gdn::swz(r, c & 7), b);
            mma_16816(o[2 * k], p[u], b[0] & keep[0], b[1] & keep[1]);
            mma_16816(o[2 * k + 1], p[u], b[2] & keep[0], b[3] & keep[1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) gdn::mbar_arrive(&sh.empty[stage]);
    }

    if (!end_segment<D>(d, sh, w, shares, rows, m, l, o)) return;
  }
}

template <int D>
int launch(const DecodeArgs& base, const gdn_kv_cache* cache, const gdn_page_table* table, void* workspace, int sms,
           cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int smem = sizeof(Smem<kConsumers, D / 8, 1>) + 1024;
  int rc = gdn_host::func_attr_once(decode_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, done);
  if (rc != GDN_OK) return rc;
  DecodeArgs d = base;
  CUtensorMap k_map, v_map;
  if ((rc = gdn_host::encode_cache_map(&k_map, cache->k, cache, d.a.box_shift)) != GDN_OK) return rc;
  if ((rc = gdn_host::encode_cache_map(&v_map, cache->v, cache, d.a.box_shift)) != GDN_OK) return rc;
  return launch_shared<D>(d, table, workspace, sms, stream, [&](int grid) {
    return gdn_host::launch_pdl(decode_attention_kernel<D>, dim3(grid), dim3(kThreads), smem, stream, d, k_map, v_map);
  });
}

}  // namespace

extern "C" size_t gdn_attention_decode_workspace_bytes(int32_t num_seqs, int32_t Hq, int32_t Hkv, int32_t D,
                                                       int32_t num_entries, int32_t page_size) {
  if (Hkv >= 1 && Hq / Hkv > kRows)  // see gdn_attention_decode_paged
    return gdn_attention_workspace_bytes(num_seqs, num_seqs, Hq, Hkv, D, num_entries, page_size);
  if (num_seqs < 0 || num_entries < 0 || page_size < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
  return workspace_bytes_of(D, whole_items(num_seqs, num_entries, page_size));
}

extern "C" int gdn_attention_decode_paged(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* o, float* lse,
                                          int32_t Hq, const gdn_kv_cache* cache, const gdn_page_table* table,
                                          float scale, const gdn_attention_options* options, void* workspace,
                                          size_t workspace_bytes, int32_t* err_word, void* stream) {
  // More query heads per key head than this kernel's rows would read the cache once
  // for every sixteen; the chunk kernel has 128 rows (64 sequences of 8,192, 17 / 64
  // / 128 query heads on one key head: 87 / 160 / 229 us here, 58 / 59 / 61 there;
  // 16: 53 here, 58 there).
  if (cache && cache->num_heads >= 1 && Hq / cache->num_heads > kRows)
    return gdn_attention_paged(q, q_token_stride, o, lse, nullptr, table ? table->num_seqs : 0, Hq, cache, table, scale,
                               options, workspace, workspace_bytes, err_word, stream);
  DecodeArgs d = {};
  const int32_t n = table ? table->num_seqs : 0;
  d.whole = cache && table && whole_items(n, table->num_entries, cache->page_size);
  const size_t need = cache ? workspace_bytes_of(cache->head_dim, d.whole) : 0;
  int rc = gdn_host::attention_args(&d.a, q, q_token_stride, o, lse, nullptr, n, Hq, cache, table, scale, options,
                                    workspace, workspace_bytes, need, err_word, cache && cache->head_dim == 64 ? kBlock<64> : kBlock<128>);
  if (rc != GDN_OK || n == 0) return rc;
  int sms = 0;
  rc = gdn_host::check_device(&sms);
  if (rc != GDN_OK) return rc;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cache->head_dim == 64 ? launch<64>(d, cache, table, workspace, sms, s)
                               : launch<128>(d, cache, table, workspace, sms, s);
}
