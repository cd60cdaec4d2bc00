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
#include "attention_common.cuh"

namespace {

using gdn::AttnArgs;
using gdn::SeqRange;

// Keys per stage: 16 KB each of K and V.
template <int D>
constexpr int kBlock = 8192 / D;
// Two stages, so 128 KB on their way per SM: with a third the queues before HBM
// grow and its rate falls (256 sequences, 8.5 GB: 1.23 ms against 1.17).
constexpr int kStages = 2;
constexpr int kConsumers = 4;  // warps, a quarter of a block's keys each
constexpr int kThreads = (kConsumers + 2) * 32;  // and one warp that copies keys, one that copies values
constexpr int kRows = 16;     // query heads of a key head at most (see gdn_attention_decode_paged)
// Fixed cost of an item (its queries, the join of the warps, its stores) in
// blocks, so that shares of many short items weigh the same as shares of long ones
// (512 sequences of 100 to 300 keys, 8 key heads of 128: 89 us, with 4 92).
constexpr int kItemCost = 2;
// Smallest piece in blocks (8 key heads of 128; 1 sequence of 1,000 / 16 of 250 / of
// 500: 9.8 / 10.9 / 12.5 us, with 4 10.9 / 11.5 / 12.5, with 8 13.6 / 13.3 / 15.0).
constexpr int kMinShare = 2;
constexpr int kMaxGrid = 2 * 160;  // two CTAs per SM
// Longest sequence that is never cut (one of 256 / 500: 6.6 / 9.2 us, cut 9.4 / 9.4;
// one of 1,000 / 2,000: 14.3 / 24.8 us, cut 9.8 / 10.4).
constexpr int kWholeKeys = 512;

struct DecodeArgs {
  AttnArgs a;
  float* part_o;     // [2 grid][kRows][D]
  float2* part_ml;   // [2 grid][kRows]
  int4* cuts;        // [grid]: (sequence, head, last CTA) of an item cut at this CTA's end, or -1
  int32_t whole;     // items are not cut
};

// The key range of sequence b's token in blocks, and its cost.
struct Item {
  SeqRange s;
  int lo, hi;      // visible keys
  int first;       // block of lo
  int blocks;
  int cost;        // 0: nothing to do
};
template <int D>
__device__ __forceinline__ Item load_item(const AttnArgs& a, int b) {
  Item it;
  it.s = gdn::seq_range(a.paged, b);
  it.hi = it.s.len;
  it.lo = gdn::key_lo(a, it.s.len - 1);
  it.first = it.lo / kBlock<D>;
  it.blocks = (it.hi + kBlock<D> - 1) / kBlock<D> - it.first;
  it.cost = it.s.new_tokens ? it.blocks + kItemCost : 0;
  return it;
}

// A CTA's share, walked item by item by producer and consumers alike.
struct Walk {
  int64_t pos, end;   // units of the batch's line (whole: item numbers)
  int64_t base;       // line position of sequence b
  int b;
  int head;
  Item it;
  int blk0, blk1;     // blocks of the item in this segment
  int64_t item0;      // line position of the item
};
template <int D>
__device__ __forceinline__ bool next_segment(const DecodeArgs& d, Walk& w) {
  const int per_seq = d.a.Hkv;
  if (d.whole) {
    while (w.pos < w.end) {
      const int id = static_cast<int>(w.pos);
      w.pos += gridDim.x;
      const int b = id / per_seq;
      if (b != w.b) w.b = b, w.it = load_item<D>(d.a, b);
      w.head = id - b * per_seq;
      w.blk0 = 0;
      w.blk1 = w.it.blocks;
      if (w.it.cost) return true;
    }
    return false;
  }
  while (w.pos < w.end) {
    const int64_t span = static_cast<int64_t>(w.it.cost) * per_seq;
    if (w.pos >= w.base + span) {
      w.base += span;
      w.it = load_item<D>(d.a, ++w.b);
      continue;
    }
    w.head = gdn::small_quotient(w.pos - w.base, w.it.cost, per_seq);
    w.item0 = w.base + static_cast<int64_t>(w.head) * w.it.cost;
    const int64_t stop = min(w.end, w.item0 + w.it.cost);
    w.blk0 = max(0, static_cast<int>(w.pos - w.item0) - kItemCost);
    w.blk1 = static_cast<int>(stop - w.item0) - kItemCost;
    w.pos = stop;
    if (w.blk1 > w.blk0) return true;
  }
  return false;
}

template <int D>
struct Smem {
  static constexpr int kTile = kBlock<D> * D * 2;  // one of K, V
  alignas(1024) uint8_t kv[kStages][2][kTile];
  float4 join_o[kConsumers][D / 8][32];  // the warps' partial results, lane by lane
  float4 join_ml[kConsumers][32];        // m, l of their two rows
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t never;  // the test hook's barrier, never completed
  int64_t scan[kThreads / 32 + 1];
  Walk walk;
  int abort;
  int stop;
};

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

// The loop out of line: this kernel's instructions are rarely in the cache (in line: 2
// short sequences 5.45 us instead of 5.35, 61 sequences 15.95 instead of 15.7).
static __device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, const volatile int* abort, uint32_t limit_ns) {
  return gdn::warp_wait_more(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort, uint32_t limit_ns) {
  if (__all_sync(0xFFFFFFFFu, gdn::mbar_try_wait(bar, parity))) return true;
  return wait_more(bar, parity, abort, limit_ns);
}

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    decode_attention_kernel(const __grid_constant__ DecodeArgs d, const __grid_constant__ CUtensorMap k_map,
                            const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ uint8_t raw[];
  Smem<D>& sh = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
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

  // ---- this CTA's share of the line ----
  const int per_seq = a.Hkv;
  Walk w;
  gdn::Shares<0> shares(0, 1, 1);
  if (d.whole) {
    w.pos = blockIdx.x;
    w.end = static_cast<int64_t>(a.paged.num_seqs) * per_seq;
    w.b = -1;
    if (blockIdx.x == 0)
      for (int b = tid; b < a.paged.num_seqs; b += kThreads)
        if (gdn::seq_range(a.paged, b).refused) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_TABLE, b);
    __syncthreads();
  } else {
    const int per = (a.paged.num_seqs + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.paged.num_seqs), b1 = min(b0 + per, a.paged.num_seqs);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      const Item it = load_item<D>(a, b);
      if (it.s.refused && blockIdx.x == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_TABLE, b);
      mine += it.cost;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sh.scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += sh.scan[i];
      total += sh.scan[i];
    }
    total *= per_seq;
    shares = gdn::Shares<0>(total, total / kMinShare, gridDim.x);
    const int c = blockIdx.x;
    const int64_t start = shares.start(c), end = shares.start(c + 1);
    // The thread whose sequences hold `start` sets up the walk.
    if (start < end && before * per_seq <= start && start < (before + mine) * per_seq) {
      Walk x;
      x.pos = start;
      x.end = end;
      x.base = before * per_seq;
      x.b = b0;
      x.it = load_item<D>(a, b0);
      while (start >= x.base + static_cast<int64_t>(x.it.cost) * per_seq) {
        x.base += static_cast<int64_t>(x.it.cost) * per_seq;
        x.it = load_item<D>(a, ++x.b);
      }
      sh.walk = x;
    }
    if (tid == 0) d.cuts[c] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    if (start >= end) return;
    w = sh.walk;
  }

  if (warp >= kConsumers) {
    // ------------------------------------------------ keys, or values
    const int kv = warp - kConsumers;
    gdn::TileCopies<D, kBlock<D>> tiles(a, kv ? &v_map : &k_map, lane);
    int n = 0;  // blocks issued
    bool ok = true;
    while (ok && next_segment<D>(d, w)) {
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
  while (next_segment<D>(d, w)) {
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

    // ---- join the four warps: each takes a quarter of the dimensions of all ----
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
    }
    consumers_sync();  // the last item's results have been read
#pragma unroll
    for (int i = 0; i < D / 8; ++i) sh.join_o[warp][i][lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
    sh.join_ml[warp][lane] = make_float4(m[0], m[1], l[0], l[1]);
    if (tid == 0) sh.stop = *static_cast<volatile int*>(&sh.abort);  // one reading for all warps
    consumers_sync();
    if (sh.stop) {
      if (tid == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_TIMEOUT, 0);
      return;
    }
    float f[kConsumers][2];
    {
      float4 ml[kConsumers];
#pragma unroll
      for (int v = 0; v < kConsumers; ++v) ml[v] = sh.join_ml[v][lane];
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
  }
}

// Joins the partial results of the items that CTAs of the kernel above cut: the
// item that CTA c started and did not end has slot 2 c + 1, then slot 0 of every
// CTA up to the one that ended it.  A thread takes one dimension of a row and every
// kGroups-th part, four of them in flight; the groups add up in a fixed order.
//   kGroups 1, many items, most cut in two: block c takes CTA c's cut, all rows at
//     once (61 sequences: the call takes 15.6 us, shared out as below 17.1).
//   kGroups 8, few items cut into many parts: the blocks share the rows of all cuts
//     out between them (4 sequences of 65,536 on one key head, 76 parts: 57 us with
//     one group, 33 with eight).
constexpr int kJoinThreads = 1024;
template <int D, int kGroups>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeArgs d, int ctas) {
  __shared__ int4 cuts[kGroups > 1 ? kMaxGrid : 1];  // with the CTA that made the cut
  __shared__ int count[kJoinThreads / 32];
  __shared__ float2 group_ml[kJoinThreads / D];
  __shared__ float group_o[kGroups > 1 ? kJoinThreads : 1];
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  const AttnArgs& a = d.a;
  const int tid = threadIdx.x, dim = tid % D, unit = tid / D, group = unit % kGroups;
  const int per_job = blockDim.x / D / kGroups;  // rows
  const int slices = (a.group + per_job - 1) / per_job;
  int job = blockIdx.x, jobs = 0, stride = gridDim.x;
  if constexpr (kGroups > 1) {
    // The cut items in the order of their CTAs, the same in every block.
    int4 mine = tid < ctas ? d.cuts[tid] : make_int4(-1, 0, 0, 0);
    mine.w = tid;
    const unsigned here = __ballot_sync(0xFFFFFFFFu, mine.x >= 0);
    if ((tid & 31) == 0) count[tid >> 5] = __popc(here);
    __syncthreads();
    int at = __popc(here & ((1u << (tid & 31)) - 1)), found = 0;
    for (int i = 0; i < blockDim.x / 32; ++i) {
      if (i < tid >> 5) at += count[i];
      found += count[i];
    }
    if (mine.x >= 0) cuts[at] = mine;
    __syncthreads();
    jobs = found * slices;
  } else {
    if (d.cuts[job].x < 0) return;
    job = 0, jobs = slices, stride = 1;
  }
  constexpr int kParts = 4;
  for (; job < jobs; job += stride) {
    int4 cut;
    if constexpr (kGroups > 1) {
      cut = cuts[job / slices];
    } else {
      cut = d.cuts[blockIdx.x];
      cut.w = blockIdx.x;
    }
    const int r = job % slices * per_job + unit / kGroups;
    float m = -INFINITY, l = 0.f, o = 0.f;
    if (r < a.group) {
      for (int i0 = cut.w + group; i0 <= cut.z; i0 += kParts * kGroups) {
        float2 ml[kParts];
        float x[kParts];
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          ml[p] = make_float2(-INFINITY, 0.f);
          const int i = i0 + p * kGroups;
          if (i > cut.z) continue;
          const int64_t at = (2 * static_cast<int64_t>(i) + (i == cut.w ? 1 : 0)) * kRows + r;
          ml[p] = d.part_ml[at];
          x[p] = d.part_o[at * D + dim];
        }
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          if (ml[p].x == -INFINITY) continue;  // no part
          const float top = fmaxf(m, ml[p].x);
          const float f = gdn::exp2_approx(m - top), g = gdn::exp2_approx(ml[p].x - top);
          m = top;
          o = o * f + x[p] * g;
          l = l * f + ml[p].y * g;
        }
      }
    }
    if constexpr (kGroups > 1) {
      __syncthreads();  // the last job's values have been read
      group_o[tid] = o;
      if (dim == 0) group_ml[unit] = make_float2(m, l);
      __syncthreads();
      if (group == 0) {
        for (int i = 1; i < kGroups; ++i) {
          const float2 ml = group_ml[unit + i];
          if (ml.x == -INFINITY) continue;
          const float top = fmaxf(m, ml.x);
          const float f = gdn::exp2_approx(m - top), g = gdn::exp2_approx(ml.x - top);
          m = top;
          o = o * f + group_o[tid + i * D] * g;
          l = l * f + ml.y * g;
        }
      }
    }
    if (group == 0 && r < a.group) {
      const int64_t row = static_cast<int64_t>(cut.x) * a.Hq + cut.y * a.group + r;
      a.o[row * D + dim] = __float2bfloat16(o / l);
      if (a.lse && dim == 0) a.lse[row] = (m + log2f(l)) / gdn::kLog2e;
    }
  }
}

// Where even the longest sequence is a few blocks, one CTA takes a whole item: the
// scan of the batch and the join's launch would cost more than the blocks.
bool whole_items(int32_t num_seqs, int32_t num_entries, int32_t page_size) {
  return gdn_host::longest_sequence(num_seqs, num_entries, page_size) <= kWholeKeys;
}
size_t workspace_bytes_of(int D, bool whole) {
  if (whole) return 0;
  return static_cast<size_t>(2) * kMaxGrid * kRows * (D * 4 + 8) + kMaxGrid * sizeof(int4);
}

template <int D>
int launch(const DecodeArgs& base, const gdn_kv_cache* cache, const gdn_page_table* table, void* workspace, int sms,
           cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int smem = sizeof(Smem<D>) + 1024;
  int rc = gdn_host::func_attr_once(decode_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, done);
  if (rc != GDN_OK) return rc;
  DecodeArgs d = base;
  CUtensorMap k_map, v_map;
  if ((rc = gdn_host::encode_cache_map(&k_map, cache->k, cache, d.a.box_shift)) != GDN_OK) return rc;
  if ((rc = gdn_host::encode_cache_map(&v_map, cache->v, cache, d.a.box_shift)) != GDN_OK) return rc;
  const int64_t items = static_cast<int64_t>(table->num_seqs) * d.a.Hkv;
  int grid = 2 * sms < kMaxGrid ? 2 * sms : kMaxGrid;
  if (d.whole && items < grid) grid = static_cast<int>(items);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  d.cuts = reinterpret_cast<int4*>(ws);
  d.part_ml = reinterpret_cast<float2*>(ws + kMaxGrid * sizeof(int4));
  d.part_o = reinterpret_cast<float*>(ws + kMaxGrid * sizeof(int4) + sizeof(float2) * 2 * kMaxGrid * kRows);
  rc = gdn_host::launch_pdl(decode_attention_kernel<D>, dim3(grid), dim3(kThreads), smem, stream, d, k_map, v_map);
  if (rc != GDN_OK || d.whole) return rc;
  if (items * 8 > grid) {
    const int rows = d.a.group * D > kJoinThreads ? kJoinThreads / D : d.a.group;
    return gdn_host::launch_pdl(decode_join_kernel<D, 1>, dim3(grid), dim3(rows * D), 0, stream, d, grid);
  }
  const int per_job = kJoinThreads / D / 8;
  const int64_t jobs = items * ((d.a.group + per_job - 1) / per_job);
  const int blocks = jobs < grid ? static_cast<int>(jobs) : grid;
  return gdn_host::launch_pdl(decode_join_kernel<D, 8>, dim3(blocks), dim3(kJoinThreads), 0, stream, d, grid);
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
