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
//     registers), one warp that issues the products, one that copies pages by
//     TMA, one that clears the value rows of keys no row may see.
//   - The batch is one line of (sequence, token tile, key head) items, as long as
//     their key ranges, and each CTA takes an equal piece of it, cutting items
//     where the piece ends (as the decode kernel does); the line's prefix sums
//     have closed forms, so that every CTA finds its piece from the page table
//     itself.  A join kernel adds up the cut items.
#include "attention_common.cuh"

namespace {

using gdn::AttnArgs;

constexpr int kRows = 128;   // rows per tile
constexpr int kKeys = 128;   // keys per block
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kClearWarp = 10, kAllocWarp = 11;
// Fixed cost of an item (queries, pipeline fill, epilogue) in keys.
constexpr int kItemCost = 2 * kKeys;
constexpr int kMinShare = 4 * kKeys;  // keys below which a cut costs more than it saves
constexpr int kMaxGrid = 160;         // one CTA per SM

struct ChunkArgs {
  AttnArgs a;
  int32_t tile_tokens;  // tokens per tile: 128 / group
  float4* part_o;       // [2 grid][2 tiles][D / 4][128 rows]
  float2* part_ml;      // [2 grid][2 tiles][128 rows]
  int4* cuts;           // [grid]: (sequence, token tile pair, key head, last CTA) of an item cut at this CTA's end, or -1
};

struct Seq {
  int first_token, n, len, entry, full;
  int pairs;  // token tile pairs
  bool refused;
};
__device__ __forceinline__ Seq load_seq(const ChunkArgs& d, int b) {
  const gdn::SeqRange s = gdn::seq_range(d.a.paged, b);
  Seq q;
  q.first_token = s.first_token;
  q.n = s.new_tokens;
  q.len = s.len;
  q.entry = s.entry;
  q.refused = s.refused;
  q.full = d.a.full_lens && s.new_tokens ? min(d.a.full_lens[b], s.len) : 0;
  q.pairs = (s.new_tokens + 2 * d.tile_tokens - 1) / (2 * d.tile_tokens);
  return q;
}
// Visible keys [lo, hi) of tile pair i of a sequence.
__device__ __forceinline__ int pair_lo(const ChunkArgs& d, const Seq& s, int i) {
  return gdn::key_lo(d.a, s.len - s.n + i * 2 * d.tile_tokens);
}
__device__ __forceinline__ int pair_hi(const ChunkArgs& d, const Seq& s, int i) {
  return max(s.len - s.n + min(s.n, (i + 1) * 2 * d.tile_tokens), s.full);
}
__device__ __forceinline__ int pair_cost(const ChunkArgs& d, const Seq& s, int i) {
  return pair_hi(d, s, i) - pair_lo(d, s, i) + kItemCost;
}
// sum over i < n of max(c, a + i step).
__device__ __forceinline__ int64_t sum_max(int64_t c, int64_t a, int64_t step, int64_t n) {
  int64_t k = c > a ? (c - a + step - 1) / step : 0;  // the first k terms are c
  k = k < n ? k : n;
  return c * k + a * (n - k) + step * (n * (n - 1) - k * (k - 1)) / 2;
}
// sum of pair_cost over the pairs before i (i < pairs: all of them full).
__device__ __forceinline__ int64_t cost_before(const ChunkArgs& d, const Seq& s, int i) {
  const int64_t p = s.len - s.n, step = 2 * d.tile_tokens;
  int64_t sum = sum_max(s.full, p + step, step, i) + static_cast<int64_t>(i) * kItemCost;
  if (d.a.window >= 0) sum -= sum_max(0, p - d.a.window, step, i);
  return sum;
}
__device__ __forceinline__ int64_t seq_cost(const ChunkArgs& d, const Seq& s) {
  return s.pairs ? cost_before(d, s, s.pairs - 1) + pair_cost(d, s, s.pairs - 1) : 0;
}

// A CTA's share of the line, walked item by item by every role alike.
struct Walk {
  int64_t pos, end;  // line positions
  int64_t item0;     // of the current item
  int b, pair, head, cost;
  Seq s;
  // The current segment:
  int lo, hi;        // keys that the item's rows see between them
  int first;         // block of lo
  int blocks;        // of the item
  int blk0, blk1;    // of this segment
};
__device__ __forceinline__ bool next_segment(const ChunkArgs& d, Walk& w) {
  while (w.pos < w.end) {
    if (w.pos >= w.item0 + w.cost) {
      w.item0 += w.cost;
      if (++w.head == d.a.Hkv) {
        w.head = 0;
        if (++w.pair >= w.s.pairs) {
          w.pair = 0;
          do w.s = load_seq(d, ++w.b);
          while (w.s.pairs == 0);
        }
        w.cost = pair_cost(d, w.s, w.pair);
      }
      continue;
    }
    w.lo = pair_lo(d, w.s, w.pair);
    w.hi = pair_hi(d, w.s, w.pair);
    w.first = w.lo / kKeys;
    w.blocks = (w.hi + kKeys - 1) / kKeys - w.first;
    const int64_t stop = min(w.end, w.item0 + w.cost);
    w.blk0 = max(0, (static_cast<int>(w.pos - w.item0) - kItemCost) / kKeys);
    w.blk1 = stop == w.item0 + w.cost ? w.blocks : max(0, (static_cast<int>(stop - w.item0) - kItemCost) / kKeys);
    w.pos = stop;
    if (w.blk1 > w.blk0) return true;
  }
  return false;
}
// Keys of the block that no row of the item sees.
__device__ __forceinline__ bool needs_clearing(const Walk& w, int key0) { return key0 < w.lo || key0 + kKeys > w.hi; }
__device__ __forceinline__ int64_t share_start(int64_t total, int eff, int c) { return total * c / eff; }
__device__ __forceinline__ int share_owner(int64_t total, int eff, int64_t x) {
  int c = static_cast<int>(x * eff / total);
  while (c + 1 < eff && share_start(total, eff, c + 1) <= x) ++c;
  while (share_start(total, eff, c) > x) --c;
  return c;
}

template <int D>
struct Layout {
  static constexpr int kHalf = kRows * 128;            // 64 dimensions of 128 rows
  static constexpr int kTile = kRows * D * 2;          // a Q, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 8;     // ring of K and V tiles
  static constexpr int kBytes = (2 + kStages) * kTile;
  static constexpr uint32_t kColS = 0, kColO = 256;    // TMEM columns: S of both tiles, O of both tiles
};

template <int D>
struct Smem {
  uint64_t full[Layout<D>::kStages];
  uint64_t empty[Layout<D>::kStages];
  uint64_t raw[Layout<D>::kStages];  // copies of values that are to be cleared before they are `full`
  uint64_t q_full, q_empty, done;
  uint64_t s_full[2], p_full[2], o_full[2];
  int64_t scan[kThreads / 32];
  Walk walk;
  Walk softmax_walk[8];  // one per softmax warp, kept here: its registers hold scores
  uint32_t tmem;
  int abort;
};

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// A bounded wait, in line: with a function call in the kernel the register split
// below cannot be allocated.
__device__ __forceinline__ bool wait_inline(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  if (gdn::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = gdn::globaltimer_ns();
  while (!gdn::mbar_try_wait_suspend(bar, parity))
    if (*abort || gdn::globaltimer_ns() - t0 > 2000000000ull) return false;
  return true;
}

// 128 fp32 columns of this thread's TMEM lane: four loads in flight, one wait.
// The registers pass through the wait, so that no use is scheduled before it.
__device__ __forceinline__ void tmem_ld32_nw(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void pin32(float* r) {
  asm volatile(""
               : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                 "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                 "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]),
                 "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]),
                 "+f"(r[30]), "+f"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, float (&r)[128]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) tmem_ld32_nw(taddr + 32 * i, r + 32 * i);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) pin32(r + 32 * i);
}
__device__ __forceinline__ void tmem_st32_nw(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, "
      "%25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// kMods: scores are capped or biased (the options that change a score; those
// that only hide keys cost nothing away from the edges).
template <int D, bool kMods>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attention_kernel(const __grid_constant__ ChunkArgs d, const __grid_constant__ CUtensorMap q_map,
                           const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using L = Layout<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Smem<D>& sh = *reinterpret_cast<Smem<D>*>(tiles + L::kBytes);
  uint8_t* ring = tiles + 2 * L::kTile;
  const AttnArgs& a = d.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* const abort_flag = &sh.abort;

  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      gdn::mbar_init(&sh.full[i], 1);
      gdn::mbar_init(&sh.empty[i], 1);
      gdn::mbar_init(&sh.raw[i], 1);
    }
    gdn::mbar_init(&sh.q_full, 1);
    gdn::mbar_init(&sh.q_empty, 1);
    gdn::mbar_init(&sh.done, 1);
    for (int t = 0; t < 2; ++t) {
      gdn::mbar_init(&sh.s_full[t], 1);
      gdn::mbar_init(&sh.p_full[t], 4);
      gdn::mbar_init(&sh.o_full[t], 1);
    }
    sh.abort = 0;
    gdn::fence_mbar_init();
  }
  // Rows past the group's share of a tile are never copied; they start at zero.
  for (int i = tid; i < 2 * L::kTile / 16; i += kThreads) reinterpret_cast<uint4*>(tiles)[i] = make_uint4(0, 0, 0, 0);
  if (warp == kAllocWarp) {
    gdn::tmem_alloc(&sh.tmem, 512);
    gdn::tmem_relinquish();
  }
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();

  // ---- this CTA's share of the line ----
  int64_t total = 0;
  int eff = gridDim.x;
  bool idle;
  {
    const int per = (a.paged.num_seqs + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.paged.num_seqs), b1 = min(b0 + per, a.paged.num_seqs);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      const Seq s = load_seq(d, b);
      if (s.refused && blockIdx.x == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_TABLE, b);
      mine += seq_cost(d, s);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sh.scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += sh.scan[i];
      total += sh.scan[i];
    }
    total *= a.Hkv;
    const int64_t most = total / kMinShare;
    eff = static_cast<int>(most < 1 ? 1 : most < gridDim.x ? most : gridDim.x);
    const int c = blockIdx.x;
    const int64_t start = c < eff ? share_start(total, eff, c) : total;
    const int64_t end = c < eff ? share_start(total, eff, c + 1) : total;
    idle = start >= end;
    // The thread whose sequences hold `start` sets up the walk.
    if (!idle && before * a.Hkv <= start && start < (before + mine) * a.Hkv) {
      Walk x;
      x.pos = start;
      x.end = end;
      x.b = b0;
      int64_t base = before * a.Hkv;
      for (;; ++x.b) {
        x.s = load_seq(d, x.b);
        const int64_t span = seq_cost(d, x.s) * a.Hkv;
        if (start < base + span) break;
        base += span;
      }
      int i = 0;  // the last pair that begins at or before start
      for (int step = 1 << 30; step; step >>= 1)
        if (step < x.s.pairs - i && cost_before(d, x.s, i + step) * a.Hkv <= start - base) i += step;
      x.pair = i;
      x.cost = pair_cost(d, x.s, i);
      base += cost_before(d, x.s, i) * a.Hkv;
      x.head = static_cast<int>((start - base) / x.cost);
      x.item0 = base + static_cast<int64_t>(x.head) * x.cost;
      sh.walk = x;
    }
    if (tid == 0) d.cuts[c] = make_int4(-1, 0, 0, 0);
  }
  gdn::fence_proxy_async();
  gdn::tc_fence_before();
  __syncthreads();
  gdn::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int tile_tokens = d.tile_tokens;

  if (idle) {
    // nothing to do but to give TMEM back below
  } else if (warp >= 8) {
    regs_dec<88>();
    Walk w = sh.walk;
    bool ok = true;
    if (warp == kLoadWarp) {
      // ------------------------------------------------------------- copies
      int n = 0, seg = 0;                    // tiles issued, segments begun
      uint32_t raw_parity = 0, raw_last = 0;  // per stage: parity of its next raw copy; its last copy was one
      const int boxes = kKeys / a.box_rows;
      while (ok && next_segment(d, w)) {
        const int token = w.s.first_token + w.pair * 2 * tile_tokens;
        const bool two = w.pair * 2 * tile_tokens + tile_tokens < w.s.n;
        for (int blk = w.blk0; ok && blk < w.blk1; ++blk) {
          const int key0 = (w.first + blk) * kKeys;
          const int first = max(0, w.lo - key0) / a.box_rows;
          const int last = (min(kKeys, w.hi - key0) + a.box_rows - 1) / a.box_rows;
          int page[4], slot[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int box = lane + 32 * i;
            if (32 * i < boxes && box >= first && box < last) {
              const int key = key0 + box * a.box_rows;
              const int entry = key / a.paged.page_size;
              slot[i] = key - entry * a.paged.page_size;
              page[i] = a.paged.pages[w.s.entry + entry];
              if (page[i] < 0 || page[i] >= a.paged.num_pages) {
                gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_ID, w.b);
                page[i] = a.paged.num_pages;  // outside the map: zeros
              }
            }
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int stage = n % L::kStages;
            const bool clear = kv && needs_clearing(w, key0);
            uint64_t* bar = clear ? &sh.raw[stage] : &sh.full[stage];
            if (lane == 0) {
              if (n >= L::kStages)
                ok = wait_inline(&sh.empty[stage], ((n / L::kStages) - 1) & 1, abort_flag);
              if (ok) gdn::mbar_arrive_expect_tx(bar, (last - first) * a.box_rows * D * 2);
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            raw_last = clear ? raw_last | (1u << stage) : raw_last & ~(1u << stage);
            raw_parity ^= clear ? 1u << stage : 0u;
            uint8_t* dst = ring + stage * L::kTile;
            const CUtensorMap* map = kv ? &v_map : &k_map;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int box = lane + 32 * i;
              if (32 * i < boxes && box >= first && box < last) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                  gdn::tma_load_4d(dst + c * L::kHalf + box * a.box_rows * 128, map, bar, c * 64, w.head,
                                   slot[i], page[i]);
              }
            }
            __syncwarp();
          }
          // The queries, behind the first block's keys and values: those need
          // no room that the segment before still holds.
          if (ok && blk == w.blk0) {
            if (lane == 0) {
              if (seg > 0) ok = wait_inline(&sh.q_empty, (seg - 1) & 1, abort_flag);
              if (ok) {
                const int bytes = a.group * tile_tokens * D * 2;
                gdn::mbar_arrive_expect_tx(&sh.q_full, two ? 2 * bytes : bytes);
                for (int t = 0; t < (two ? 2 : 1); ++t)
                  for (int c = 0; c < D / 64; ++c)
                    gdn::tma_load_4d(tiles + t * L::kTile + c * L::kHalf, &q_map, &sh.q_full, c * 64, 0,
                                     token + t * tile_tokens, w.head);
              }
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            ++seg;
          }
        }
      }
      if (!ok && lane == 0) {
        // Leave no copy in flight behind (bounded waits, as everywhere).
        *abort_flag = 1;
        for (int i = max(0, n - L::kStages); i < n; ++i) {
          const int stage = i % L::kStages;
          if ((raw_last >> stage) & 1)
            gdn::mbar_wait(&sh.raw[stage], ((raw_parity >> stage) & 1) ^ 1);
          else
            gdn::mbar_wait(&sh.full[stage], (i / L::kStages) & 1);
        }
        if (seg > 0) gdn::mbar_wait(&sh.q_full, (seg - 1) & 1);
      }
    } else if (warp == kMmaWarp) {
      // ----------------------------------------------------------- products
      if (lane == 0) {
        const uint32_t id_s = gdn::idesc_f16(kRows, kKeys, true, true, false, false);
        const uint32_t id_o = gdn::idesc_f16(kRows, D, true, true, false, true);
        const uint32_t q_addr = gdn::smem_u32(tiles), ring_addr = gdn::smem_u32(ring);
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          ok = ok && wait_inline(bar, parity, abort_flag);
          return ok;
        };
        // S_t = Q_t K^T
        auto scores = [&](int t, int stage) {
          const uint64_t qd = gdn::sdesc(q_addr + t * L::kTile, 16, 1024);
          const uint64_t kd = gdn::sdesc(ring_addr + stage * L::kTile, 16, 1024);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            gdn::tc_mma4(tmem + L::kColS + t * kKeys, qd + c * (L::kHalf >> 4), 2, kd + c * (L::kHalf >> 4), 2, id_s, c);
          gdn::tc_commit(&sh.s_full[t]);
        };
        // O_t += P_t V, P_t in TMEM over the first half of S_t
        auto values = [&](int t, int stage, uint32_t acc) {
          const uint64_t vd = gdn::sdesc(ring_addr + stage * L::kTile, L::kHalf, 1024);
          const uint32_t p = tmem + L::kColS + t * kKeys, o = tmem + L::kColO + t * D;
          gdn::tc_mma4_ts(o, p, 8, vd, 128, id_o, acc);
          gdn::tc_mma4_ts(o, p + 32, 8, vd + 4 * 128, 128, id_o, 1);
          gdn::tc_commit(&sh.o_full[t]);
        };
        uint32_t n = 0, seg = 0, np[2] = {0, 0};  // ring tiles, segments, weights taken
        while (ok && next_segment(d, w)) {
          const bool two = w.pair * 2 * tile_tokens + tile_tokens < w.s.n;
          const int nb = w.blk1 - w.blk0;
          wait(&sh.q_full, seg & 1);
          ++seg;
          if (!wait(&sh.full[n % L::kStages], (n / L::kStages) & 1)) break;
          gdn::tc_fence_after();
          scores(0, n % L::kStages);
          if (two) scores(1, n % L::kStages);
          gdn::tc_commit(&sh.empty[n % L::kStages]);
          if (nb == 1) gdn::tc_commit(&sh.q_empty);
          ++n;
          for (int j = 0; j < nb; ++j) {
            const uint32_t v = n, k = n + 1;  // ring tiles of V(j) and K(j + 1)
            const bool more = j + 1 < nb;
            wait(&sh.full[v % L::kStages], (v / L::kStages) & 1);
            if (!wait(&sh.p_full[0], np[0]++ & 1)) break;
            gdn::tc_fence_after();
            values(0, v % L::kStages, j > 0);
            if (more) {
              if (!wait(&sh.full[k % L::kStages], (k / L::kStages) & 1)) break;
              gdn::tc_fence_after();
              scores(0, k % L::kStages);
            }
            if (two) {
              if (!wait(&sh.p_full[1], np[1]++ & 1)) break;
              gdn::tc_fence_after();
              values(1, v % L::kStages, j > 0);
            }
            gdn::tc_commit(&sh.empty[v % L::kStages]);
            if (more) {
              if (two) scores(1, k % L::kStages);
              gdn::tc_commit(&sh.empty[k % L::kStages]);
              if (j + 2 == nb) gdn::tc_commit(&sh.q_empty);
            }
            n += more ? 2 : 1;
          }
        }
        if (!ok) *abort_flag = 1;
        // Every product is complete before TMEM is given back.
        gdn::tc_commit(&sh.done);
        gdn::mbar_wait(&sh.done, 0);
      }
      __syncwarp();
    } else if (warp == kClearWarp) {
      // ------------------------------ value rows that no row of the item sees
      // Slots past the sequence's end or before every window may hold anything,
      // and 0 * NaN would reach the sum: they become zeros in shared memory.
      // Their copies complete on `raw`, and this warp completes `full`.
      uint32_t n = 0, raw_parity = 0;
      while (ok && next_segment(d, w)) {
        for (int blk = w.blk0; blk < w.blk1; ++blk, n += 2) {
          const int key0 = (w.first + blk) * kKeys;
          if (!needs_clearing(w, key0)) continue;
          const uint32_t stage = (n + 1) % L::kStages;  // K, V, K, V, ...
          ok = wait_inline(&sh.raw[stage], (raw_parity >> stage) & 1, abort_flag);
          raw_parity ^= 1u << stage;
          if (!__all_sync(0xFFFFFFFFu, ok)) {
            ok = false;
            break;
          }
          uint8_t* dst = ring + stage * L::kTile;
          const int from = max(0, w.lo - key0), to = min(kKeys, w.hi - key0);
          for (int i = lane; i < kKeys * D / 8; i += 32) {
            const int row = (i >> 3) & (kKeys - 1);
            if (row < from || row >= to) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0, 0, 0, 0);
          }
          gdn::fence_proxy_async();
          __syncwarp();
          if (lane == 0) gdn::mbar_arrive(&sh.full[stage]);
        }
      }
      if (!ok) *abort_flag = 1;
    }
  } else {
    // --------------------------------------------------------------- softmax
    regs_inc<208>();
    Walk& w = sh.softmax_walk[warp];
    if (lane == 0) w = sh.walk;
    auto next = [&] {
      int more = 0;
      __syncwarp();
      if (lane == 0) more = next_segment(d, w);
      return __shfl_sync(0xFFFFFFFFu, more, 0) != 0;
    };
    const int t = warp >> 2;                       // tile
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 (warp % 4)
    const uint32_t s_addr = tmem + L::kColS + t * kKeys + lane_bits, o_addr = tmem + L::kColO + t * D + lane_bits;
    const int my_token = row / a.group, my_head = row % a.group;
    uint32_t n = 0;  // blocks taken
    bool ok = true;
    while (ok && next()) {
      const int first_token = (w.pair * 2 + t) * tile_tokens;  // of the tile, within the new tokens
      if (first_token >= w.s.n) continue;
      const int token = first_token + my_token;
      const bool valid = my_token < tile_tokens && token < w.s.n;
      // Rows without a token copy the range of the tile's last one.
      const int pos = w.s.len - w.s.n + min(min(token, first_token + tile_tokens - 1), w.s.n - 1);
      const int lo = gdn::key_lo(a, pos), hi = max(pos + 1, w.s.full);
      float slope = 0.f;
      if (kMods && a.slopes) slope = a.slopes[w.head * a.group + my_head] * gdn::kLog2e;
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      for (int blk = w.blk0; blk < w.blk1; ++blk, ++n) {
        const int key0 = (w.first + blk) * kKeys;
        ok = wait_inline(&sh.s_full[t], n & 1, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        gdn::tc_fence_after();
        float s[128];
        tmem_ld128(s_addr, s);
        if (kMods) {
          if (a.cap_log2 > 0.f) {
#pragma unroll
            for (int i = 0; i < 128; ++i) s[i] = gdn::capped(s[i] * a.scale_log2, a.cap_log2);
          } else {
#pragma unroll
            for (int i = 0; i < 128; ++i) s[i] *= a.scale_log2;
          }
          if (a.slopes) {
            const float back = static_cast<float>(pos - key0);
#pragma unroll
            for (int i = 0; i < 128; ++i) s[i] = fmaf(-slope, fabsf(back - static_cast<float>(i)), s[i]);
          }
        }
        if (__any_sync(0xFFFFFFFFu, key0 < lo || key0 + kKeys > hi)) {
          const int from = lo - key0, to = hi - key0;
#pragma unroll
          for (int i = 0; i < 128; ++i) s[i] = i >= from && i < to ? s[i] : -INFINITY;
        }
        float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 128; ++i) top[i & 3] = fmaxf(top[i & 3], s[i]);
        float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        if (!kMods) mx *= a.scale_log2;
        // The reference moves when a maximum is more than 2^8 above it.
        const bool grow = mx > m + 8.f || (m == -INFINITY && mx > m);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float to = fmaxf(m, mx);
          const float r = m == -INFINITY ? 0.f : gdn::exp2_approx(m - to);
          m = to;
          l2 = __fmul2_rn(l2, make_float2(r, r));
          if (blk > w.blk0) {
            ok = wait_inline(&sh.o_full[t], (n - 1) & 1, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
              ok = false;
              break;
            }
            gdn::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float x[16];
              gdn::tmem_ld16(o_addr + c, x);
              uint32_t y[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(x[i] * r);
              gdn::tmem_st16(o_addr + c, y);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;  // a row that has seen no key yet: weights 2^-inf = 0
        const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), ref2 = make_float2(-ref, -ref);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float2 x = make_float2(s[64 * h + 2 * i], s[64 * h + 2 * i + 1]);
            x = kMods ? __fadd2_rn(x, ref2) : __ffma2_rn(x, scale2, ref2);
            x = make_float2(gdn::exp2_approx(x.x), gdn::exp2_approx(x.y));
            // fp32 into the sum; bf16, as the values are, into the product.
            l2 = __fadd2_rn(l2, x);
            p[i] = gdn::pack_bf162(x);
          }
          tmem_st32_nw(s_addr + 32 * h, p);
        }
        gdn::tmem_wait_st();
        gdn::tc_fence_before();
        __syncwarp();
        if (lane == 0) gdn::mbar_arrive(&sh.p_full[t]);
      }
      if (!ok) break;
      // ---- epilogue ----
      ok = wait_inline(&sh.o_full[t], (n - 1) & 1, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        ok = false;
        break;
      }
      gdn::tc_fence_after();
      const float l = l2.x + l2.y;
      const bool starts = w.blk0 == 0, ends = w.blk1 == w.blocks;
      if (starts && ends) {
        const float inv = 1.f / l;
        const int64_t out = (static_cast<int64_t>(w.s.first_token) + token) * a.Hq + w.head * a.group + my_head;
        uint4* dst = reinterpret_cast<uint4*>(a.o + out * D);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float x[32];
          gdn::tmem_ld32(o_addr + c, x);
          if (valid) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[c / 8 + i] =
                  make_uint4(gdn::pack_bf162(x[8 * i] * inv, x[8 * i + 1] * inv), gdn::pack_bf162(x[8 * i + 2] * inv, x[8 * i + 3] * inv),
                             gdn::pack_bf162(x[8 * i + 4] * inv, x[8 * i + 5] * inv), gdn::pack_bf162(x[8 * i + 6] * inv, x[8 * i + 7] * inv));
          }
        }
        if (valid && a.lse) a.lse[out] = (m + log2f(l)) / gdn::kLog2e;
      } else {
        // One segment of a CTA at most starts an item that it does not end, and
        // one at most continues one: two slots per CTA.
        const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (starts ? 1 : 0)) * 2 + t;
        float4* dst = d.part_o + slot * (D / 4) * kRows + row;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float x[32];
          gdn::tmem_ld32(o_addr + c, x);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[(c / 4 + i) * kRows] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
        d.part_ml[slot * kRows + row] = make_float2(m, l);
        if (starts && t == 0 && row == 0)
          d.cuts[blockIdx.x] = make_int4(w.b, w.pair, w.head, share_owner(total, eff, w.item0 + w.cost - 1));
      }
      // The next segment's first P V overwrites O: these loads come first.
      gdn::tc_fence_before();
    }
    if (!ok) *abort_flag = 1;
  }
  gdn::tc_fence_before();
  __syncthreads();
  gdn::tc_fence_after();
  if (tid == 0 && sh.abort) gdn::record_error(a.paged.err_word, GDN_DEVERR_TIMEOUT, 0);
  if (warp == kAllocWarp) gdn::tmem_dealloc(tmem, 512);
}

// Joins the partial results of the items that CTAs of the kernel above cut: the
// item that CTA c = blockIdx.x started and did not end has slot 1 of c, then slot
// 0 of every CTA up to the one that ended it.  blockIdx.y: 32 rows; a thread
// takes one row and every eighth group of four dimensions.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ ChunkArgs d) {
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  const int c = blockIdx.x;
  const int4 cut = d.cuts[c];
  if (cut.x < 0) return;
  const AttnArgs& a = d.a;
  const int t = blockIdx.y >> 2, row = (blockIdx.y & 3) * 32 + (threadIdx.x & 31);
  const gdn::SeqRange s = gdn::seq_range(a.paged, cut.x);
  const int in_tile = row / a.group;
  const int token = (cut.y * 2 + t) * d.tile_tokens + in_tile;
  if (in_tile >= d.tile_tokens || token >= s.new_tokens) return;
  constexpr int kG = D / 32;  // groups of four dimensions per thread
  float m = -INFINITY, l = 0.f;
  float4 o[kG];
#pragma unroll
  for (int k = 0; k < kG; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = c; i <= cut.w; ++i) {
    const int64_t slot = (2 * static_cast<int64_t>(i) + (i == c ? 1 : 0)) * 2 + t;
    const float2 ml = d.part_ml[slot * kRows + row];
    const float top = fmaxf(m, ml.x);
    const float ra = m == -INFINITY ? 0.f : gdn::exp2_approx(m - top);
    const float rb = ml.x == -INFINITY ? 0.f : gdn::exp2_approx(ml.x - top);
    l = l * ra + ml.y * rb;
    m = top;
#pragma unroll
    for (int k = 0; k < kG; ++k) {
      const float4 x = d.part_o[(slot * (D / 4) + (threadIdx.x >> 5) + 8 * k) * kRows + row];
      o[k].x = o[k].x * ra + x.x * rb;
      o[k].y = o[k].y * ra + x.y * rb;
      o[k].z = o[k].z * ra + x.z * rb;
      o[k].w = o[k].w * ra + x.w * rb;
    }
  }
  const float inv = 1.f / l;
  const int64_t out = (static_cast<int64_t>(s.first_token) + token) * a.Hq + cut.z * a.group + row % a.group;
#pragma unroll
  for (int k = 0; k < kG; ++k)
    reinterpret_cast<uint2*>(a.o + out * D)[(threadIdx.x >> 5) + 8 * k] =
        make_uint2(gdn::pack_bf162(o[k].x * inv, o[k].y * inv), gdn::pack_bf162(o[k].z * inv, o[k].w * inv));
  if (a.lse && threadIdx.x < 32) a.lse[out] = (m + log2f(l)) / gdn::kLog2e;
}

constexpr size_t kCutBytes = kMaxGrid * sizeof(int4);
size_t workspace_bytes_of(int D) {
  return kCutBytes + static_cast<size_t>(4) * kMaxGrid * kRows * (sizeof(float2) + D * sizeof(float));
}

template <int D, bool kMods>
int launch(ChunkArgs d, int32_t total_tokens, const gdn_kv_cache* cache, void* workspace, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  constexpr int smem = Layout<D>::kBytes + sizeof(Smem<D>) + 1024;
  static_assert(smem <= 232448, "shared memory of one CTA");
  int rc = gdn_host::func_attr_once(chunk_attention_kernel<D, kMods>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem,
                                    done);
  if (rc != GDN_OK) return rc;
  CUtensorMap q_map, k_map, v_map;
  const int64_t dims[4] = {D, d.a.group, total_tokens, d.a.Hkv};
  const int64_t strides[3] = {2 * D, 2 * d.a.q_stride, 2 * static_cast<int64_t>(d.a.group) * D};
  if ((rc = gdn_host::encode_map_4d(&q_map, d.a.q, dims, strides, d.a.group, d.tile_tokens)) != GDN_OK) return rc;
  if ((rc = gdn_host::encode_cache_map(&k_map, cache->k, cache, d.a.box_rows)) != GDN_OK) return rc;
  if ((rc = gdn_host::encode_cache_map(&v_map, cache->v, cache, d.a.box_rows)) != GDN_OK) return rc;
  const int grid = sms < kMaxGrid ? sms : kMaxGrid;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  d.cuts = reinterpret_cast<int4*>(ws);
  d.part_ml = reinterpret_cast<float2*>(ws + kCutBytes);
  d.part_o = reinterpret_cast<float4*>(ws + kCutBytes + sizeof(float2) * 4 * kMaxGrid * kRows);
  rc = gdn_host::launch_pdl(chunk_attention_kernel<D, kMods>, dim3(grid), dim3(kThreads), smem, stream, d, q_map, k_map,
                            v_map);
  if (rc != GDN_OK) return rc;
  return gdn_host::launch_pdl(chunk_join_kernel<D>, dim3(grid, 8), dim3(256), 0, stream, d);
}

}  // namespace

extern "C" size_t gdn_attention_workspace_bytes(int32_t num_seqs, int32_t total_tokens, int32_t Hq, int32_t Hkv,
                                                int32_t D) {
  if (num_seqs < 0 || total_tokens < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
  return workspace_bytes_of(D);
}

extern "C" int gdn_attention_paged(const gdn_bf16* q, int64_t q_token_stride, gdn_bf16* o, float* lse,
                                   const int32_t* cu_seqlens, int32_t total_tokens, int32_t Hq,
                                   const gdn_kv_cache* cache, const gdn_page_table* table, float scale,
                                   const gdn_attention_options* options, void* workspace, size_t workspace_bytes,
                                   int32_t* err_word, void* stream) {
  ChunkArgs d = {};
  const size_t need = cache ? workspace_bytes_of(cache->head_dim) : 0;
  int rc = gdn_host::attention_args(&d.a, q, q_token_stride, o, lse, cu_seqlens, total_tokens, Hq, cache, table, scale,
                                    options, workspace, workspace_bytes, need, err_word, kKeys);
  if (rc != GDN_OK || table->num_seqs == 0 || total_tokens == 0) return rc;
  int sms = 0;
  rc = gdn_host::check_device(&sms);
  if (rc != GDN_OK) return rc;
  d.tile_tokens = kRows / d.a.group;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool mods = d.a.cap_log2 > 0.f || d.a.slopes;
  if (cache->head_dim == 64)
    return mods ? launch<64, true>(d, total_tokens, cache, workspace, sms, s)
                : launch<64, false>(d, total_tokens, cache, workspace, sms, s);
  return mods ? launch<128, true>(d, total_tokens, cache, workspace, sms, s)
              : launch<128, false>(d, total_tokens, cache, workspace, sms, s);
}
