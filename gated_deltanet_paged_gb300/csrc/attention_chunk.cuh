// attention_chunk.cuh -- the chunk attention kernel of both caches (attention.cu, which
// describes it, and attention8.cu), and the join of the items that its CTAs cut.
#pragma once

#include <type_traits>

#include "attention_common.cuh"
#include "cache8.cuh"

namespace {  // each kernel's file has its own

using gdn::AttnArgs;

constexpr int kRows = 128;   // rows per tile
constexpr int kKeys = 128;   // keys per block
// Warps 0-3 and 4-7: softmax of tiles 0 and 1; 8 and 9: products of tiles 0 and
// 1; 10: segments, queries and keys; 11: values; 12-15: epilogue.
constexpr int kThreads = 512;
constexpr int kMmaWarp = 8, kLoadWarp = 10, kValueWarp = 11, kEpilogueWarp = 12;
// 65,536 registers: 256 softmax threads hold 128 scores each, the others little; but
// where the cache is in 8 bits, the epilogue's warps convert it.
template <bool kCodes>
struct Registers {
  static constexpr int kSoftmax = kCodes ? 184 : 200, kIssue = 56, kEpilogue = kCodes ? 88 : 56;
  static constexpr int kSum = 128 * (2 * kSoftmax + kIssue + kEpilogue);
  static_assert(kSum == 65536, "register split of the block");
};
constexpr int kSegments = 4;  // segments announced ahead
// How the batch is shared out; times at 32 query heads on 8 key heads of 128, a
// prompt of 1,000 tokens after 2,000 written 1,000 + 2,000.
// Fixed cost of an item (queries, pipeline fill, epilogue) in keys.  With 4 blocks
// short items weigh too much (8 prompts of 1,000 to 1,300: 121 us, 111 with 2).
constexpr int kItemCost = 2 * kKeys;
// Smallest piece of the line in keys: with 2 blocks, and an item's cost of one, the
// pieces are worth less than their joins (32 x 128 after up to 800: 66 us, 59 with 4).
constexpr int kMinShare = 4 * kKeys;
// What a CTA's second segment costs, in blocks: with 3, calls of few short items are
// cut along the line (1,000 + 1,000: 40 us, 33 with 8); without a bound, 64 items
// leave 24 of 152 CTAs idle (512 + 131,072: 670 us, 610 with one).
constexpr int kCrossing = 8;
// Blocks of a piece, where items are cut evenly: 16 + 4,000 take 20.8 / 16.7 / 18.8 us
// with pieces of 1 / 2 / 5 blocks.
// (With one, a last piece could begin past the end of its item on the line, which is
// shorter than its blocks by the keys that a window hides in the first.)
constexpr int kMinBlocks = 2;
static_assert(kMinBlocks >= 2, "no piece of an evenly cut item is empty");
// Items are not cut if no sequence is longer: 1,000 tokens take 19 us, cut 28;
// 8 x (64 + 400) 16 us, cut 20.  Of 4,000 keys they are: 16 + 4,000 take 17 us,
// whole 42.
constexpr int kWholeKeys = 8 * kKeys;
constexpr int kMaxGrid = 160;         // one CTA per SM

struct ChunkArgs {
  AttnArgs a;
  int32_t tile_tokens;  // tokens per tile: 128 / group
  float4* part_o;       // [2 grid][2 tiles][D / 4][128 rows]
  float2* part_ml;      // [2 grid][2 tiles][128 rows]
  int32_t whole;        // no sequence can be longer than kWholeKeys: there is no join and no workspace
  int4* cuts;           // [grid]: (first token, tokens, key head, last CTA) of an item cut at this CTA's end, or -1
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
  q.full = d.a.full_lens ? min(d.a.full_lens[b], s.len) : 0;
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
__device__ __forceinline__ int64_t sum_max(int c, int a, int step, int n) {
  const int64_t k = c > a ? min((c - a + step - 1) / step, n) : 0;  // the first k terms are c
  const int64_t m = n;
  return c * k + a * (m - k) + step * (m * (m - 1) - k * (k - 1)) / 2;
}
// sum of pair_cost over the pairs before i (i < pairs: all of them full).
__device__ __forceinline__ int64_t cost_before(const ChunkArgs& d, const Seq& s, int i) {
  const int p = s.len - s.n, step = 2 * d.tile_tokens;
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
  int last;          // CTA that takes the end of the item; -1: as the line is shared out
  bool whole;        // items are not cut: a CTA takes those that begin in its piece
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
    const int64_t stop = w.whole ? w.item0 + w.cost : min(w.end, w.item0 + w.cost);
    w.blk0 = max(0, (static_cast<int>(w.pos - w.item0) - kItemCost) / kKeys);
    w.blk1 = stop == w.item0 + w.cost ? w.blocks : max(0, (static_cast<int>(stop - w.item0) - kItemCost) / kKeys);
    w.pos = stop;
    if (w.blk1 > w.blk0) return true;
  }
  return false;
}
template <int D, bool kCodes>
struct Layout {
  static constexpr int kHalf = kRows * 128;            // 64 dimensions of 128 rows
  static constexpr int kTile = kRows * D * 2;          // a Q, K or V tile
  // Ring of K and V tiles: with a fifth at D = 128 nothing is faster (4 x 8,192
  // tokens 1.36 ms either way, 64 x 512 228 us against 224).
  static constexpr int kStages = D == 64 ? 8 : kCodes ? 3 : 4;
  // Ring of tiles of codes behind it: as many bytes ahead as the ring has without.
  static constexpr int kCodeTile = kKeys * D;
  static constexpr int kCodeStages = !kCodes ? 0 : D == 64 ? 6 : 4;
  static constexpr int kBytes = (2 + kStages) * kTile + kCodeStages * kCodeTile;
  static constexpr uint32_t kColS = 0, kColO = 256;    // TMEM columns: S of both tiles, O of both tiles
};

// Sum over the CTA's threads before this one, and over all.  Two sums go as one:
// one of less than kFlag, and that of a flag above it.
constexpr int kFlag = 1 << 20;
static_assert(kThreads * (kMaxGrid + 1) < kFlag && kThreads < (1 << 11), "sums of both parts");
template <typename T>
__device__ __forceinline__ T scan_block(int64_t* scratch64, T mine, T* total) {
  T* const scratch = reinterpret_cast<T*>(scratch64);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  T before = incl - mine, sum = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += scratch[i];
    sum += scratch[i];
  }
  __syncthreads();
  *total = sum;
  return before;
}

// One segment of the CTA's share, as the copying warp announces it to the others.
struct alignas(16) Segment {
  int blocks;       // in this segment; 0: no more segments
  int key0;         // first key of the first block
  int lo, hi;       // keys that are copied
  int first_token;  // row of the item's first token in q and o
  int tokens;       // of the item
  int pos;          // position of its first token
  int full;         // prefix mask
  int head;
  int part;         // -1: the whole item; else its partial slot
  int entry;        // first page table entry of the sequence
  int seq;
};

template <int D, bool kCodes>
struct Smem {
  using L = Layout<D, kCodes>;
  uint64_t full[L::kStages];
  uint64_t empty[L::kStages];
  uint64_t raw[L::kStages];  // copies of values that are to be cleared before they are `full`
  uint64_t q_full, q_empty, done[2];
  uint64_t s_full[2];      // S is there, and the O of the blocks before is complete
  uint64_t p_full[2][2];   // [tile][half]: 64 keys' weights are there
  uint64_t o_last[2];      // O of a segment is complete
  uint64_t o_free[2];      // ... and has been read
  uint64_t stat_full[2];
  uint64_t mid[2];         // the first half of P V of a block is complete (kCapped)
  uint64_t turn[2];        // the other tile's products of a block have been issued
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  uint64_t never;          // the test hook's barrier, never completed
  int64_t scan[kThreads / 32];
  Walk walk;
  Segment seg[kSegments];
  float2 stat[2][kRows];  // [tile][row]: reference and sum of a segment
  uint32_t tmem;
  int abort;
  // Of an 8-bit cache: the copies of a tile of codes, and its groups' scales.
  static constexpr int kCodeStages = kCodes ? L::kCodeStages : 1;
  uint64_t code_full[kCodeStages], code_empty[kCodeStages];
  float code_scale[kCodeStages][kKeys / gdn::kGroup];
};
template <int D, bool kCodes>
constexpr int kSmemBytes = Layout<D, kCodes>::kBytes + sizeof(Smem<D, kCodes>);

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// This warp has read its part of O.
__device__ __forceinline__ void release(uint64_t* bar, int lane) {
  gdn::tc_fence_before();
  __syncwarp();
  if (lane == 0) gdn::mbar_arrive(bar);
}
// Four columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
      : "memory");
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
__device__ __forceinline__ void tmem_wait_ld32(float (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  pin32(r);
}
__device__ __forceinline__ float max128(const float (&s)[128]) {
  float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int i = 4; i < 124; i += 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) top[k] = gdn::max3(top[k], s[i + 2 * k], s[i + 2 * k + 1]);
  }
  return gdn::max3(gdn::max3(top[0], top[1], s[124]), gdn::max3(top[2], s[125], s[126]), fmaxf(top[3], s[127]));
}
// The largest of 32 values either way, and of `top`.
__device__ __forceinline__ float largest32(const float (&x)[32], float top) {
  float big[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int i = 4; i < 28; i += 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) big[k] = gdn::max3_abs(big[k], x[i + 2 * k], x[i + 2 * k + 1]);
  }
  return gdn::max3_abs(gdn::max3_abs(big[0], x[28], x[29]), gdn::max3_abs(big[1], x[30], x[31]),
                       gdn::max3_abs(big[2], big[3], top));
}
__device__ __forceinline__ float max32(const float (&x)[32]) {
  float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int i = 4; i < 28; i += 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) top[k] = gdn::max3(top[k], x[i + 2 * k], x[i + 2 * k + 1]);
  }
  return gdn::max3(gdn::max3(top[0], x[28], x[29]), gdn::max3(top[1], x[30], x[31]), fmaxf(top[2], top[3]));
}
// Of 32 capped scores whose originals are in TMEM columns from addr: those of the groups
// of four columns in which any row of the warp has a score beyond the polynomial, less
// `minus`, one group after the other.  Keys that a row does not see, and whatever stands
// in slots that no row sees, choose groups too: the scores within the polynomial have the
// bits that they had.
__device__ __forceinline__ void cap_far(const AttnArgs& a, uint32_t addr, float minus, float (&x)[32]) {
  uint32_t groups = 0;
  {
    float s[32];
    gdn::tmem_ld32(addr, s);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (!(gdn::max3_abs(gdn::max3_abs(s[4 * k], s[4 * k + 1], s[4 * k + 2]), s[4 * k + 3], 0.f) <= a.cap_near)) groups |= 1u << k;
  }
  groups = __reduce_or_sync(0xFFFFFFFFu, groups);
#pragma unroll 1
  for (; groups; groups &= groups - 1) {
    const int group = __ffs(groups) - 1;
    uint32_t z[4];
    tmem_ld4(addr + 4 * group, z);
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = __float_as_uint(gdn::capped(__uint_as_float(z[k]), a, minus));
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (group == k / 4) x[k] = __uint_as_float(z[k % 4]);
  }
}
// Cap of 32 scores in TMEM columns from addr, into units of log2.  Where the warp's
// scores stay within the cap (they mostly do), the polynomial, which is evaluated
// beside the maximum that decides it.  Else any form for the groups of four columns that
// hold a score beyond, read from TMEM once more, one group after the other: its
// instructions would stand between the others.  (For all eight groups: 64 mixed
// sequences, 16 heads, a cap of 30 and scores of up to 6 times their deviation, 4.6 ms.)
__device__ __forceinline__ void cap_scores(const AttnArgs& a, const gdn::CapPoly& poly, uint32_t addr, float (&x)[32]) {
  const float most = largest32(x, 0.f);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 y = gdn::capped_near(make_float2(x[i], x[i + 1]), poly);
    x[i] = y.x;
    x[i + 1] = y.y;
  }
  if (!__all_sync(0xFFFFFFFFu, most <= a.cap_near)) cap_far(a, addr, 0.f, x);
}
// Scores outside [from, to) are hidden.
__device__ __forceinline__ void hide(int from, int to, float as, float (&x)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = i >= from && i < to ? x[i] : as;
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

// A tile of 128 keys or values from the 8-bit cache, as the copies left it at `codes`, to
// bf16 at `tile`, in the layout that the copies of a 16-bit cache have: four warps, of
// which D / 16 lanes take a row, 16 codes each.  A value is its code times its scale,
// exactly, so that everything behind is the same.  Rows outside [from, to) become zeros.
template <int D>
__device__ __forceinline__ void convert_tile(uint32_t codes, const float* scales, uint8_t* tile, int warp, int lane, int from,
                                             int to) {
  constexpr int kLanes = D / 16, kRowsOfWarp = 32 / kLanes, kRowsOfStep = 4 * kRowsOfWarp;
  const int row = warp * kRowsOfWarp + lane / kLanes, chunk = lane % kLanes;
  // Lanes of the second 64 dimensions write their two chunks in the other order: all
  // eight of a row then meet different banks.
  const bool swap = chunk >= 4;
  uint8_t* const dst = tile + (chunk >> 2) * (kRows * 128);
  // Rolled, as little code as gives two rows in flight: the kernel's instructions are
  // fetched more slowly than issued (unrolled, 4 x 8,192 tokens take 2.3 ms, with four
  // rows in flight 2.1, with a conversion in integers, which needs a second path for
  // NaN and for large scales, 2.0 and unrolled 3.5; so 1.8).
  constexpr int kBatch = 2;
#pragma unroll 1
  for (int i0 = 0; i0 < kKeys / kRowsOfStep; i0 += kBatch) {
    uint4 x[kBatch];
    float scale[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = (i0 + i) * kRowsOfStep + row;
      x[i] = gdn::lds128(codes + gdn::chunk_at<D>(r, chunk));
      scale[i] = scales[r / gdn::kGroup];
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = (i0 + i) * kRowsOfStep + row;
      if (r < from || r >= to) x[i] = make_uint4(0, 0, 0, 0);
      if (swap) x[i] = make_uint4(x[i].z, x[i].w, x[i].x, x[i].y);
      const float2 f = make_float2(scale[i], scale[i]);
      const uint2 a0 = gdn::e4m3_to_bf16(x[i].x, f), a1 = gdn::e4m3_to_bf16(x[i].y, f);
      const uint2 b0 = gdn::e4m3_to_bf16(x[i].z, f), b1 = gdn::e4m3_to_bf16(x[i].w, f);
      const int c0 = (chunk & 3) * 2 + (swap ? 1 : 0);
      *reinterpret_cast<uint4*>(dst + gdn::swz(r, c0)) = make_uint4(a0.x, a0.y, a1.x, a1.y);
      *reinterpret_cast<uint4*>(dst + gdn::swz(r, c0 ^ 1)) = make_uint4(b0.x, b0.y, b1.x, b1.y);
    }
  }
}

// How scores become weights.
//   kPlain: scale and reference in one multiply-add.
//   kBiased: a bias that is linear in the key (no prefix mask: every visible key is
//     behind the token) first.
//   kGeneral: a bias beside a cap or a prefix mask, both first (the options that change
//     a score; those that only hide keys cost nothing away from the edges).
//   kCapped: a cap and no bias.  Small scores take the cap's polynomial straight to the
//     weights, without a maximum, 32 keys at a time.
enum Scores { kPlain, kBiased, kGeneral, kCapped };
// kCapped's reference is kAbove to begin with or kAbove over the largest score that a row
// has, and moves in the first block with a score of more than kOver over it (the cap alone
// would bound the weights too, but by 2^80 at 55, and from below by nothing: times large
// or small values they would leave fp32).  A row's first keys may also set it below
// kAbove: with one way (kOneWay) where all of them score below 0, with two where one of
// the block's scores is far from 0.  So weights stay below 2^16, and the largest of a row
// is 2^-48 at least, with one way 2^-17.  Moving is slow, and leaves the tiles out of step
// for a while: 64 mixed sequences take 1.54 ms, with no distance above the largest score
// and 16 or 24 over that 1.65 and 1.73.
constexpr float kAbove = 16.f, kOver = 16.f;

// kCodes: the cache is in 8 bits, and `codes` says where its scales are.  kOneWay: scores
// under a cap take one way, large or not (attention.cu's results keep their bits by two).
template <int D, Scores kScores, bool kCodes, bool kOneWay>
__device__ __forceinline__ void chunk_attention(const ChunkArgs& d, const CUtensorMap& q_map, const CUtensorMap& k_map,
                                                const CUtensorMap& v_map, const gdn::Cache8& codes) {
  using L = Layout<D, kCodes>;
  using R = Registers<kCodes>;
  // Dynamic shared memory starts behind the 1 KB that the system keeps, on a
  // 1,024-byte boundary as the swizzle needs; there is no room to round up.
  extern __shared__ __align__(1024) uint8_t tiles[];
  uint8_t* const code_ring = tiles + (2 + L::kStages) * L::kTile;
  Smem<D, kCodes>& sh = *reinterpret_cast<Smem<D, kCodes>*>(tiles + L::kBytes);
  uint8_t* ring = tiles + 2 * L::kTile;
  const AttnArgs& a = d.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // uniform, so that the roles' addresses are
  volatile int* const abort_flag = &sh.abort;

  if ((gdn::smem_u32(tiles) & 1023u) != 0) {
    if (tid == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_TIMEOUT, 0);
    return;
  }
  // Forty barriers, by several warps.
  if (tid < L::kStages) {
    gdn::mbar_init(&sh.full[tid], kCodes ? 4 : 1);
    gdn::mbar_init(&sh.empty[tid], 2);
    gdn::mbar_init(&sh.raw[tid], 1);
    gdn::fence_mbar_init();
  } else if (tid >= 32 && tid < 34) {
    const int t = tid - 32;
    gdn::mbar_init(&sh.done[t], 1);
    gdn::mbar_init(&sh.s_full[t], 1);
    gdn::mbar_init(&sh.p_full[t][0], 4);
    gdn::mbar_init(&sh.p_full[t][1], 4);
    gdn::mbar_init(&sh.o_last[t], 1);
    gdn::mbar_init(&sh.o_free[t], 4);
    gdn::mbar_init(&sh.stat_full[t], 4);
    gdn::mbar_init(&sh.turn[t], 1);
    gdn::mbar_init(&sh.mid[t], 1);
    gdn::fence_mbar_init();
  } else if (tid >= 64 && tid < 64 + kSegments) {
    gdn::mbar_init(&sh.seg_full[tid - 64], 1);
    gdn::mbar_init(&sh.seg_empty[tid - 64], kThreads / 32 - 1);
    gdn::fence_mbar_init();
  } else if (kCodes && tid >= 128 && tid < 128 + sh.kCodeStages) {
    gdn::mbar_init(&sh.code_full[tid - 128], 1);
    gdn::mbar_init(&sh.code_empty[tid - 128], 4);
    gdn::fence_mbar_init();
  } else if (tid == 96) {
    gdn::mbar_init(&sh.q_full, 1);
    gdn::mbar_init(&sh.q_empty, 2);
    gdn::mbar_init(&sh.never, 1);
    sh.abort = 0;
    gdn::fence_mbar_init();
  }
  // Rows past the group's share of a tile are never copied; they start at zero.
  if (a.group * d.tile_tokens < kRows)
    for (int i = tid; i < 2 * L::kTile / 16; i += kThreads) reinterpret_cast<uint4*>(tiles)[i] = make_uint4(0, 0, 0, 0);
  if (tid == kLoadWarp * 32) {
    gdn::prefetch_tensormap(&q_map);
    gdn::prefetch_tensormap(&k_map);
    gdn::prefetch_tensormap(&v_map);
  }
  if (warp == kMmaWarp) {
    gdn::tmem_alloc(&sh.tmem, 512);
    gdn::tmem_relinquish();
  }
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();

  // ---- this CTA's share ----
  gdn::Shares<7> shares(0, 1, 1);
  bool idle = true;
  {
    const int c = blockIdx.x, grid = gridDim.x;
    const int per = (a.paged.num_seqs + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.paged.num_seqs), b1 = min(b0 + per, a.paged.num_seqs);
    Seq s = {};
    int pairs = 0;
    bool is_long = false;
    for (int b = b0; b < b1; ++b) {
      s = load_seq(d, b);
      if (s.refused && c == 0) gdn::record_error(a.paged.err_word, GDN_DEVERR_PAGE_TABLE, b);
      pairs = min(pairs + s.pairs, kMaxGrid + 1);  // no more are told apart
      is_long = is_long || (s.pairs && s.len > kWholeKeys);
    }
    // Pairs, and in the upper bits threads with a long sequence.
    int all;
    const int pairs_before = scan_block(sh.scan, pairs + (is_long ? kFlag : 0), &all) % kFlag;
    const bool whole = d.whole || all < kFlag;
    const int64_t all_items = static_cast<int64_t>(all % kFlag) * a.Hkv;
    bool aligned = all_items <= min(grid, kMaxGrid);
    if (aligned && whole) {
      // A CTA for every item.
      idle = c >= all_items;
      const int pair = c / a.Hkv - pairs_before;
      if (!idle && pair >= 0 && pair < pairs) {
        Walk x = {};
        x.b = b0;
        x.s = s;  // one sequence per thread, unless there are more than threads
        x.pair = pair;
        for (; per > 1; x.pair -= x.s.pairs, ++x.b) {
          x.s = load_seq(d, x.b);
          if (x.pair < x.s.pairs) break;
        }
        x.head = c % a.Hkv;
        x.cost = pair_cost(d, x.s, x.pair);
        x.end = x.cost;
        sh.walk = x;
      }
    } else if (aligned) {
      // Few items: each gets CTAs to itself, by its length, and they cut it evenly.
      // Cutting the line instead gives many a CTA the end of one item and the start
      // of the next, and an item's fixed cost twice (452 tokens over 2,500: the
      // CTAs end between 10.6 and 17 us, aligned between 10 and 12).
      int2* table = reinterpret_cast<int2*>(tiles + 2 * L::kTile);  // pairs; the ring is not in use yet
      int at = pairs_before;
      for (int b = b0; b < b1; ++b) {
        if (per > 1) s = load_seq(d, b);
        for (int i = 0; i < s.pairs; ++i) table[at++] = make_int2(b, i);
      }
      __syncthreads();
      Walk x = {};
      int blocks = 0;
      const int items = static_cast<int>(all_items);
      if (tid < items) {
        const int2 pair = table[tid / a.Hkv];
        x.b = pair.x, x.pair = pair.y, x.head = tid % a.Hkv;
        x.s = load_seq(d, x.b);
        x.cost = pair_cost(d, x.s, x.pair);
        blocks = (pair_hi(d, x.s, x.pair) + kKeys - 1) / kKeys - pair_lo(d, x.s, x.pair) / kKeys;
      }
      int sum, pieces_total;
      scan_block(sh.scan, x.cost / kKeys, &sum);
      int pieces = tid < items ? 1 : 0;
      if (tid < items) {
        pieces += static_cast<int>(__fdividef(static_cast<float>(grid - items) * static_cast<float>(x.cost / kKeys),
                                              static_cast<float>(sum)));
        pieces = min(pieces, max(1, blocks / kMinBlocks));
      }
      // Unless a piece is longer than a share of the line and the cost of a second
      // segment (512 tokens over 131,072 are 64 items: 128 of 152 CTAs would work).
      const bool longer = pieces && x.cost / pieces > (sum / grid + kCrossing) * kKeys;
      const int piece = c - scan_block(sh.scan, pieces + (longer ? kFlag : 0), &pieces_total) % kFlag;
      aligned = pieces_total < kFlag;
      idle = c >= pieces_total;
      if (aligned && piece >= 0 && piece < pieces) {
        // As a walk along a line on which the item begins at 0.
        const int blk0 = blocks * piece / pieces, blk1 = blocks * (piece + 1) / pieces;
        x.pos = blk0 ? kItemCost + static_cast<int64_t>(blk0) * kKeys : 0;
        x.end = blk1 < blocks ? kItemCost + static_cast<int64_t>(blk1) * kKeys : x.cost;
        x.last = c - piece + pieces - 1;
        sh.walk = x;
      }
    }
    if (!aligned) {
      int64_t cost = 0, mine = 0, total;
      for (int b = b0; b < b1; ++b) {
        if (per > 1) s = load_seq(d, b);
        cost = seq_cost(d, s);
        mine += cost;
      }
      const int64_t before = scan_block(sh.scan, mine, &total);
      total *= a.Hkv;
      // Whole items need no smallest piece: every one can have a CTA to itself.
      shares = gdn::Shares<7>(total, total / (whole ? kItemCost : kMinShare), grid);
      const int64_t start = shares.start(c), end = shares.start(c + 1);
      idle = start >= end;
      // The thread whose sequences hold `start` sets up the walk.
      if (!idle && before * a.Hkv <= start && start < (before + mine) * a.Hkv) {
        Walk x;
        x.pos = start;
        x.end = end;
        x.last = -1;
        x.b = b0;
        int64_t base = before * a.Hkv;
        x.s = s;  // one sequence per thread, unless there are more than threads
        for (; per > 1; ++x.b) {
          x.s = load_seq(d, x.b);
          cost = seq_cost(d, x.s);
          if (start < base + cost * a.Hkv) break;
          base += cost * a.Hkv;
        }
        int i = 0;  // the last pair that begins at or before start
        for (int step = x.s.pairs > 1 ? 1 << (31 - __clz(x.s.pairs - 1)) : 0; step; step >>= 1)
          if (step < x.s.pairs - i && cost_before(d, x.s, i + step) * a.Hkv <= start - base) i += step;
        x.pair = i;
        x.cost = pair_cost(d, x.s, i);
        base += cost_before(d, x.s, i) * a.Hkv;
        x.head = gdn::small_quotient(start - base, x.cost, a.Hkv);
        x.item0 = base + static_cast<int64_t>(x.head) * x.cost;
        x.whole = whole;
        if (whole && start > x.item0) x.pos = x.item0 + x.cost;
        sh.walk = x;
      }
    }
    if (tid == 0 && !d.whole) d.cuts[c] = make_int4(-1, 0, 0, 0);
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
    // Behind its own branch, so that its warps alone have the epilogue's registers.
    const bool epilogue_regs = kCodes && warp >= kEpilogueWarp;
    if (!epilogue_regs) regs_dec<R::kIssue>();
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = ok && gdn::warp_wait(bar, parity, abort_flag, a.wait_ns); };
    // What has to end before the CTA does, whatever the others do.
    auto last = [&](uint64_t* bar, uint32_t parity) { return gdn::warp_wait(bar, parity, nullptr, 2000000000u); };
    // Segment i as announced; false when there is none or a wait ran out.
    auto next = [&](uint32_t i, Segment& g) {
      if (!wait(&sh.seg_full[i % kSegments], (i / kSegments) & 1)) return false;
      g = sh.seg[i % kSegments];
      __syncwarp();
      if (lane == 0) gdn::mbar_arrive(&sh.seg_empty[i % kSegments]);
      return g.blocks > 0;
    };
    // Copies in flight, and their barriers.
    constexpr uint32_t kCopies = kCodes ? sh.kCodeStages : L::kStages;
    uint64_t* const copied = kCodes ? sh.code_full : sh.full;
    // Tile n of codes with its scales; false: a wait ran out.
    auto send_codes = [&](auto& tile, auto& scale, uint32_t n, bool more) {
      const uint32_t at = n % kCopies;
      if (n >= kCopies && !wait(&sh.code_empty[at], ((n / kCopies) - 1) & 1)) return false;
      if (lane < kKeys / gdn::kGroup) sh.code_scale[at][lane] = gdn::scale_of(scale.byte);
      __syncwarp();
      if (lane == 0) gdn::mbar_arrive_expect_tx(&sh.code_full[at], tile.bytes());
      __syncwarp();
      tile.copy(code_ring + at * L::kCodeTile, &sh.code_full[at], more);
      scale.next(more);
      return true;
    };
    auto epilogue = [&] {
      // ----------------------------------------------------------- epilogue
      // Reads a segment's O while the softmax warps are on the next one.
      const int row = (warp & 3) * 32 + lane;
      const uint32_t o_addr = tmem + L::kColO + (static_cast<uint32_t>(warp & 3) << 21);  // TMEM lane 32 (warp % 4)
      const int my_token = row / a.group, my_head = row % a.group;
      const bool aligned32 = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
      uint32_t taken[2] = {0, 0};  // segments of each tile
      // Writes the results of a segment, or its part of them.
      auto write = [&](const Segment& g) {
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          if (t * tile_tokens >= g.tokens) continue;
          if (!wait(&sh.stat_full[t], taken[t] & 1) || !wait(&sh.o_last[t], taken[t] & 1)) break;
          gdn::tc_fence_after();
          const float2 ml = sh.stat[t][row];
          ++taken[t];
          const uint32_t o = o_addr + t * D;
          const int token = t * tile_tokens + my_token;
          const bool valid = my_token < tile_tokens && token < g.tokens;
          if (g.part < 0) {
            const float inv = 1.f / ml.y;
            const int64_t out = (static_cast<int64_t>(g.first_token) + token) * a.Hq + g.head * a.group + my_head;
            __nv_bfloat16* dst = a.o + out * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float x[32];
              gdn::tmem_ld32(o + c, x);
              if (c + 32 == D) release(&sh.o_free[t], lane);
              if (valid) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  uint32_t y[8];
#pragma unroll
                  for (int e = 0; e < 8; ++e) y[e] = gdn::pack_bf162(x[16 * i + 2 * e] * inv, x[16 * i + 2 * e + 1] * inv);
                  gdn::store32(dst + c + 16 * i, y, aligned32);
                }
              }
            }
            if (valid && a.lse) a.lse[out] = (ml.x + log2f(ml.y)) / gdn::kLog2e;
          } else {
            const int64_t slot = 2 * static_cast<int64_t>(g.part) + t;
            float4* dst = d.part_o + slot * (D / 4) * kRows + row;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float x[32];
              gdn::tmem_ld32(o + c, x);
              if (c + 32 == D) release(&sh.o_free[t], lane);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[(c / 4 + i) * kRows] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            }
            d.part_ml[slot * kRows + row] = ml;
          }
        }
      };
      Segment g;
      if constexpr (!kCodes) {
        for (uint32_t segs = 0; ok && next(segs, g); ++segs) write(g);
      } else {
        // These warps convert keys and values as well, and a segment's results are written
        // between the tiles of the next as soon as they are there.
        Segment done;
        bool pending = false;
        uint32_t n = 0;  // ring tiles
        for (uint32_t segs = 0;; ++segs) {
          const bool more = next(segs, g);
          const int count = more ? 2 * g.blocks : 0;
          for (int i = 0; ok; ++i) {
            if (pending) {
              // At the latest where the next tile's room depends on it.
              bool there = i >= count || i >= L::kStages;
              if (!there) {
                there = gdn::mbar_test(&sh.stat_full[0], taken[0] & 1) && gdn::mbar_test(&sh.o_last[0], taken[0] & 1);
                if (tile_tokens < done.tokens)
                  there = there && gdn::mbar_test(&sh.stat_full[1], taken[1] & 1) && gdn::mbar_test(&sh.o_last[1], taken[1] & 1);
                there = __all_sync(0xFFFFFFFFu, there);
              }
              if (there) {
                write(done);  // the one place: the kernel's code is fetched more slowly than issued
                pending = false;
              }
            }
            if (!ok || i >= count) break;
            const uint32_t stage = n % L::kStages, at = n % kCopies;
            const int key0 = g.key0 + (i >> 1) * kKeys;
            if (!wait(&sh.code_full[at], (n / kCopies) & 1)) break;
            if (n >= L::kStages && !wait(&sh.empty[stage], ((n / L::kStages) - 1) & 1)) break;
            convert_tile<D>(gdn::smem_u32(code_ring + at * L::kCodeTile), sh.code_scale[at], ring + stage * L::kTile, warp & 3,
                            lane, g.lo - key0, g.hi - key0);
            gdn::fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              gdn::mbar_arrive(&sh.full[stage]);
              gdn::mbar_arrive(&sh.code_empty[at]);
            }
            ++n;
          }
          if (!ok || !more) break;
          done = g;
          pending = true;
        }
      }
      if (!ok) *abort_flag = 1;
    };
    if (epilogue_regs) {
      regs_dec<R::kEpilogue>();
      epilogue();
    } else if (warp == kLoadWarp) {
      // ------------------------------------ segments, queries and keys
      Walk w = sh.walk;
      gdn::TileCopies<D, kKeys, kCodes ? 1 : 2> keys(a, &k_map, lane);
      gdn::ScaleCopies<kKeys> key_scales(a, codes, 0, lane);
      uint32_t n = 0, segs = 0;  // ring tiles (keys are the even ones), segments announced
      uint32_t queries = 0;      // sent
      for (;; ++segs) {
        const bool more = next_segment(d, w);
        if (segs >= kSegments && !wait(&sh.seg_empty[segs % kSegments], ((segs / kSegments) - 1) & 1)) break;
        Segment g = {};
        if (more) {
          const bool starts = w.blk0 == 0, ends = w.blk1 == w.blocks;
          const int pair0 = w.pair * 2 * tile_tokens;  // first token of the item within the sequence's new ones
          g.blocks = w.blk1 - w.blk0;
          g.key0 = (w.first + w.blk0) * kKeys;
          g.lo = w.lo;
          // To the end of the last block, as far as the sequence goes: those tokens'
          // weights are 0 and their values finite, so that only blocks which a
          // sequence ends in, or a window begins in, have values to clear.
          g.hi = min(w.s.len, (w.hi + kKeys - 1) / kKeys * kKeys);
          g.first_token = w.s.first_token + pair0;
          g.tokens = min(2 * tile_tokens, w.s.n - pair0);
          g.pos = w.s.len - w.s.n + pair0;
          g.full = w.s.full;
          g.head = w.head;
          // One segment of a CTA at most starts an item that it does not end, and
          // one at most continues one: two partial slots per CTA.
          g.part = starts && ends ? -1 : 2 * static_cast<int>(blockIdx.x) + (starts ? 1 : 0);
          g.entry = w.s.entry;
          g.seq = w.b;
          if (lane == 0 && starts && !ends)
            d.cuts[blockIdx.x] = make_int4(g.first_token, g.tokens, g.head, w.last >= 0 ? w.last : shares.owner(w.item0 + w.cost - 1));
        }
        if (lane == 0) {
          sh.seg[segs % kSegments] = g;
          gdn::mbar_arrive(&sh.seg_full[segs % kSegments]);
        }
        __syncwarp();
        if (!more) break;
        keys.begin(g.lo, g.hi, g.head, g.seq, g.entry, g.key0);
        if constexpr (kCodes) key_scales.begin(g.lo, g.hi, g.head, g.entry, g.key0);
        // The queries go first where their room is free; else behind the first
        // block's keys, which need none that the segment before holds.
        auto send_queries = [&](bool must) {
          if (segs > 0) {
            const uint32_t parity = (segs - 1) & 1;
            if (must) {
              if (!wait(&sh.q_empty, parity)) return false;
            } else if (!__all_sync(0xFFFFFFFFu, gdn::mbar_test(&sh.q_empty, parity))) {
              return false;
            }
          }
          if (lane == 0) {
            const int bytes = a.group * tile_tokens * D * 2, tiles_used = g.tokens > tile_tokens ? 2 : 1;
            gdn::mbar_arrive_expect_tx(&sh.q_full, tiles_used * bytes);
            for (int t = 0; t < tiles_used; ++t)
              for (int c = 0; c < D / 64; ++c)
                gdn::tma_load_4d(tiles + t * L::kTile + c * L::kHalf, &q_map, &sh.q_full, c * 64, 0,
                                 g.first_token + t * tile_tokens, g.head);
          }
          __syncwarp();
          ++queries;
          return true;
        };
        bool q_sent = send_queries(false);
        for (int j = 0; j < g.blocks; ++j) {
          if constexpr (kCodes) {
            if (!send_codes(keys, key_scales, n, j + 1 < g.blocks)) break;
          } else {
            const uint32_t stage = n % L::kStages;
            if (n >= L::kStages && !wait(&sh.empty[stage], ((n / L::kStages) - 1) & 1)) break;
            if (lane == 0) gdn::mbar_arrive_expect_tx(&sh.full[stage], keys.bytes());
            __syncwarp();
            keys.copy(ring + stage * L::kTile, &sh.full[stage], j + 1 < g.blocks);
          }
          n += 2;
          if (!q_sent && !(q_sent = send_queries(true))) break;
        }
        if (!ok) break;
      }
      if (!ok) *abort_flag = 1;
      // Leave no copy in flight behind, whoever gave up (bounded waits, as everywhere).
      ok = !queries || last(&sh.q_full, (queries - 1) & 1);
#pragma unroll 1
      for (uint32_t i = n > kCopies ? n - kCopies : 0; i < n; i += 2) ok = last(&copied[i % kCopies], (i / kCopies) & 1) && ok;
      if (!ok) *abort_flag = 1;
    } else if (warp < kLoadWarp) {
      // ----------------------------------------------------------- products
      // One warp per tile, of which one elected lane does it all: there is no other
      // to disagree with when a wait runs out.  (Lane 0 instead of an elected one: 4 x
      // 8,192 tokens 1.60 ms instead of 1.32.  All lanes with a vote at each wait:
      // 1.36.)  Its products run in the order of their issue, so S of the next block
      // may overwrite the weights that P V before it reads.
      const int t = warp - kMmaWarp;
      const uint32_t id_s = gdn::idesc_f16(kRows, kKeys, true, true, false, false);
      const uint32_t id_o = gdn::idesc_f16(kRows, D, true, true, false, true);
      const uint64_t q_desc = gdn::sdesc(gdn::smem_u32(tiles) + t * L::kTile, 16, 1024);
      const uint64_t k_desc = gdn::sdesc(gdn::smem_u32(ring), 16, 1024);
      const uint64_t v_desc = gdn::sdesc(gdn::smem_u32(ring), L::kHalf, 1024);
      const uint32_t s_col = tmem + L::kColS + t * kKeys, o_col = tmem + L::kColO + t * D;
      constexpr uint32_t kStep = L::kTile >> 4;  // a stage, in descriptor units
      uint32_t np = 0, done_segs = 0, turns = 0;  // blocks and segments of this tile, blocks of both
      uint32_t stage = 0, phase = 0;
      auto advance = [&] {
        if (++stage == L::kStages) stage = 0, phase ^= 1;
      };
      // S = Q K^T of the ring's current tile, which is released with it.
      auto scores = [&](bool last) {
        gdn::tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          gdn::tc_mma4(s_col, q_desc + c * (L::kHalf >> 4), 2, k_desc + stage * kStep + c * (L::kHalf >> 4), 2, id_s, c);
        gdn::tc_commit(&sh.s_full[t]);
        gdn::tc_commit(&sh.empty[stage]);
        if (last) gdn::tc_commit(&sh.q_empty);
        advance();
      };
      if (gdn::elect_one()) {
        auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = ok && gdn::lane_wait(bar, parity, abort_flag, a.wait_ns); };
        for (uint32_t segs = 0;; ++segs) {
          if (!wait(&sh.seg_full[segs % kSegments], (segs / kSegments) & 1)) break;
          const Segment g = sh.seg[segs % kSegments];
          gdn::mbar_arrive(&sh.seg_empty[segs % kSegments]);
          if (g.blocks <= 0) break;
          const bool active = t * tile_tokens < g.tokens, two = tile_tokens < g.tokens;
          if (!wait(&sh.q_full, segs & 1)) break;
          if (!active) {
            // Keep in step: release every tile of the segment unread.
            gdn::mbar_arrive(&sh.q_empty);
            for (int i = 0; ok && i < 2 * g.blocks; ++i) {
              if (!wait(&sh.full[stage], phase)) break;
              gdn::mbar_arrive(&sh.empty[stage]);
              advance();
            }
            continue;
          }
          if (!wait(&sh.full[stage], phase)) break;
          scores(g.blocks == 1);
          for (int j = 0; ok && j < g.blocks; ++j) {
            const uint32_t v_stage = stage;
            if (!wait(&sh.full[stage], phase)) break;
            advance();
            if (j == 0 && done_segs > 0 && !wait(&sh.o_free[t], (done_segs - 1) & 1)) break;
            if (!wait(&sh.p_full[t][0], np & 1)) break;
            gdn::tc_fence_after();
            gdn::tc_mma4_ts(o_col, s_col, 8, v_desc + v_stage * kStep, 128, id_o, j > 0);
            if (kScores == kCapped) gdn::tc_commit(&sh.mid[t]);
            if (!wait(&sh.p_full[t][1], np & 1)) break;
            // The tiles take turns with the rest of P V and the next S.  Interleaved,
            // both would end together, and both softmaxes would then run beside an
            // idle tensor core (measured: two stable rhythms, 3,450 cycles per block
            // that way and 2,600 when the tiles are half a period apart).
            if (two && (t == 1 || turns > 0) && !wait(&sh.turn[t], (t == 1 ? turns : turns - 1) & 1)) break;
            gdn::tc_fence_after();
            gdn::tc_mma4_ts(o_col, s_col + 32, 8, v_desc + v_stage * kStep + 4 * 128, 128, id_o, 1);
            if (j + 1 == g.blocks) gdn::tc_commit(&sh.o_last[t]);
            gdn::tc_commit(&sh.empty[v_stage]);
            ++np;
            if (j + 1 < g.blocks) {
              if (!wait(&sh.full[stage], phase)) break;
              scores(j + 2 == g.blocks);
            }
            if (two) {
              gdn::mbar_arrive(&sh.turn[t ^ 1]);
              ++turns;
            }
          }
          ++done_segs;
        }
        if (!ok) *abort_flag = 1;
        // Every product is complete before TMEM is given back.
        gdn::tc_commit(&sh.done[t]);
      }
      __syncwarp();
      if (!last(&sh.done[t], 0)) *abort_flag = 1;
    } else if (kCodes && warp == kValueWarp) {
      // ---------------------------------------------------- codes of values
      gdn::TileCopies<D, kKeys, 1> values(a, &v_map, lane);
      gdn::ScaleCopies<kKeys> scales(a, codes, 1, lane);
      uint32_t n = 1;
      Segment g;
      for (uint32_t segs = 0; ok && next(segs, g); ++segs) {
        values.begin(g.lo, g.hi, g.head, g.seq, g.entry, g.key0);
        scales.begin(g.lo, g.hi, g.head, g.entry, g.key0);
        for (int j = 0; j < g.blocks && send_codes(values, scales, n, j + 1 < g.blocks); ++j) n += 2;
      }
      if (!ok) *abort_flag = 1;
      ok = true;
#pragma unroll 1
      for (uint32_t i = n > kCopies ? n - kCopies : 1; i < n; i += 2) ok = last(&copied[i % kCopies], (i / kCopies) & 1) && ok;
      if (!ok) *abort_flag = 1;
    } else if (warp == kValueWarp) {
      // ------------------------------------------------------------- values
      // Slots past the sequence's end or before every window may hold anything,
      // and 0 * NaN would reach the sum: their value rows become zeros in shared
      // memory.  The tile's copies complete on `raw`, and this warp completes `full`.
      gdn::TileCopies<D, kKeys> values(a, &v_map, lane);
      uint32_t n = 1, raw_parity = 0;  // ring tiles (values are the odd ones); per stage, parity of its next raw copy
      int uncleared = -1;              // stage of a raw copy that was not waited for to the end
      Segment g;
      for (uint32_t segs = 0; ok && next(segs, g); ++segs) {
        values.begin(g.lo, g.hi, g.head, g.seq, g.entry, g.key0);
        for (int j = 0; j < g.blocks; ++j, n += 2) {
          const uint32_t stage = n % L::kStages;
          const int key0 = g.key0 + j * kKeys;
          const bool partial = key0 < g.lo || key0 + kKeys > g.hi;
          uint64_t* bar = partial ? &sh.raw[stage] : &sh.full[stage];
          if (n >= L::kStages && !wait(&sh.empty[stage], ((n / L::kStages) - 1) & 1)) break;
          if (lane == 0) gdn::mbar_arrive_expect_tx(bar, values.bytes());
          __syncwarp();
          values.copy(ring + stage * L::kTile, bar, j + 1 < g.blocks);
          if (!partial) continue;
          if (!wait(bar, (raw_parity >> stage) & 1)) {
            uncleared = static_cast<int>(stage);
            break;
          }
          raw_parity ^= 1u << stage;
          const int from = max(0, g.lo - key0), to = min(kKeys, g.hi - key0);
          uint4* dst = reinterpret_cast<uint4*>(ring + stage * L::kTile);
          for (int i = lane; i < (from + kKeys - to) * 8; i += 32) {
            const int r = i >> 3, row = r < from ? r : r - from + to;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) dst[(c * kRows + row) * 8 + (i & 7)] = make_uint4(0, 0, 0, 0);
          }
          gdn::fence_proxy_async();
          __syncwarp();
          if (lane == 0) gdn::mbar_arrive(&sh.full[stage]);
        }
      }
      if (!ok) *abort_flag = 1;
      ok = uncleared < 0 || last(&sh.raw[uncleared], (raw_parity >> uncleared) & 1);
#pragma unroll 1
      for (uint32_t i = n > L::kStages ? n - L::kStages : 1; i < n; i += 2)
        ok = last(&sh.full[i % L::kStages], (i / L::kStages) & 1) && ok;
      if (!ok) *abort_flag = 1;
    } else if constexpr (!kCodes) {
      epilogue();
    }
  } else {
    // --------------------------------------------------------------- softmax
    regs_inc<R::kSoftmax>();
    const int t = warp >> 2;  // tile
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 (warp % 4)
    const uint32_t s_addr = tmem + L::kColS + t * kKeys + lane_bits, o_addr = tmem + L::kColO + t * D + lane_bits;
    const int my_token = row / a.group, my_head = row % a.group;
    uint32_t n = 0, taken = 0;  // blocks, segments of this tile
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = gdn::warp_wait(bar, parity, abort_flag, a.wait_ns); };
    for (uint32_t segs = 0;; ++segs) {
      const int at = segs % kSegments;
      if (!wait(&sh.seg_full[at], (segs / kSegments) & 1)) break;
      const Segment& g = sh.seg[at];
      const int blocks = g.blocks, seg_key0 = g.key0, tokens = g.tokens, seg_lo = g.lo, seg_hi = g.hi;
      // Rows without a token copy the range of the tile's last one.
      const int pos = g.pos + min(t * tile_tokens + min(my_token, tile_tokens - 1), tokens - 1);
      const int lo = gdn::key_lo(a, pos), hi = max(pos + 1, g.full);
      float slope = 0.f;
      if ((kScores == kGeneral || kScores == kBiased) && a.slopes) slope = a.slopes[g.head * a.group + my_head] * gdn::kLog2e;
      __syncwarp();
      if (lane == 0) gdn::mbar_arrive(&sh.seg_empty[at]);
      if (blocks == 0) break;
      if (t * tile_tokens >= tokens) continue;
      if (a.debug_stall && !wait(&sh.never, 0)) break;
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      const gdn::CapPoly poly(a);
      const float inv_scale = 1.f / a.scale_log2;
      for (int j = 0; j < blocks; ++j, ++n) {
        const int key0 = seg_key0 + j * kKeys;
        ok = __all_sync(0xFFFFFFFFu, gdn::lane_wait(&sh.s_full[t], n & 1, abort_flag, a.wait_ns));
        if (!ok) break;
        gdn::tc_fence_after();
        const bool edge = __any_sync(0xFFFFFFFFu, key0 < lo || key0 + kKeys > hi);
        // Plain and biased scores stay in registers from the maximum to the weights, all 128.
        // The others go through loops of 32, read from TMEM again where needed:
        // unrolled, their instructions were fetched more slowly than issued (ncu: 1.5
        // warps per issue waited for one, against 0.4 on the plain path; rolling
        // took the 64 mixed sequences, under a cap on the general path, from 2.13 to 1.73
        // ms, but would take 4 x 8,192 plain tokens from 1.39 to 1.48).
        constexpr bool kInRegisters = kScores == kPlain || kScores == kBiased;
        float s[kInRegisters ? 128 : 1];
        const float first_bias = slope * static_cast<float>(key0 - pos);  // kBiased: of the block's first key
        if constexpr (kInRegisters) {
          tmem_ld128(s_addr, s);
          if constexpr (kScores == kBiased) {
            // The bias of key i of the block less that of its first, from two products of
            // the slope and a whole number, each rounded once (a running sum would add a
            // rounding for every two keys, each of the bias's own size where the first
            // key's is not taken out).
            const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
            float per_key = slope;
            asm volatile("" : "+f"(per_key));  // not computed ahead of the blocks: there are no registers for it
            float2 within8[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) within8[i] = make_float2(per_key * (2 * i), per_key * (2 * i + 1));
#pragma unroll
            for (int c = 0; c < 128; c += 8) {
              const float2 eights = make_float2(per_key * c, per_key * c);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int k = c + 2 * i;
                const float2 x = __ffma2_rn(make_float2(s[k], s[k + 1]), scale2, __fadd2_rn(eights, within8[i]));
                s[k] = x.x;
                s[k + 1] = x.y;
              }
            }
          }
          if (edge) {
#pragma unroll
            for (int i = 0; i < 128; ++i) s[i] = i >= lo - key0 && i < hi - key0 ? s[i] : -INFINITY;
          }
        }
        auto publish = [&](int h) {
          gdn::tmem_wait_st();
          gdn::tc_fence_before();
          __syncwarp();
          if (lane == 0) gdn::mbar_arrive(&sh.p_full[t][h]);
        };
        // The reference moves from m (-inf: none yet) to `to`; with O already there
        // (`summed`) to what it holds.
        auto move = [&](float to, bool summed) -> float {
          const float r = m == -INFINITY ? 0.f : gdn::exp2_approx(m - to);
          m = to;
          l2 = __fmul2_rn(l2, make_float2(r, r));
#pragma unroll 1
          for (int c = 0; c < D && summed; c += 16) {
            float x[16];
            gdn::tmem_ld16(o_addr + c, x);
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(x[i] * r);
            gdn::tmem_st16(o_addr + c, y);
          }
          return r;
        };
        if constexpr (kScores == kCapped) {
          auto weights = [&](const float (&z)[32], int c) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 w = make_float2(gdn::exp2_approx(z[i]), gdn::exp2_approx(z[i + 1]));
              l2 = __fadd2_rn(l2, w);
              p[i / 2] = gdn::pack_bf162(w);
            }
            gdn::tmem_st16_nw(s_addr + c / 2, p);
          };
          if constexpr (kOneWay) {
            // 32 keys at a time and one way for all of them: two copies of it, with the next
            // 32 scores on their way meanwhile, are fetched more slowly than they save,
            // and a rare way of its own for large scores costs thousands of cycles to fetch.
#pragma unroll 1
            for (int c = 0; c < kKeys; c += 32) {
              float z[32];
              gdn::tmem_ld32(s_addr + c, z);
              if (edge) hide(lo - key0 - c, hi - key0 - c, 0.f, z);  // slots may hold anything
              const float most = largest32(z, 0.f);
              const bool unset = m == -INFINITY;  // the row has seen no key yet
              const float ref = unset ? kAbove : m;
              const float2 minus = make_float2(-ref, -ref);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 u = gdn::capped_near(make_float2(z[i], z[i + 1]), poly, minus);
                z[i] = u.x, z[i + 1] = u.y;
              }
              if (!__all_sync(0xFFFFFFFFu, most <= a.cap_near)) cap_far(a, s_addr + c, ref, z);
              if (edge) hide(lo - key0 - c, hi - key0 - c, -INFINITY, z);
              // The first keys that a row sees set its reference, downwards too: later ones
              // only raise it.  Such a row has nothing in O or l that would have to follow.
              if (__any_sync(0xFFFFFFFFu, unset || fminf(most * a.scale_log2, a.cap_log2) > ref + kOver)) {
                const bool first = unset && lo < key0 + c + 32 && hi > key0 + c;
                const float top = max32(z);  // over the reference
                const bool moves = top > kOver || (first && top < -kAbove);
                const float to = moves ? ceilf(top + ref) + kAbove : ref;
                if (__any_sync(0xFFFFFFFFu, moves && !first)) {
                  // O is complete up to this half: S came behind the blocks before, and the
                  // first half's product is waited for.
                  if (c >= 64 && !wait(&sh.mid[t], n & 1)) break;
                  gdn::tc_fence_after();
                  const bool none = unset && !first;
                  const float r = move(to, j > 0 || c >= 64);
                  if (none) m = -INFINITY;
                  if (c & 32) {
                    // The half's first 32 weights have been written.
                    float w[16];
                    uint32_t v[16];
                    gdn::tmem_wait_st();
                    gdn::tmem_ld16(s_addr + c / 2 - 16, w);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                      const float2 f = gdn::unpack_bf162(__float_as_uint(w[i]));
                      v[i] = gdn::pack_bf162(f.x * r, f.y * r);
                    }
                    gdn::tmem_st16(s_addr + c / 2 - 16, v);
                  }
                } else if (first) {
                  m = to;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] += ref - to;
              }
              weights(z, c);
              if (c & 32) publish(c > 64);
            }
          } else {
            // 32 keys at a time, the next 32 scores on their way meanwhile.
            float x[32], y[32];
            const float ref = m == -INFINITY ? kAbove : m;
            const float limit = fminf(a.cap_near, (ref + kOver) * inv_scale);
            const float2 minus = make_float2(-ref, -ref);
            auto small = [&](float (&z)[32], int c) {
              const float most = largest32(z, 0.f);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 u = gdn::capped_near(make_float2(z[i], z[i + 1]), poly, minus);
                z[i] = u.x, z[i + 1] = u.y;
              }
              if (!__all_sync(0xFFFFFFFFu, most <= limit)) return false;
              if (edge) hide(lo - key0 - c, hi - key0 - c, -INFINITY, z);
              weights(z, c);
              return true;
            };
            int c = 0;  // keys done
            // Not where slots are junk (past the sequence's end, or before every window):
            // they would take part in the choice.
            if (key0 >= seg_lo && key0 + kKeys <= seg_hi) {
              tmem_ld32_nw(s_addr, x);
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {
                tmem_wait_ld32(x);
                tmem_ld32_nw(s_addr + 64 * h + 32, y);
                if (!small(x, 64 * h)) break;
                c += 32;
                tmem_wait_ld32(y);
                if (h == 0) tmem_ld32_nw(s_addr + 64, x);
                if (!small(y, 64 * h + 32)) break;
                c += 32;
                publish(h);
              }
              if (c < kKeys) {  // no load is left on its way
                tmem_wait_ld32(x);
                pin32(y);
              }
            }
            if (c > 0 && m == -INFINITY && lo < key0 + c && hi > key0) m = kAbove;
            // The rest of a block with a score that is not small.
#pragma unroll 1
            for (; c < kKeys; c += 32) {
              float z[32];
              gdn::tmem_ld32(s_addr + c, z);
              cap_scores(a, poly, s_addr + c, z);
              if (edge) hide(lo - key0 - c, hi - key0 - c, -INFINITY, z);
              const float mx = ceilf(max32(z)) + kAbove;
              if (__any_sync(0xFFFFFFFFu, mx > m)) {
                // O is complete up to this half: S came behind the blocks before, and the
                // first half's product is waited for.
                if (c >= 64 && !wait(&sh.mid[t], n & 1)) break;
                gdn::tc_fence_after();
                const float r = move(fmaxf(m, mx), j > 0 || c >= 64);
                if (c & 32) {
                  // The half's first 32 weights have been written: by a power of two, exactly.
                  float w[16];
                  uint32_t v[16];
                  gdn::tmem_wait_st();
                  gdn::tmem_ld16(s_addr + c / 2 - 16, w);
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    const float2 f = gdn::unpack_bf162(__float_as_uint(w[i]));
                    v[i] = gdn::pack_bf162(f.x * r, f.y * r);
                  }
                  gdn::tmem_st16(s_addr + c / 2 - 16, v);
                }
              }
              const float by = m == -INFINITY ? 0.f : m;
#pragma unroll
              for (int i = 0; i < 32; ++i) z[i] -= by;
              weights(z, c);
              if (c & 32) publish(c > 64);
            }
          }
          if (!ok) break;
        } else {
          float mx;
          if constexpr (kInRegisters) {
            mx = max128(s);
            if (kScores == kPlain) mx *= a.scale_log2;
            if (kScores == kBiased) mx += first_bias;
          } else {
            // Changed and masked scores go back to TMEM.
            mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kKeys; c += 32) {
              float x[32];
              gdn::tmem_ld32(s_addr + c, x);
              if (a.cap_log2 > 0.f) {
                cap_scores(a, poly, s_addr + c, x);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= a.scale_log2;
              }
              if (a.slopes) {
                const float back = static_cast<float>(pos - key0 - c);  // distance of the first key
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = fmaf(-slope, fabsf(back - static_cast<float>(i)), x[i]);
              }
              if (edge) hide(lo - key0 - c, hi - key0 - c, -INFINITY, x);
              tmem_st32_nw(s_addr + c, reinterpret_cast<const uint32_t*>(x));
              float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
              for (int i = 4; i < 32; ++i) top[i & 3] = fmaxf(top[i & 3], x[i]);
              mx = fmaxf(mx, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
            }
            gdn::tmem_wait_st();
          }
          // The reference moves when a maximum is more than 2^8 above it.  O of the blocks
          // before is complete: S came behind it.
          const bool grow = mx > m + 8.f || (m == -INFINITY && mx > m);
          if (__any_sync(0xFFFFFFFFu, grow)) move(fmaxf(m, mx), j > 0);
          float ref = m == -INFINITY ? 0.f : m;  // a row that has seen no key yet: weights 2^-inf = 0
          if (kScores == kBiased) ref -= first_bias;
          // Weights over the first half of their S columns: fp32 into the sum; bf16, as
          // the values are, into the product (the tensor core takes both operands in one
          // type; outputs differ from 64 bits by 0.0020 to 0.0023 of their norm, where
          // rounding the exact ones to bf16 gives 0.0017).  64 keys at a time, so that
          // the first half of P V runs beside the exponentials of the second.
          const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), ref2 = make_float2(-ref, -ref);
          auto weight = [&](float2 x) {
            if (kScores == kPlain) x = __ffma2_rn(x, scale2, ref2);
            if (kScores == kGeneral || kScores == kBiased) x = __fadd2_rn(x, ref2);
            x = make_float2(gdn::exp2_approx(x.x), gdn::exp2_approx(x.y));
            l2 = __fadd2_rn(l2, x);
            return gdn::pack_bf162(x);
          };
          if constexpr (kInRegisters) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t p[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) p[i] = weight(make_float2(s[64 * h + 2 * i], s[64 * h + 2 * i + 1]));
              tmem_st32_nw(s_addr + 32 * h, p);
              publish(h);
            }
          } else {
            auto weights = [&](float (&x)[32], int c) {
              uint32_t p[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) p[i] = weight(make_float2(x[2 * i], x[2 * i + 1]));
              gdn::tmem_st16_nw(s_addr + c / 2, p);
            };
            // The next 32 scores are on their way meanwhile.
            float x[32], y[32];
            tmem_ld32_nw(s_addr, x);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              tmem_wait_ld32(x);
              tmem_ld32_nw(s_addr + 64 * h + 32, y);
              weights(x, 64 * h);
              tmem_wait_ld32(y);
              if (h == 0) tmem_ld32_nw(s_addr + 64, x);
              weights(y, 64 * h + 32);
              publish(h);
            }
          }
        }
      }
      if (!ok) break;
      if (taken > 0 && !wait(&sh.o_free[t], (taken - 1) & 1)) break;  // the epilogue has taken the last segment's
      sh.stat[t][row] = make_float2(m, l2.x + l2.y);
      ++taken;
      __syncwarp();
      if (lane == 0) gdn::mbar_arrive(&sh.stat_full[t]);
    }
    if (!ok) *abort_flag = 1;
  }
  gdn::tc_fence_before();
  __syncthreads();
  gdn::tc_fence_after();
  if (tid == 0 && sh.abort) {
    gdn::record_error(a.paged.err_word, GDN_DEVERR_TIMEOUT, 0);
    if (!d.whole) d.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);  // nothing to join
  }
  __syncwarp();
  if (warp == kMmaWarp) gdn::tmem_dealloc(tmem, 512);
}

// Joins the partial results of the items that CTAs of the kernel above cut: the
// item that CTA c started and did not end has slot 1 of c, then slot 0 of every
// CTA up to the one that ended it.  Four blocks per SM share the cut items out
// between them, in slices of 32 rows and half of the dimensions (a block for every
// CTA and slice took 4 us to launch, most of them to find nothing); a thread takes
// one row and D / 64 groups of four dimensions.  Latency-bound: the parts are added
// in a fixed order, four of them in flight.
constexpr int kJoinSlices = 16;
constexpr int kJoinThreads = 256;
static_assert(kMaxGrid <= kJoinThreads, "one thread per record");
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4) chunk_join_kernel(const __grid_constant__ ChunkArgs d, int ctas) {
  __shared__ int4 cuts[kMaxGrid];
  __shared__ int owners[kMaxGrid];
  __shared__ int count[kJoinThreads / 32];
  gdn::pdl_wait();
  gdn::pdl_launch_dependents();
  const AttnArgs& a = d.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int4 mine = tid < ctas ? d.cuts[tid] : make_int4(-1, 0, 0, 0);
  const unsigned found = __ballot_sync(0xFFFFFFFFu, mine.x >= 0);
  if (lane == 0) count[warp] = __popc(found);
  __syncthreads();
  int at = __popc(found & ((1u << lane) - 1)), total = 0;
  for (int i = 0; i < kJoinThreads / 32; ++i) {
    if (i < warp) at += count[i];
    total += count[i];
  }
  if (mine.x >= 0) cuts[at] = mine, owners[at] = tid;
  __syncthreads();
  constexpr int kG = D / 64;  // groups of four dimensions per thread
  constexpr int kParts = 4;
  for (int job = blockIdx.x; job < total * kJoinSlices; job += gridDim.x) {
    const int4 cut = cuts[job / kJoinSlices];
    const int c = owners[job / kJoinSlices], slice = job % kJoinSlices;
    const int t = slice >> 3, row = (slice & 3) * 32 + lane;
    const int in_tile = row / a.group;
    const int token = t * d.tile_tokens + in_tile;
    if (in_tile >= d.tile_tokens || token >= cut.y) continue;
    const int group0 = warp + 8 * kG * ((slice >> 2) & 1);
    float m = -INFINITY, l = 0.f;
    float4 o[kG];
#pragma unroll
    for (int k = 0; k < kG; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = c; i0 <= cut.w; i0 += kParts) {
      float2 ml[kParts];
      float4 x[kParts][kG];
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        ml[p] = make_float2(-INFINITY, 0.f);
        const int i = i0 + p;
        if (i > cut.w) continue;
        const int64_t slot = (2 * static_cast<int64_t>(i) + (i == c ? 1 : 0)) * 2 + t;
        ml[p] = d.part_ml[slot * kRows + row];
#pragma unroll
        for (int k = 0; k < kG; ++k) x[p][k] = d.part_o[(slot * (D / 4) + group0 + 8 * k) * kRows + row];
      }
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        if (ml[p].x == -INFINITY) continue;  // no part, or one in which the row saw no key
        const float top = fmaxf(m, ml[p].x);
        const float f = gdn::exp2_approx(m - top), g = gdn::exp2_approx(ml[p].x - top);
        m = top;
        l = l * f + ml[p].y * g;
#pragma unroll
        for (int k = 0; k < kG; ++k) {
          o[k].x = o[k].x * f + x[p][k].x * g;
          o[k].y = o[k].y * f + x[p][k].y * g;
          o[k].z = o[k].z * f + x[p][k].z * g;
          o[k].w = o[k].w * f + x[p][k].w * g;
        }
      }
    }
    const float inv = 1.f / l;
    const int64_t out = (static_cast<int64_t>(cut.x) + token) * a.Hq + cut.z * a.group + row % a.group;
#pragma unroll
    for (int k = 0; k < kG; ++k)
      reinterpret_cast<uint2*>(a.o + out * D)[group0 + 8 * k] =
          make_uint2(gdn::pack_bf162(o[k].x * inv, o[k].y * inv), gdn::pack_bf162(o[k].z * inv, o[k].w * inv));
    if (a.lse && group0 == 0) a.lse[out] = (m + log2f(l)) / gdn::kLog2e;
  }
}

constexpr size_t kCutBytes = kMaxGrid * sizeof(int4);
// Known before the launch: then there is no join either (2 us of GPU time, 4 with the
// workspace's allocation: 16 x 100 on pages of 128 take 16.5 us, 20 with it).  The page
// table is on the device; here every sequence is taken to own a page, which one
// without new tokens need not.  Where that is certainly not so, or a mistake would
// leave more than a few blocks whole, the kernel decides, which sees the lengths (16
// tokens over 131,072 beside 128 sequences without pages: 1,143 us whole, 94 so).
bool whole_items(int32_t num_seqs, int32_t num_entries, int32_t page_size) {
  return num_entries >= num_seqs && static_cast<int64_t>(num_entries) * page_size <= 4 * kWholeKeys &&
         gdn_host::longest_sequence(num_seqs, num_entries, page_size) <= kWholeKeys;
}
size_t workspace_bytes_of(int D, bool whole) {
  if (whole) return 0;
  return kCutBytes + static_cast<size_t>(4) * kMaxGrid * kRows * (sizeof(float2) + D * sizeof(float));
}

// queue(kernel, smem): launches it.
template <int D, bool kCodes, typename Kernel, typename Queue>
int launch_chunk(Kernel kernel, ChunkArgs& d, int32_t total_tokens, std::atomic<uint64_t>& done, void* workspace,
                 int sms, cudaStream_t stream, const Queue& queue) {
  constexpr int smem = kSmemBytes<D, kCodes>;
  static_assert(smem <= 232448, "shared memory of one CTA");
  int rc = gdn_host::func_attr_once(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem, done);
  if (rc != GDN_OK) return rc;
  // The register split would wait for ever in a block that holds fewer.
  static const bool fits = [&] {
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, kernel) == cudaSuccess && attr.numRegs * kThreads >= Registers<kCodes>::kSum;
  }();
  if (!fits) return GDN_ERR_CUDA;
  CUtensorMap q_map;
  const int64_t dims[4] = {D, d.a.group, total_tokens, d.a.Hkv};
  const int64_t strides[3] = {2 * D, 2 * d.a.q_stride, 2 * static_cast<int64_t>(d.a.group) * D};
  if ((rc = gdn_host::encode_map_4d(&q_map, d.a.q, dims, strides, d.a.group, d.tile_tokens)) != GDN_OK) return rc;
  const int grid = sms < kMaxGrid ? sms : kMaxGrid;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  d.cuts = reinterpret_cast<int4*>(ws);
  d.part_ml = reinterpret_cast<float2*>(ws + kCutBytes);
  d.part_o = reinterpret_cast<float4*>(ws + kCutBytes + sizeof(float2) * 4 * kMaxGrid * kRows);
  if ((rc = queue(dim3(grid), dim3(kThreads), smem, q_map)) != GDN_OK || d.whole) return rc;
  return gdn_host::launch_pdl(chunk_join_kernel<D>, dim3(4 * grid), dim3(kJoinThreads), 0, stream, d, grid);
}

// Calls run with the dimension and what the options make of the scores.
template <typename Run>
int by_scores(const AttnArgs& a, int32_t D, const Run& run) {
  const bool capped = a.cap_log2 > 0.f && !a.slopes;
  const bool linear = a.slopes && a.cap_log2 == 0.f && !a.full_lens;
  const Scores scores = capped ? kCapped : linear ? kBiased : a.slopes ? kGeneral : kPlain;
  const auto of = [&](auto dim) {
    switch (scores) {
      case kPlain: return run(dim, std::integral_constant<Scores, kPlain>());
      case kBiased: return run(dim, std::integral_constant<Scores, kBiased>());
      case kGeneral: return run(dim, std::integral_constant<Scores, kGeneral>());
      default: return run(dim, std::integral_constant<Scores, kCapped>());
    }
  };
  return D == 64 ? of(std::integral_constant<int, 64>()) : of(std::integral_constant<int, 128>());
}

}  // namespace
