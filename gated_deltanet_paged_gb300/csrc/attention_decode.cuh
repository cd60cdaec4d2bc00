// attention_decode.cuh -- what the single-token kernels of both caches share: how a batch
// is shared out, the join of a CTA's warps and that of the items that CTAs cut.  A block
// is kBlock keys, as many as 16 KB hold.
#pragma once

#include "attention_common.cuh"

namespace {  // each kernel's file has its own

using gdn::AttnArgs;
using gdn::SeqRange;

// Two stages, so 128 KB on their way per SM: with a third the queues before HBM
// grow and its rate falls (256 sequences, 8.5 GB: 1.23 ms against 1.17).
constexpr int kStages = 2;
// Consumer warps, each with its part of a block's keys, beside one warp that copies keys
// and one that copies values.
constexpr int threads_of(int consumers) { return (consumers + 2) * 32; }
constexpr int kRows = 16;     // query heads of a key head at most (see gdn_attention_decode_paged)
constexpr int kTileBytes = 16384;
// Fixed cost of an item (its queries, the join of the warps, its stores) in
// blocks, so that shares of many short items weigh the same as shares of long ones
// (512 sequences of 100 to 300 keys, 8 key heads of 128: 89 us, with 4 92).  Over an 8-bit
// cache, whose blocks have twice the keys, one (61 sequences of up to 9,000 17.1 us, with
// two 18.1).
constexpr int kItemCost16 = 2, kItemCost8 = 1;
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
template <int kBlock, int kItemCost>
__device__ __forceinline__ Item load_item(const AttnArgs& a, int b) {
  Item it;
  it.s = gdn::seq_range(a.paged, b);
  it.hi = it.s.len;
  it.lo = gdn::key_lo(a, it.s.len - 1);
  it.first = it.lo / kBlock;
  it.blocks = (it.hi + kBlock - 1) / kBlock - it.first;
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
template <int kBlock, int kItemCost>
__device__ __forceinline__ bool next_segment(const DecodeArgs& d, Walk& w) {
  const int per_seq = d.a.Hkv;
  if (d.whole) {
    while (w.pos < w.end) {
      const int id = static_cast<int>(w.pos);
      w.pos += gridDim.x;
      const int b = id / per_seq;
      if (b != w.b) w.b = b, w.it = load_item<kBlock, kItemCost>(d.a, b);
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
      w.it = load_item<kBlock, kItemCost>(d.a, ++w.b);
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

// kTiles: the join's tiles of a warp, a float4 a lane; kPairs: pairs of rows whose maximum
// and sum a lane has.
template <int kConsumers, int kTiles, int kPairs>
struct Smem {
  static constexpr int kTile = kTileBytes;  // one of K, V
  alignas(1024) uint8_t kv[kStages][2][kTile];
  float4 join_o[kConsumers][kTiles][32];  // the warps' partial results, lane by lane
  float4 join_ml[kConsumers][kPairs][32];  // m, l of two rows
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t never;  // the test hook's barrier, never completed
  int64_t scan[kConsumers + 3];
  Walk walk;
  int abort;
  int stop;
};

// The loop out of line: this kernel's instructions are rarely in the cache (in line: 2
// short sequences 5.45 us instead of 5.35, 61 sequences 15.95 instead of 15.7).
static __device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, const volatile int* abort, uint32_t limit_ns) {
  return gdn::warp_wait_more(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort, uint32_t limit_ns) {
  if (__all_sync(0xFFFFFFFFu, gdn::mbar_try_wait(bar, parity))) return true;
  return wait_more(bar, parity, abort, limit_ns);
}

template <int kConsumers>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}

// This CTA's share of the line; false: none.  All threads take it together.
template <int kBlock, int kItemCost, int kConsumers, int kTiles, int kPairs>
__device__ __forceinline__ bool take_share(const DecodeArgs& d, Smem<kConsumers, kTiles, kPairs>& sh, Walk& w, gdn::Shares<0>& shares) {
  constexpr int kThreads = threads_of(kConsumers);
  const AttnArgs& a = d.a;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int per_seq = a.Hkv;
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
      const Item it = load_item<kBlock, kItemCost>(a, b);
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
      x.it = load_item<kBlock, kItemCost>(a, b0);
      while (start >= x.base + static_cast<int64_t>(x.it.cost) * per_seq) {
        x.base += static_cast<int64_t>(x.it.cost) * per_seq;
        x.it = load_item<kBlock, kItemCost>(a, ++x.b);
      }
      sh.walk = x;
    }
    if (tid == 0) d.cuts[c] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    if (start >= end) return false;
    w = sh.walk;
  }
  return true;
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

// The kernel over the batch and, where items may be cut, the join.  queue(grid): launches
// the kernel.
template <int D, typename Queue>
int launch_shared(DecodeArgs& d, const gdn_page_table* table, void* workspace, int sms, cudaStream_t stream, const Queue& queue) {
  const int64_t items = static_cast<int64_t>(table->num_seqs) * d.a.Hkv;
  int grid = 2 * sms < kMaxGrid ? 2 * sms : kMaxGrid;
  if (d.whole && items < grid) grid = static_cast<int>(items);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  d.cuts = reinterpret_cast<int4*>(ws);
  d.part_ml = reinterpret_cast<float2*>(ws + kMaxGrid * sizeof(int4));
  d.part_o = reinterpret_cast<float*>(ws + kMaxGrid * sizeof(int4) + sizeof(float2) * 2 * kMaxGrid * kRows);
  const int rc = queue(grid);
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
