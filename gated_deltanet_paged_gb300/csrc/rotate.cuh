// rotate.cuh -- pieces of heads, their rotation, and the sequence of a token, as the
// kernels of rope.cu and cache8.cu share them.
#pragma once

#include "attention_common.cuh"

namespace gdn {

template <int W>
struct Piece {  // W bf16 elements
  uint32_t r[W >= 2 ? W / 2 : 1];
};
template <int W>
__device__ __forceinline__ Piece<W> load_piece(const __nv_bfloat16* p) {
  Piece<W> x;
  if constexpr (W == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    x.r[0] = u.x, x.r[1] = u.y, x.r[2] = u.z, x.r[3] = u.w;
  } else if constexpr (W == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    x.r[0] = u.x, x.r[1] = u.y;
  } else if constexpr (W == 2) {
    x.r[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    x.r[0] = *reinterpret_cast<const uint16_t*>(p);
  }
  return x;
}
template <int W>
__device__ __forceinline__ void store_piece(__nv_bfloat16* p, const Piece<W>& x) {
  if constexpr (W == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(x.r[0], x.r[1], x.r[2], x.r[3]);
  else if constexpr (W == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(x.r[0], x.r[1]);
  else if constexpr (W == 2)
    *reinterpret_cast<uint32_t*>(p) = x.r[0];
  else
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(x.r[0]);
}
template <int W>
__device__ __forceinline__ float get(const Piece<W>& x, int i) {
  return __uint_as_float((i & 1) ? (x.r[i >> 1] & 0xFFFF0000u) : (x.r[i >> 1] << 16));
}
template <int W>
__device__ __forceinline__ Piece<W> pack(const float (&f)[W]) {
  Piece<W> x;
  if constexpr (W == 1) {
    x.r[0] = gdn::pack_bf162(f[0], 0.f) & 0xFFFFu;
  } else {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) x.r[i] = gdn::pack_bf162(f[2 * i], f[2 * i + 1]);
  }
  return x;
}

// The pair of pieces (a, b) rotated by cs[0 .. W): the halves of W pairs where
// the layout keeps them apart, 2 W consecutive elements where it interleaves
// them.  fp32 throughout, one rounding per result.
template <int W>
__device__ __forceinline__ void rotate(Piece<W>& a, Piece<W>& b, const float2* cs, bool interleaved) {
  float x[W], y[W];
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      // Pair i is elements 2 i and 2 i + 1 of the 2 W.
      const float e = 2 * i < W ? get<W>(a, (2 * i) % W) : get<W>(b, (2 * i) % W);
      const float o = 2 * i + 1 < W ? get<W>(a, (2 * i + 1) % W) : get<W>(b, (2 * i + 1) % W);
      const float2 c = cs[i];
      const float re = e * c.x - o * c.y, im = e * c.y + o * c.x;
      if (2 * i < W) x[(2 * i) % W] = re; else y[(2 * i) % W] = re;
      if (2 * i + 1 < W) x[(2 * i + 1) % W] = im; else y[(2 * i + 1) % W] = im;
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float e = get<W>(a, i), o = get<W>(b, i);
      const float2 c = cs[i];
      x[i] = e * c.x - o * c.y;
      y[i] = e * c.y + o * c.x;
    }
  }
  a = pack<W>(x);
  b = pack<W>(y);
}

// The sequence of token t: the last b with cu_seqlens[b] <= t, by a 32-way
// search of the warp (sequences without new tokens share their start with the
// next one, so the last is the one that holds t).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int num_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = num_seqs;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < lo + n && cu[at] <= t;
    const int k = max(__popc(__ballot_sync(0xFFFFFFFFu, below)) - 1, 0);
    n = min(step, lo + n - (lo + k * step));
    lo += k * step;
  }
  return lo;
}

constexpr int kMaxPairs = 256;  // rotary_dim <= 512

// Sine and cosine of a pair at a position, times the amplitude.
__device__ __forceinline__ float2 pair_turn(int position, int64_t frequency, float amplitude, float sign) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(position)) * static_cast<uint64_t>(frequency);
  const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
  float sn, cn;
  sincospif(half_turns, &sn, &cn);
  return make_float2(cn * amplitude, sn * amplitude * sign);
}

}  // namespace gdn

namespace gdn_host {

inline bool bad_rotation(const int64_t* frequencies, int32_t rotary_dim, int32_t D, float amplitude) {
  if (!frequencies) return rotary_dim != 0;
  return rotary_dim <= 0 || rotary_dim % 2 != 0 || rotary_dim > D || rotary_dim / 2 > gdn::kMaxPairs ||
         (reinterpret_cast<uintptr_t>(frequencies) & 7u) != 0 || !isfinite(amplitude);
}

inline const __nv_bfloat16* bf(const gdn_bf16* p) { return reinterpret_cast<const __nv_bfloat16*>(p); }
inline __nv_bfloat16* bf(gdn_bf16* p) { return reinterpret_cast<__nv_bfloat16*>(p); }

// The widest piece that divides the rotated halves and the copied rest.
inline int piece_width(int32_t half, int32_t D) {
  int W = 8;
  while (half % W != 0 || (D / 2 - half) % W != 0) W >>= 1;
  return W;
}

}  // namespace gdn_host
