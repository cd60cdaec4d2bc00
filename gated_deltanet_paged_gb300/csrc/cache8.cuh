// cache8.cuh -- the 8-bit cache as its kernels share it: its layout on the device,
// conversions, and the host checks.
#pragma once

#include "attention_common.cuh"

namespace gdn {

constexpr int kGroup = GDN_FP8_GROUP;  // tokens per scale
// Scale bytes that an append writes: 2^-112 to 2^119.  Every code times such a scale is
// a normal bf16 number (or zero): 2^-9 * 2^-112 and 448 * 2^119 < 2^128 are.
constexpr int kScaleLeast = 127 - 112, kScaleMost = 127 + 119;

struct Cache8 {
  uint8_t* codes[2];   // keys, values
  uint8_t* scales[2];
  int64_t page_stride, token_stride, head_stride;
  int64_t scale_page, scale_group, scale_head;
};

// 2^(byte - 127).  0 stands for 2^-127, which is less than any float that a product
// with it could need; it becomes 0.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Four e4m3 codes as fp16, exactly (NaN stays NaN): those in the low half of a word, and
// those in the high half.
__device__ __forceinline__ void e4m3_to_half4(uint32_t four, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(four));
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Four codes times a scale, in bf16 (exact for the scales that an append writes).
__device__ __forceinline__ uint2 e4m3_to_bf16(uint32_t four, float2 scale) {
  uint32_t a, b;
  e4m3_to_half4(four, a, b);
  return make_uint2(pack_bf162(__fmul2_rn(half2_to_float2(a), scale)), pack_bf162(__fmul2_rn(half2_to_float2(b), scale)));
}
// Rounded to nearest, ties to even; beyond 448 (infinities too) to 448; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
  return x;
}
// Byte offset of 16-byte chunk c of key r of a tile: swizzled over 128 or 64 bytes.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(uint32_t r, uint32_t c) {
  if constexpr (D == 128) return swz(r, c);
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

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

  __device__ __forceinline__ ScaleCopies(const AttnArgs& args, const Cache8& c, int kv, int l)
      : a(args), scales(c.scales[kv]), page_stride(c.scale_page), group_stride(c.scale_group), head_stride(c.scale_head),
        lane(l) {}
  __device__ __forceinline__ void look_ahead() {
    byte = 127;
    if (lane >= kBlockKeys / kGroup || key + kGroup <= lo || key >= hi) return;
    const int p = pages[entry];
    if (p >= 0 && p < a.paged.num_pages)  // else its codes are zeros, reported by the copies
      byte = scales[p * page_stride + (slot / kGroup) * group_stride + head_at];
  }
  __device__ __forceinline__ void begin(int from, int to, int head, int table_entry, int first) {
    lo = from, hi = to, head_at = head * head_stride;
    pages = a.paged.pages + table_entry;
    key = first + lane * kGroup;
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

}  // namespace gdn

namespace gdn_host {

// Checks of an 8-bit cache and a page table that need no device data.  `shell`
// receives the same as a cache of codes, for what both kinds of cache share.
inline int check_paged8(const gdn_kv_cache_fp8* c, const gdn_page_table* t, const int32_t* cu_seqlens,
                        int32_t total_tokens, gdn_kv_cache* shell) {
  if (!c || !c->k_scales || !c->v_scales) return GDN_ERR_INVALID_ARGUMENT;
  *shell = gdn_kv_cache{reinterpret_cast<gdn_bf16*>(c->k), reinterpret_cast<gdn_bf16*>(c->v), c->num_pages, c->page_size,
                        c->num_heads, c->head_dim, c->page_stride, c->token_stride, c->head_stride};
  const int rc = check_paged(shell, t, cu_seqlens, total_tokens);
  if (rc != GDN_OK) return rc;
  if (c->head_dim != 64 && c->head_dim != 128) return GDN_ERR_UNSUPPORTED;
  if (c->page_size % gdn::kGroup != 0 || c->num_heads > 65535) return GDN_ERR_UNSUPPORTED;
  if (c->page_stride % 16 != 0 || c->token_stride % 16 != 0 || c->head_stride % 16 != 0) return GDN_ERR_INVALID_ARGUMENT;
  // An axis of one entry may have any stride.
  if ((c->num_pages > 1 && c->scale_page_stride < 1) || (c->page_size > gdn::kGroup && c->scale_group_stride < 1) ||
      (c->num_heads > 1 && c->scale_head_stride < 1))
    return GDN_ERR_INVALID_ARGUMENT;
  return GDN_OK;
}

// Tensor map of one array of codes, {D, heads, slots, pages}, with boxes of 2^box_shift
// slots of one head.
inline int encode_codes_map(CUtensorMap* map, const uint8_t* base, const gdn_kv_cache_fp8* c, int box_shift) {
  const int64_t dims[4] = {c->head_dim, c->num_heads, c->page_size, c->num_pages};
  const int64_t strides[3] = {c->num_heads > 1 ? c->head_stride : c->head_dim, c->page_size > 1 ? c->token_stride : c->head_dim,
                              c->num_pages > 1 ? c->page_stride : c->head_dim};
  return encode_bytes_map_4d(map, base, dims, strides, 1, 1 << box_shift);
}

inline gdn::Cache8 cache8(const gdn_kv_cache_fp8* c) {
  return gdn::Cache8{{c->k, c->v},      {c->k_scales, c->v_scales}, c->page_stride,        c->token_stride,
                     c->head_stride, c->scale_page_stride,       c->scale_group_stride, c->scale_head_stride};
}

// What a batch's new tokens may see, as bf16 pages [num_entries, Hkv, page_size, D] (32-byte
// aligned) in the order of the table, and their numbers.
int expand8(const gdn_kv_cache_fp8* cache, const gdn::PagedTokens& paged, int32_t window, gdn_bf16* k, gdn_bf16* v,
            int32_t* pages, int sms, cudaStream_t stream);

}  // namespace gdn_host
