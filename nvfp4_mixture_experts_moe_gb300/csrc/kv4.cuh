// The NVFP4 key/value cache as the kernels see it (include/moe_block.h has
// the layout) and the launchers of the block operators.
#pragma once

#include "common.cuh"
#include "moe_block.h"

namespace moe {

constexpr int kKvBlock = 16;  // tokens of one contiguous block of a (page, head)

// Byte offsets inside a block of 16 tokens.
template <int D>
struct Kv4Block {
  static constexpr int kCodeRow = D / 2, kScaleRow = D / 16;
  static constexpr int kKeyScales = kKvBlock * kCodeRow;
  static constexpr int kValueCodes = kKeyScales + kKvBlock * kScaleRow;
  static constexpr int kValueScales = kValueCodes + kKvBlock * kCodeRow;
  static constexpr int kBytes = kValueScales + kKvBlock * kScaleRow;
  static_assert(kBytes == 18 * D, "block bytes");
};

// Offset of the 16-token block that holds a slot, for one head. 64-bit: a
// pool of 2^31 tokens is far larger than 2^32 bytes.
__device__ __forceinline__ size_t kv4_block_offset(int64_t page, int head, int kv_heads, int blocks_per_page,
                                                   int block, int block_bytes) {
  return (((size_t)page * kv_heads + head) * blocks_per_page + block) * (size_t)block_bytes;
}

// (x * y + z) / d of non-negative numbers; a 64-bit division (some 300
// cycles) only where 32 bits do not hold the product.
__device__ __forceinline__ int mul_div(int x, int y, int d, int z = 0) {
  const unsigned long long t = (unsigned long long)x * y + z;
  return t >> 32 ? (int)(t / d) : (int)((unsigned)t / (unsigned)d);
}

moe_status launch_kv4_append(const moe_kv4_cache& c, const uint16_t* k, const uint16_t* v, long long k_stride,
                             long long v_stride, const int32_t* slots, int tokens, int32_t* status, cudaStream_t s);
moe_status launch_kv4_read(const moe_kv4_cache& c, const int32_t* slots, int n, uint16_t* k_out, uint16_t* v_out,
                           int32_t* status, cudaStream_t s);
moe_status launch_kv_step(const moe_kv_step_args& a, cudaStream_t s);
moe_status launch_block_norm(const moe_block_norm_args& a, cudaStream_t s);

// Attention of requests with up to max_rows (at most kKvDecodeRows) query rows
// per key/value head; the others are skipped.
constexpr int kKvDecodeRows = 16;
constexpr int kKvMaxCtas = 160;      // CTAs of the attention kernels, one per SM
constexpr int kKvTilesPerCta = 4;    // fewer decode tiles than this do not get a CTA of their own
size_t kv4_decode_ws_floats(int head_dim, int rows);
moe_status launch_kv4_decode(const moe_kv4_attn_args& a, int max_rows, int* status, int* counters, float* partials,
                             cudaStream_t s);
// Attention of requests with more than min_rows rows; overlap: the launch
// before in the stream is launch_kv4_decode's, with other partials.
size_t kv4_prompt_ws_floats(int head_dim);
long long kv4_prompt_units(const moe_kv4_attn_args& a);   // a bound on the units of work it counts in 32 bits
moe_status launch_kv4_prompt(const moe_kv4_attn_args& a, int min_rows, int* status, float* partials, bool overlap,
                             cudaStream_t s);

size_t kv4_attention_ws_bytes(const moe_kv4_attn_args& a);
moe_status launch_kv4_attention(const moe_kv4_attn_args& a, void* ws, cudaStream_t s);

}  // namespace moe
