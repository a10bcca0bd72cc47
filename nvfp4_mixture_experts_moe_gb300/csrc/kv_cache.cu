// Rows of keys and values into the paged NVFP4 cache, and back to bf16.
//
// The quantiser is moe_nvfp4_quantize_static's: per 16 elements s = (amax /
// 6) * gs to E4M3, codes e2m1(x * (gs / scale)), every step a correctly
// rounded fp32 operation ("vLLM on the NVIDIA DGX Spark: A Complete
// Technical Guide", section 6.1; the cache's format: "Qwen3.8-Flash-Next-NVFP4
// . 2x DGX Spark . SGLang TP2").
#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// One thread per block of 16 elements: 32 bytes of bf16 in, 8 bytes of codes
// and a scale byte out. A warp takes D/16 blocks of 512/D consecutive tokens
// of one head, so with consecutive slots its codes and scales are whole
// 32-byte sectors.
template <int D>
struct Place {
  static constexpr int kBlocks = D / 16;
  static constexpr int kTokens = 32 / kBlocks;
  int blk, h, kv, t;
  __device__ __forceinline__ explicit Place(size_t i, int Hk) {
    blk = (int)(i % kBlocks);
    i /= kBlocks;
    const int tl = (int)(i % kTokens);
    i /= kTokens;
    h = (int)(i % Hk);
    i /= Hk;
    kv = (int)(i & 1);
    t = (int)(i >> 1) * kTokens + tl;
  }
  static size_t threads(int tokens, int Hk) {
    return (size_t)((tokens + kTokens - 1) / kTokens) * 2 * Hk * 32;
  }
};

// The block and the row within it of a slot; false for a slot outside the pool.
template <int D>
__device__ __forceinline__ uint8_t* slot_row(const moe_kv4_cache& c, int slot, int h, int& row) {
  const int page = slot / c.page_tokens, pos = slot - page * c.page_tokens;
  row = pos % kKvBlock;
  return static_cast<uint8_t*>(c.pool) +
         kv4_block_offset(page, h, c.kv_heads, c.page_tokens / kKvBlock, pos / kKvBlock, Kv4Block<D>::kBytes);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    kv4_append_kernel(moe_kv4_cache c, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                      long long k_stride, long long v_stride, const int32_t* __restrict__ slots, int tokens,
                      int32_t* status) {
  using L = Kv4Block<D>;
  const Place<D> p(blockIdx.x * (size_t)kThreads + threadIdx.x, c.kv_heads);
  if (p.t >= tokens) return;
  const int slot = slots[p.t];
  if (slot < 0) return;
  if (slot >= c.num_pages * c.page_tokens) {
    if (status != nullptr) *status = MOE_ERR_DEVICE;
    return;
  }
  const uint16_t* src = p.kv ? v + (size_t)p.t * v_stride : k + (size_t)p.t * k_stride;
  src += (size_t)p.h * D + p.blk * 16;
  const uint4 v0 = ldg_stream(src), v1 = ldg_stream(src + 8);
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  float f[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16);
    f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (!(f[j] == f[j])) f[j] = 0.0f;  // a NaN has no code: stored as 0
    amax = fmaxf(amax, fabsf(f[j]));
  }
  const float gs = p.kv ? c.v_gs : c.k_gs;
  const uint32_t scale = e4m3_encode_sat(__fmul_rn(__fdiv_rn(amax, 6.0f), gs));
  const float sval = e4m3_decode(scale);
  uint32_t lo = 0, hi = 0;
  if (sval > 0.0f) {
    const float r = __fdiv_rn(gs, sval);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = e2m1x2_rn(__fmul_rn(f[2 * j], r), __fmul_rn(f[2 * j + 1], r));
      if (j < 4) lo |= b << (8 * j);
      else hi |= b << (8 * (j - 4));
    }
  }
  int row;
  uint8_t* blk = slot_row<D>(c, slot, p.h, row) + (p.kv ? L::kValueCodes : 0);
  *reinterpret_cast<uint2*>(blk + row * L::kCodeRow + p.blk * 8) = make_uint2(lo, hi);
  blk[L::kKeyScales + row * L::kScaleRow + p.blk] = (uint8_t)scale;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(moe_kv4_cache c, const int32_t* __restrict__ slots, int n, uint16_t* k_out, uint16_t* v_out,
                    int32_t* status) {
  using L = Kv4Block<D>;
  const Place<D> p(blockIdx.x * (size_t)kThreads + threadIdx.x, c.kv_heads);
  if (p.t >= n) return;
  uint16_t* out = p.kv ? v_out : k_out;
  if (out == nullptr) return;
  out += ((size_t)p.t * c.kv_heads + p.h) * D + p.blk * 16;
  const int slot = slots[p.t];
  uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (slot >= c.num_pages * c.page_tokens) {
    if (status != nullptr) *status = MOE_ERR_DEVICE;
  } else if (slot >= 0) {
    int row;
    const uint8_t* blk = slot_row<D>(c, slot, p.h, row) + (p.kv ? L::kValueCodes : 0);
    const uint2 codes = *reinterpret_cast<const uint2*>(blk + row * L::kCodeRow + p.blk * 8);
    const float s = e4m3_decode(blk[L::kKeyScales + row * L::kScaleRow + p.blk]);
    const float inv = 1.0f / (p.kv ? c.v_gs : c.k_gs);
    uint32_t h2[8];
    uint32_t a[4], b[4];
    cvt_e2m1x8_f16(codes.x, a);
    cvt_e2m1x8_f16(codes.y, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h2[j] = a[j];
      h2[4 + j] = b[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&h2[j]));
      // code * scale is exact in fp32
      o[j] = float2_to_bf16x2_bits(e.x * s * inv, e.y * s * inv);
    }
  }
  reinterpret_cast<uint4*>(out)[0] = make_uint4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<uint4*>(out)[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace

moe_status launch_kv4_append(const moe_kv4_cache& c, const uint16_t* k, const uint16_t* v, long long k_stride,
                             long long v_stride, const int32_t* slots, int tokens, int32_t* status, cudaStream_t s) {
  const bool d64 = c.head_dim == 64;
  const size_t n = d64 ? Place<64>::threads(tokens, c.kv_heads) : Place<128>::threads(tokens, c.kv_heads);
  const size_t ctas = (n + kThreads - 1) / kThreads;
  if (ctas > 0x7fffffffu) return MOE_ERR_UNSUPPORTED;
  auto kern = d64 ? kv4_append_kernel<64> : kv4_append_kernel<128>;
  cudaError_t e = launch_ex(false, kern, dim3((unsigned)ctas), dim3(kThreads), 0, s, c, k, v, k_stride, v_stride,
                            slots, tokens, status);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

moe_status launch_kv4_read(const moe_kv4_cache& c, const int32_t* slots, int n, uint16_t* k_out, uint16_t* v_out,
                           int32_t* status, cudaStream_t s) {
  const bool d64 = c.head_dim == 64;
  const size_t threads = d64 ? Place<64>::threads(n, c.kv_heads) : Place<128>::threads(n, c.kv_heads);
  const size_t ctas = (threads + kThreads - 1) / kThreads;
  if (ctas > 0x7fffffffu) return MOE_ERR_UNSUPPORTED;
  auto kern = d64 ? kv4_read_kernel<64> : kv4_read_kernel<128>;
  cudaError_t e =
      launch_ex(false, kern, dim3((unsigned)ctas), dim3(kThreads), 0, s, c, slots, n, k_out, v_out, status);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

}  // namespace moe
