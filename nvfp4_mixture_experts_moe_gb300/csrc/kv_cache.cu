// Rows of keys and values into the paged NVFP4 cache, and back to bf16.
//
// The quantiser is moe_nvfp4_quantize_static's: per 16 elements s = (amax /
// 6) * gs to E4M3, codes e2m1(x * (gs / scale)), every step a correctly
// rounded fp32 operation ("vLLM on the NVIDIA DGX Spark: A Complete
// Technical Guide", section 6.1; the cache's format: "Qwen3.8-Flash-Next-NVFP4
// . 2x DGX Spark . SGLang TP2").
//
// What bounds them: bytes for prompts, latency for a decode step (1.8 us a
// launch, replayed). 8191 tokens of 8 heads x 128 written and read back move
// 86 MB, 12.7 us at the measured copy rate; replayed, the two take 7.9 and 7.3
// us (L2 holds what was just written), from and to memory 10 each, some 3 of
// them launch, first loads and last stores. Instructions issue in 0.61 and 0.65
// of the cycles (206 and 178 a warp and 512 elements; append's have three
// correctly rounded divisions among them).
#include <cmath>

#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

// One thread per block of 16 elements: 32 bytes of bf16 on one side, 8 bytes
// of codes and a scale byte on the other. A warp takes D/16 blocks of 512/D
// consecutive tokens of one head's keys or values, so with consecutive slots
// its codes and scales are whole 32-byte sectors; the warps of a CTA take
// the heads and sides of those tokens, which lie side by side in a row.
constexpr int kMaxWarps = 16;
template <int D>
struct Place {
  static constexpr int kBlocks = D / 16;
  static constexpr int kTokens = 32 / kBlocks;
  int blk, h, kv, t;
  __device__ __forceinline__ Place() {
    const int pair = blockIdx.y * blockDim.y + threadIdx.y;
    blk = threadIdx.x % kBlocks;
    t = blockIdx.x * kTokens + threadIdx.x / kBlocks;
    h = pair >> 1;
    kv = pair & 1;
  }
};

template <class K, class... A>
moe_status launch_cache(K kernel, int D, int Hk, int tokens, cudaStream_t s, A... args) {
  const int warps = 2 * Hk < kMaxWarps ? 2 * Hk : kMaxWarps, per = 512 / D;
  const dim3 grid((unsigned)(((long long)tokens + per - 1) / per), (2 * Hk + warps - 1) / warps);
  const cudaError_t e = launch_ex(true, kernel, grid, dim3(32, warps), 0, s, args...);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

// The cache with what every thread would work out again: page_tokens is a
// power of two. Keys' and values' global scales: gs itself for append, for
// read, which divides by it, its reciprocal as the sum of two floats.
struct Cache {
  uint8_t* pool;
  int slots, heads, page_log;
  float2 gs[2];
};

float2 reciprocal(float gs) {
  const double inv = 1.0 / gs;
  const float x = (float)inv;
  return {x, std::isfinite(x) ? (float)(inv - x) : 0.0f};
}

Cache cache_of(const moe_kv4_cache& c, float2 k_gs, float2 v_gs) {
  return {static_cast<uint8_t*>(c.pool), c.num_pages * c.page_tokens, c.kv_heads, __builtin_ctz(c.page_tokens),
          {k_gs, v_gs}};
}

// e * scale / gs of a pair of codes, rounded once to bf16: e * (t + rest) is
// truncated to fp32 and its last bit set (round to odd) before it is rounded.
// e * scale has at most six significant bits, so the quotient is either a bf16
// value, which the last bit does not move, or not half way between two, and
// what was cut off no longer counts. (e * scale times the rounded reciprocal
// in fp32 is off in one of some 50,000 values.)
__device__ __forceinline__ uint32_t quotients(uint32_t e_f16x2, uint64_t t, uint64_t rest) {
  const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&e_f16x2));
  uint32_t x, y;
  asm("{\n .reg .b64 e, r;\n mov.b64 e, {%2, %3};\n mul.rn.f32x2 r, e, %5;\n fma.rz.f32x2 r, e, %4, r;\n"
      " mov.b64 {%0, %1}, r;\n}"
      : "=r"(x), "=r"(y)
      : "f"(e.x), "f"(e.y), "l"(t), "l"(rest));
  return float2_to_bf16x2_bits(__uint_as_float(x | 1u), __uint_as_float(y | 1u));
}

__device__ __forceinline__ uint64_t twice(float x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}

// The block of a slot, and the row within it.
template <int D>
__device__ __forceinline__ uint8_t* slot_row(const Cache& c, int slot, int h, int& row) {
  const int page = slot >> c.page_log, block = (slot & ((1 << c.page_log) - 1)) / kKvBlock;
  row = slot % kKvBlock;
  return c.pool + kv4_block_offset(page, h, c.heads, (1 << c.page_log) / kKvBlock, block, Kv4Block<D>::kBytes);
}

// 32 bytes of one thread: one load of a sector where the address allows it.
template <bool kWide>
__device__ __forceinline__ void load_32(const void* p, uint32_t (&w)[8]) {
  if constexpr (kWide) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// Largest magnitude of 16 bf16, as fp32; NaN if there is one.
__device__ __forceinline__ float amax16(const uint32_t (&w)[8]) {
  uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    uint32_t x = w[j] & 0x7fff7fffu;
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x));
  }
  const float lo = __uint_as_float(m << 16), hi = __uint_as_float(m & 0xffff0000u);
  return lo != lo ? lo : hi != hi ? hi : fmaxf(lo, hi);
}

template <int D, bool kWide>
__global__ void __launch_bounds__(kMaxWarps * 32)
    kv4_append_kernel(Cache c, const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                      long long k_stride, long long v_stride, const int32_t* __restrict__ slots, int tokens,
                      int32_t* status) {
  using L = Kv4Block<D>;
  pdl_wait();
  const Place<D> p;
  if (p.t >= tokens || p.h >= c.heads) return;
  const uint16_t* src = p.kv ? v + (size_t)p.t * v_stride : k + (size_t)p.t * k_stride;
  uint32_t w[8];
  load_32<kWide>(src + (size_t)p.h * D + p.blk * 16, w);   // next to the slot's load, not behind it
  const int slot = slots[p.t];
  if (slot < 0) return;
  if (slot >= c.slots) {
    if (status != nullptr) *status = MOE_ERR_DEVICE;
    return;
  }
  float amax = amax16(w);
  if (amax != amax) {   // a NaN has no code: stored as 0
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if ((w[j] & 0x7fffu) > 0x7f80u) w[j] &= 0xffff0000u;
      if ((w[j] & 0x7fff0000u) > 0x7f800000u) w[j] &= 0xffffu;
    }
    amax = amax16(w);
  }
  const float gs = c.gs[p.kv].x;
  const KvScale scale = kv_scale(amax, gs);
  uint32_t lo = 0, hi = 0;
  if (scale.r > 0.0f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = kv_codes2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u), scale.r);
      if (j < 4) lo |= b << (8 * j);
      else hi |= b << (8 * (j - 4));
    }
  }
  int row;
  uint8_t* blk = slot_row<D>(c, slot, p.h, row) + (p.kv ? L::kValueCodes : 0);
  *reinterpret_cast<uint2*>(blk + row * L::kCodeRow + p.blk * 8) = make_uint2(lo, hi);
  blk[L::kKeyScales + row * L::kScaleRow + p.blk] = (uint8_t)scale.code;
}

template <int D, bool kWide>
__global__ void __launch_bounds__(kMaxWarps * 32)
    kv4_read_kernel(Cache c, const int32_t* __restrict__ slots, int n, uint16_t* k_out, uint16_t* v_out,
                    int32_t* status) {
  using L = Kv4Block<D>;
  pdl_wait();
  const Place<D> p;
  if (p.t >= n || p.h >= c.heads) return;
  uint16_t* out = p.kv ? v_out : k_out;
  if (out == nullptr) return;
  out += ((size_t)p.t * c.heads + p.h) * D + p.blk * 16;
  const int slot = slots[p.t];
  uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (slot >= c.slots) {
    if (status != nullptr) *status = MOE_ERR_DEVICE;
  } else if (slot >= 0) {
    int row;
    const uint8_t* blk = slot_row<D>(c, slot, p.h, row) + (p.kv ? L::kValueCodes : 0);
    const uint2 codes = *reinterpret_cast<const uint2*>(blk + row * L::kCodeRow + p.blk * 8);
    const float s = e4m3_decode(blk[L::kKeyScales + row * L::kScaleRow + p.blk]);
    const float2 inv = c.gs[p.kv];
    const float t = s * inv.x;
    const uint64_t t2 = twice(t), rest2 = twice(fmaf(s, inv.x, -t) + s * inv.y);
    uint32_t a[4], b[4];
    cvt_e2m1x8_f16(codes.x, a);
    cvt_e2m1x8_f16(codes.y, b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] = quotients(a[j], t2, rest2);
      o[4 + j] = quotients(b[j], t2, rest2);
    }
  }
  if constexpr (kWide) {
    stg_v8(out, o);
  } else {
    reinterpret_cast<uint4*>(out)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(out)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

moe_status launch_kv4_append(const moe_kv4_cache& c, const uint16_t* k, const uint16_t* v, long long k_stride,
                             long long v_stride, const int32_t* slots, int tokens, int32_t* status, cudaStream_t s) {
  const bool wide = reinterpret_cast<uintptr_t>(k) % 32 == 0 && reinterpret_cast<uintptr_t>(v) % 32 == 0 &&
                    k_stride % 16 == 0 && v_stride % 16 == 0;
  auto kern = c.head_dim == 64 ? (wide ? kv4_append_kernel<64, true> : kv4_append_kernel<64, false>)
                               : (wide ? kv4_append_kernel<128, true> : kv4_append_kernel<128, false>);
  return launch_cache(kern, c.head_dim, c.kv_heads, tokens, s, cache_of(c, {c.k_gs, 0.0f}, {c.v_gs, 0.0f}), k, v, k_stride,
                      v_stride, slots, tokens, status);
}

moe_status launch_kv4_read(const moe_kv4_cache& c, const int32_t* slots, int n, uint16_t* k_out, uint16_t* v_out,
                           int32_t* status, cudaStream_t s) {
  const bool wide = reinterpret_cast<uintptr_t>(k_out) % 32 == 0 && reinterpret_cast<uintptr_t>(v_out) % 32 == 0;
  auto kern = c.head_dim == 64 ? (wide ? kv4_read_kernel<64, true> : kv4_read_kernel<64, false>)
                               : (wide ? kv4_read_kernel<128, true> : kv4_read_kernel<128, false>);
  return launch_cache(kern, c.head_dim, c.kv_heads, n, s, cache_of(c, reciprocal(c.k_gs), reciprocal(c.v_gs)), slots, n,
                      k_out, v_out, status);
}

}  // namespace moe
