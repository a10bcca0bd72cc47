// Arithmetic that the attention kernels have in common, few rows and many, so
// that they round alike.
#pragma once

#include "common.cuh"

namespace moe {
namespace kv {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// log2: m is set this far below the running maximum, and again when a score is
// further above it than the slack.
constexpr float kLead = 7.0f, kSlack = 15.0f;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^k for -126 <= k <= 127.
__device__ __forceinline__ float pow2(int k) { return __int_as_float((127 + k) << 23); }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace kv
}  // namespace moe
