// Norm after a block, its gate, the residual and the norm before the next
// block: n = x rsqrt(mean x^2 + eps) w_post, r = a residual + b gate n, out =
// r rsqrt(mean r^2 + eps) w_pre, one CTA per row, the row in registers
// between the two reductions, so every array is read or written once.
#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

// V neighbouring elements as fp32: one 16-byte load (two for fp32) with V = 8.
template <int V>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&f)[V]) {
  if constexpr (V == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
    f[0] = bf16_bits_to_float(*p);
  }
}

template <int V>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&f)[V]) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(float2_to_bf16x2_bits(f[0], f[1]), float2_to_bf16x2_bits(f[2], f[3]),
                   float2_to_bf16x2_bits(f[4], f[5]), float2_to_bf16x2_bits(f[6], f[7]));
  } else {
    *p = float_to_bf16_bits(f[0]);
  }
}

template <int V, bool F32>
__device__ __forceinline__ void load_res(const void* base, size_t at, float (&f)[V]) {
  if constexpr (!F32) {
    load_bf16<V>(static_cast<const uint16_t*>(base) + at, f);
  } else if constexpr (V == 8) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    f[0] = static_cast<const float*>(base)[at];
  }
}

template <int V, bool F32>
__device__ __forceinline__ void store_res(void* base, size_t at, const float (&f)[V]) {
  if constexpr (!F32) {
    store_bf16<V>(static_cast<uint16_t*>(base) + at, f);
  } else if constexpr (V == 8) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    static_cast<float*>(base)[at] = f[0];
  }
}

// Sum over the CTA, in an order fixed by the thread count.
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

constexpr int kMaxH = 16384;
constexpr int threads_max(int V, int N) { return kMaxH / (V * N) < 1024 ? kMaxH / (V * N) : 1024; }

// V elements per vector, N vectors per thread (thread i takes vectors i, i + threads, ...).
template <int V, int N, bool F32>
__global__ void __launch_bounds__(threads_max(V, N)) block_norm_kernel(moe_block_norm_args a) {
  __shared__ float red[2][32];
  const int vecs = a.H / V;
  const size_t row = blockIdx.x;
  const float inv_h = 1.0f / (float)a.H;
  float x[N][V], r[N][V], g[N][V];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = i * blockDim.x + threadIdx.x;
    if (c < vecs) {
      if (a.x != nullptr) load_bf16<V>(a.x + row * a.x_stride + (size_t)c * V, x[i]);
      load_res<V, F32>(a.residual, row * a.residual_stride + (size_t)c * V, r[i]);
      if (a.gate != nullptr) load_bf16<V>(a.gate + row * a.gate_stride + (size_t)c * V, g[i]);
    }
  }
  float scale = a.branch_scale;
  if (a.x != nullptr && a.w_post != nullptr) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i * blockDim.x + threadIdx.x < vecs) {
#pragma unroll
        for (int j = 0; j < V; ++j) s += x[i][j] * x[i][j];
      }
    scale *= rsqrtf(cta_sum(s, red[0]) * inv_h + a.eps);
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = i * blockDim.x + threadIdx.x;
    if (c < vecs) {
      float w[V];
      if (a.x != nullptr && a.w_post != nullptr) load_bf16<V>(a.w_post + (size_t)c * V, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float v = a.residual_scale * r[i][j];
        if (a.x != nullptr) {
          float n = x[i][j] * scale;
          if (a.w_post != nullptr) n *= w[j] + a.w_offset;
          if (a.gate != nullptr) n *= g[i][j];
          v += n;
        }
        r[i][j] = v;
        s += v * v;
      }
      if (a.residual_out != nullptr) store_res<V, F32>(a.residual_out, row * a.H + (size_t)c * V, r[i]);
    }
  }
  if (a.w_pre == nullptr) return;
  const float inv = rsqrtf(cta_sum(s, red[1]) * inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = i * blockDim.x + threadIdx.x;
    if (c < vecs) {
      float w[V];
      load_bf16<V>(a.w_pre + (size_t)c * V, w);
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = r[i][j] * inv * (w[j] + a.w_offset);
      store_bf16<V>(a.out + row * a.H + (size_t)c * V, w);
    }
  }
}

template <int V, int N>
cudaError_t launch(const moe_block_norm_args& a, cudaStream_t s) {
  const int vecs = (a.H + V - 1) / V;
  const int threads = ((vecs + N - 1) / N + 31) / 32 * 32;
  auto k = a.residual_f32 ? block_norm_kernel<V, N, true> : block_norm_kernel<V, N, false>;
  return launch_ex(false, k, dim3(a.T), dim3(threads), 0, s, a);
}

bool vector_ok(const void* p, long long stride, size_t elem) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (stride * (long long)elem) % 16 == 0;
}

}  // namespace

moe_status launch_block_norm(const moe_block_norm_args& a, cudaStream_t s) {
  const size_t re = a.residual_f32 ? 4 : 2;
  const bool vec = a.H % 8 == 0 && vector_ok(a.x, a.x_stride, 2) && vector_ok(a.gate, a.gate_stride, 2) &&
                   vector_ok(a.residual, a.residual_stride, re) && vector_ok(a.residual_out, a.H, re) &&
                   vector_ok(a.out, a.H, 2) && vector_ok(a.w_post, 0, 2) && vector_ok(a.w_pre, 0, 2);
  cudaError_t e;
  if (!vec) {
    e = a.H <= 4096 ? launch<1, 4>(a, s) : launch<1, 16>(a, s);
  } else if (a.H <= 8192 && a.T <= 304) {
    e = launch<8, 1>(a, s);   // few rows: as many threads per row as it has vectors
  } else {
    e = launch<8, 4>(a, s);
  }
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

}  // namespace moe
