// Norm after a block, its gate, the residual and the norm before the next
// block: n = x rsqrt(mean x^2 + eps) w_post, r = a residual + b gate n, out =
// r rsqrt(mean r^2 + eps) w_pre, the row in registers between the two
// reductions, so every array is read or written once.
//
// What bounds it: bytes. Few rows run one CTA each (8 x 4096: 2.3 us, launch
// and one trip to memory), more rows than CTAs the stream kernel: 16384 x 7168
// with a gate per row in 192 us, 6.1 TB/s or 90 % of the measured copy rate. One CTA
// per row took 303 us there: its loads stop while its reductions run, and
// with scalar arithmetic the instructions alone (370 per warp and 256
// elements, now 150) took 240.
#include "kernels.cuh"
#include "kv4.cuh"
#include "tc_ptx.cuh"

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
constexpr int kStages = 2;                      // rows a CTA of the stream kernel holds or fetches
constexpr size_t kStreamSmem = 226 * 1024;      // of an SM's CTAs, 1 KiB each for the reductions
constexpr int threads_max(int V, int N) { return kMaxH / (V * N) < 1024 ? kMaxH / (V * N) : 1024; }

// V elements per vector, N vectors per thread (thread i takes vectors i, i + threads, ...).
template <int V, int N, bool F32>
__global__ void __launch_bounds__(threads_max(V, N)) block_norm_kernel(moe_block_norm_args a) {
  __shared__ float red[2][32];
  pdl_wait();
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

// Two fp32 at a time: bf16 pairs and the packed arithmetic of sm_100 on.
struct Pair {
  float x, y;
};
__device__ __forceinline__ unsigned long long bits(Pair p) {
  unsigned long long v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(p.x), "f"(p.y));
  return v;
}
__device__ __forceinline__ Pair pair(unsigned long long v) {
  Pair p;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(p.x), "=f"(p.y) : "l"(v));
  return p;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair(d);
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair(d);
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair(d);
}
__device__ __forceinline__ Pair bf16_pair(uint32_t w) { return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)}; }

struct Vec {   // eight bf16, or four fp32
  uint32_t w[4];
};
__device__ __forceinline__ Vec vec16(const void* p, int at) {
  const uint4 v = static_cast<const uint4*>(p)[at];
  return {v.x, v.y, v.z, v.w};
}

// Many rows: persistent CTAs whose threads copy their own vectors of the rows
// to come into shared memory (16-byte asynchronous copies, kStages rows deep),
// so memory is busy through both reductions of a row. A thread reads only
// what it copied: no barrier but the reductions'. The weights come from L1
// for each row, asked for before the reduction in front of them: held in
// registers they and the row do not fit 64.
template <int N, bool F32>
__global__ void __launch_bounds__(512, 2) block_norm_stream_kernel(moe_block_norm_args a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][32];
  constexpr int kRes = F32 ? 2 : 1;                 // 16-byte pieces of a residual vector
  const int vecs = a.H / 8, threads = blockDim.x, tid = threadIdx.x;
  const bool has_x = a.x != nullptr, post = has_x && a.w_post != nullptr, pre = a.w_pre != nullptr;
  const bool gated = has_x && a.gate != nullptr, gate_rows = gated && a.gate_stride != 0;
  const int piece = vecs * 16, stage = piece * (has_x + kRes + gate_rows);   // bytes
  const int res_at = has_x ? piece : 0, gate_at = res_at + kRes * piece;
  pdl_wait();
  const float inv_h = 1.0f / (float)a.H;
  const Pair offset{a.w_offset, a.w_offset}, keep{a.residual_scale, a.residual_scale};
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  auto fetch = [&](long long row, int slot) {
    if (row < a.T) {
      const uint32_t at = base + slot * stage;
      const uint16_t* x = a.x + row * a.x_stride;
      const uint16_t* g = a.gate + row * a.gate_stride;
      const uint8_t* r = static_cast<const uint8_t*>(a.residual) + row * a.residual_stride * (F32 ? 4 : 2);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * threads + tid;
        if (c < vecs) {
          if (has_x) tc::cp_async_16(at + c * 16, x + c * 8, 16);
#pragma unroll
          for (int k = 0; k < kRes; ++k) tc::cp_async_16(at + res_at + k * piece + c * 16, r + (c * kRes + k) * 16, 16);
          if (gate_rows) tc::cp_async_16(at + gate_at + c * 16, g + c * 8, 16);
        }
      }
    }
    tc::cp_async_commit();
  };
  for (int s = 0; s < kStages; ++s) fetch(blockIdx.x + (long long)s * gridDim.x, s);
  int slot = 0;
  for (long long row = blockIdx.x; row < a.T; row += gridDim.x) {
    tc::cp_async_wait<kStages - 1>();
    const uint8_t* at = ring + slot * stage;
    Vec w[N];
    Pair r[N][4];
    float scale = a.branch_scale;
    if (post) {
      Pair s{0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * threads + tid;
        if (c < vecs) {
          w[i] = vec16(a.w_post, c);
          const Vec x = vec16(at, c);
#pragma unroll
          for (int j = 0; j < 4; ++j) s = fma2(bf16_pair(x.w[j]), bf16_pair(x.w[j]), s);
        }
      }
      scale *= rsqrtf(cta_sum(s.x + s.y, red[0]) * inv_h + a.eps);
    }
    Pair s{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = i * threads + tid;
      if (c < vecs) {
        Vec q = vec16(at + res_at, c);
        if constexpr (F32) {
          const Vec q1 = vec16(at + res_at, vecs + c);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            r[i][j] = mul2(keep, {__uint_as_float(q.w[2 * j]), __uint_as_float(q.w[2 * j + 1])});
            r[i][2 + j] = mul2(keep, {__uint_as_float(q1.w[2 * j]), __uint_as_float(q1.w[2 * j + 1])});
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) r[i][j] = mul2(keep, bf16_pair(q.w[j]));
        }
        if (has_x) {
          Pair n[4];
          const Vec x = vec16(at, c);
#pragma unroll
          for (int j = 0; j < 4; ++j) n[j] = mul2(bf16_pair(x.w[j]), {scale, scale});
          if (post) {
#pragma unroll
            for (int j = 0; j < 4; ++j) n[j] = mul2(n[j], add2(bf16_pair(w[i].w[j]), offset));
          }
          if (gated) {
            const Vec g = gate_rows ? vec16(at + gate_at, c) : vec16(a.gate, c);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[i][j] = fma2(n[j], bf16_pair(g.w[j]), r[i][j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) r[i][j] = add2(n[j], r[i][j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s = fma2(r[i][j], r[i][j], s);
        if (a.residual_out != nullptr) {
          const float v[8] = {r[i][0].x, r[i][0].y, r[i][1].x, r[i][1].y, r[i][2].x, r[i][2].y, r[i][3].x, r[i][3].y};
          store_res<8, F32>(a.residual_out, row * a.H + (size_t)c * 8, v);
        }
        if (pre) w[i] = vec16(a.w_pre, c);
      }
    }
    fetch(row + (long long)kStages * gridDim.x, slot);   // this thread has read its part of the slot
    slot = slot + 1 == kStages ? 0 : slot + 1;
    if (pre) {
      const float inv = rsqrtf(cta_sum(s.x + s.y, red[1]) * inv_h + a.eps);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * threads + tid;
        if (c < vecs) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const Pair y = mul2(mul2(r[i][j], {inv, inv}), add2(bf16_pair(w[i].w[j]), offset));
            v[2 * j] = y.x, v[2 * j + 1] = y.y;
          }
          store_bf16<8>(a.out + row * a.H + (size_t)c * 8, v);
        }
      }
    }
    if (!(post && pre)) __syncthreads();   // one reduction a row: its buffer is read by all before the next
  }
}

// Rows that are not whole vectors at 16-byte addresses (odd H, offset or odd
// strided views): the stream kernel with every array's aligned 16-byte
// granules copied to shared memory as they lie, read there at any offset, and
// the outputs packed there before they go out as granules. 16384 x 5003 with a
// gate per row takes 252 us, 616 an element at a time (128 as whole vectors:
// the rest is five barriers a row and twice the shared-memory reads).
__device__ __forceinline__ Vec load_at(const uint8_t* smem, int off) {   // 16 bytes at an even offset
  const uint4* p = reinterpret_cast<const uint4*>(smem) + (off >> 4);
  const uint4 a = p[0], b = p[1];
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (off & 8) {
#pragma unroll
    for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
  }
  if (off & 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
  }
  return {w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ int lead_of(const void* p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15); }

// The granules that hold `bytes` bytes at src. One that reaches past an end of
// the array (`first`: src is its start, `last`: src + bytes its end) is copied
// element by element; elsewhere its other bytes lie between rows.
__device__ __forceinline__ void fetch_bytes(uint8_t* dst, const uint8_t* src, int bytes, bool first, bool last) {
  const int lead = lead_of(src), n = (lead + bytes + 15) >> 4;
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    const int at = 16 * c - lead;   // in the row
    if ((at >= 0 || !first) && (at + 16 <= bytes || !last)) {
      tc::cp_async_16(static_cast<uint32_t>(__cvta_generic_to_shared(dst + 16 * c)), src + at, 16);
    } else {
      for (int e = 0; e < 16; e += 2)
        if (at + e >= 0 && at + e < bytes)
          *reinterpret_cast<uint16_t*>(dst + 16 * c + e) = *reinterpret_cast<const uint16_t*>(src + at + e);
    }
  }
}

// `bytes` bytes from packed + 16 on to dst, as granules but for the ends.
__device__ __forceinline__ void store_bytes(uint8_t* dst, const uint8_t* packed, int bytes) {
  const int lead = lead_of(dst), n = (lead + bytes + 15) >> 4;
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    const int at = 16 * c - lead;
    const Vec v = load_at(packed, 16 + at);
    if (at >= 0 && at + 16 <= bytes) {
      *reinterpret_cast<uint4*>(dst + at) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; e += 2)
        if (at + e >= 0 && at + e < bytes)
          *reinterpret_cast<uint16_t*>(dst + at + e) = (uint16_t)(v.w[e / 4] >> (e % 4 * 8));
    }
  }
}

// Vector c of a weight of H elements, zeros past its end.
__device__ __forceinline__ Vec weight_at(const uint16_t* p, int c, int H) {
  if (8 * c + 8 <= H && lead_of(p) == 0) return vec16(p, c);
  Vec v = {{0u, 0u, 0u, 0u}};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (8 * c + e < H) v.w[e / 2] |= (uint32_t)p[8 * c + e] << (e % 2 * 16);
  return v;
}

template <int N, bool F32>
__global__ void __launch_bounds__(512, 2) block_norm_shift_kernel(moe_block_norm_args a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][32];
  constexpr int kElem = F32 ? 4 : 2;
  pdl_wait();
  const int H = a.H, vecs = (H + 7) / 8, threads = blockDim.x, tid = threadIdx.x;
  const bool has_x = a.x != nullptr, post = has_x && a.w_post != nullptr, pre = a.w_pre != nullptr;
  const bool gated = has_x && a.gate != nullptr, gate_rows = gated && a.gate_stride != 0;
  // a row's granules, one more for its offset and one that load_at() touches
  const int piece = (vecs + 2) * 16, res_piece = (vecs * (F32 ? 2 : 1) + 2) * 16;
  const int res_at = has_x ? piece : 0, gate_at = res_at + res_piece, stage = gate_at + (gate_rows ? piece : 0);
  uint8_t* const packed = ring + kStages * stage;   // r on its way out, then y
  const float inv_h = 1.0f / (float)H;
  const Pair offset{a.w_offset, a.w_offset}, keep{a.residual_scale, a.residual_scale};
  auto x_row = [&](long long row) { return reinterpret_cast<const uint8_t*>(a.x + row * a.x_stride); };
  auto g_row = [&](long long row) { return reinterpret_cast<const uint8_t*>(a.gate + row * a.gate_stride); };
  auto r_row = [&](long long row) { return static_cast<const uint8_t*>(a.residual) + row * a.residual_stride * kElem; };
  auto fetch = [&](long long row, int slot) {
    if (row < a.T) {
      uint8_t* at = ring + slot * stage;
      const bool first = row == 0, last = row == a.T - 1;
      if (has_x) fetch_bytes(at, x_row(row), 2 * H, first, last);
      fetch_bytes(at + res_at, r_row(row), kElem * H, first, last);
      if (gate_rows) fetch_bytes(at + gate_at, g_row(row), 2 * H, first, last);
    }
    tc::cp_async_commit();
  };
  for (int s = 0; s < kStages; ++s) fetch(blockIdx.x + (long long)s * gridDim.x, s);
  int slot = 0;
  for (long long row = blockIdx.x; row < a.T; row += gridDim.x) {
    tc::cp_async_wait<kStages - 1>();
    __syncthreads();   // a vector's granules are copies of two threads
    const uint8_t* at = ring + slot * stage;
    const int x_lead = lead_of(x_row(row)), r_lead = lead_of(r_row(row)), g_lead = lead_of(g_row(row));
    // the row's last vector may go on into what lies behind it
    auto tail = [&](int c, int j, Pair v) {
      return Pair{8 * c + 2 * j < H ? v.x : 0.0f, 8 * c + 2 * j + 1 < H ? v.y : 0.0f};
    };
    Pair r[N][4];
    float scale = a.branch_scale;
    if (post) {
      Pair s{0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * threads + tid;
        if (c < vecs) {
          const Vec x = load_at(at, 16 * c + x_lead);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const Pair v = tail(c, j, bf16_pair(x.w[j]));
            s = fma2(v, v, s);
          }
        }
      }
      scale *= rsqrtf(cta_sum(s.x + s.y, red[0]) * inv_h + a.eps);
    }
    Pair s{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = i * threads + tid;
      if (c < vecs) {
        if constexpr (F32) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const Vec q = load_at(at + res_at, 32 * c + 16 * k + r_lead);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              r[i][2 * k + j] = mul2(keep, {__uint_as_float(q.w[2 * j]), __uint_as_float(q.w[2 * j + 1])});
          }
        } else {
          const Vec q = load_at(at + res_at, 16 * c + r_lead);
#pragma unroll
          for (int j = 0; j < 4; ++j) r[i][j] = mul2(keep, bf16_pair(q.w[j]));
        }
        if (has_x) {
          Pair n[4];
          const Vec x = load_at(at, 16 * c + x_lead);
#pragma unroll
          for (int j = 0; j < 4; ++j) n[j] = mul2(bf16_pair(x.w[j]), {scale, scale});
          if (post) {
            const Vec w = weight_at(a.w_post, c, H);
#pragma unroll
            for (int j = 0; j < 4; ++j) n[j] = mul2(n[j], add2(bf16_pair(w.w[j]), offset));
          }
          if (gated) {
            const Vec g = gate_rows ? load_at(at + gate_at, 16 * c + g_lead) : weight_at(a.gate, c, H);
#pragma unroll
            for (int j = 0; j < 4; ++j) r[i][j] = fma2(n[j], bf16_pair(g.w[j]), r[i][j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) r[i][j] = add2(n[j], r[i][j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          r[i][j] = tail(c, j, r[i][j]);
          s = fma2(r[i][j], r[i][j], s);
        }
        const float v[8] = {r[i][0].x, r[i][0].y, r[i][1].x, r[i][1].y, r[i][2].x, r[i][2].y, r[i][3].x, r[i][3].y};
        store_res<8, F32>(packed + 16, (size_t)c * 8, v);
      }
    }
    const float sum = cta_sum(s.x + s.y, red[1]);   // and all have read the slot and written their part of r
    fetch(row + (long long)kStages * gridDim.x, slot);
    slot = slot + 1 == kStages ? 0 : slot + 1;
    if (a.residual_out != nullptr)
      store_bytes(static_cast<uint8_t*>(a.residual_out) + row * H * kElem, packed, kElem * H);
    if (pre) {
      __syncthreads();
      const float inv = rsqrtf(sum * inv_h + a.eps);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = i * threads + tid;
        if (c < vecs) {
          const Vec w = weight_at(a.w_pre, c, H);
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const Pair y = mul2(mul2(r[i][j], {inv, inv}), add2(bf16_pair(w.w[j]), offset));
            v[2 * j] = y.x, v[2 * j + 1] = y.y;
          }
          store_bf16<8>(reinterpret_cast<uint16_t*>(packed + 16) + c * 8, v);
        }
      }
      __syncthreads();
      store_bytes(reinterpret_cast<uint8_t*>(a.out + row * H), packed, 2 * H);
    }
  }
}

// Some 1024 threads an SM, in CTAs of a row each: at 64 registers more would
// not fit, and two rows a CTA keep 64 KiB or more in flight at every H.
struct Stream {
  int n, threads, per_sm;
  size_t smem;
};
Stream plan_stream(const moe_block_norm_args& a, bool shift) {
  Stream p;
  const size_t vecs = (a.H + 7) / 8, more = shift ? 2 : 0;   // granules of an array
  const size_t x = a.x ? vecs + more : 0, res = vecs * (a.residual_f32 ? 2 : 1) + more,
               gate = a.gate && a.gate_stride ? vecs + more : 0;
  p.n = a.H <= 4096 ? 1 : 2;
  p.threads = (int)((vecs + p.n - 1) / p.n + 31) / 32 * 32;
  p.smem = 16 * (kStages * (x + res + gate) + (shift ? res : 0));
  p.per_sm = 1024 / p.threads < 8 ? 1024 / p.threads : 8;
  const int fit = (int)(kStreamSmem / (p.smem + 1024));
  if (shift && p.per_sm > fit) p.per_sm = fit;
  if (a.H > 8192 || fit < p.per_sm) p.per_sm = 0;
  return p;
}

template <class K>
cudaError_t launch_stream(K k, const moe_block_norm_args& a, const Stream& p, std::atomic<unsigned long long>& done,
                          cudaStream_t s) {
  cudaError_t e = opt_in_smem(k, kStreamSmem, done);
  if (e != cudaSuccess) return e;
  const int ctas = p.per_sm * sm_count();
  return launch_ex(true, k, dim3(a.T < ctas ? a.T : ctas), dim3(p.threads), p.smem, s, a);
}

template <int N>
cudaError_t launch_vectors(const moe_block_norm_args& a, const Stream& p, cudaStream_t s) {
  static std::atomic<unsigned long long> done[2];
  return a.residual_f32 ? launch_stream(block_norm_stream_kernel<N, true>, a, p, done[1], s)
                        : launch_stream(block_norm_stream_kernel<N, false>, a, p, done[0], s);
}

template <int N>
cudaError_t launch_shift(const moe_block_norm_args& a, const Stream& p, cudaStream_t s) {
  static std::atomic<unsigned long long> done[2];
  return a.residual_f32 ? launch_stream(block_norm_shift_kernel<N, true>, a, p, done[1], s)
                        : launch_stream(block_norm_shift_kernel<N, false>, a, p, done[0], s);
}

template <int V, int N>
cudaError_t launch(const moe_block_norm_args& a, cudaStream_t s) {
  const int vecs = (a.H + V - 1) / V;
  const int threads = ((vecs + N - 1) / N + 31) / 32 * 32;
  auto k = a.residual_f32 ? block_norm_kernel<V, N, true> : block_norm_kernel<V, N, false>;
  return launch_ex(true, k, dim3(a.T), dim3(threads), 0, s, a);
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
  const Stream p = plan_stream(a, !vec);
  // Whole vectors: a CTA per row and a thread per vector as long as all rows
  // run at once, which is one row an SM from H = 5120 on, and as many as the
  // stream kernel has CTAs below; with more rows the stream kernel. (us, row by
  // row / streamed: 152 x 8192 3.1 / 3.1, 160 x 8192 5.0 / 4.1, 304 x 7168 5.0 /
  // 4.0, 304 x 5120 3.2 / 3.3, 304 x 4096 2.9 / 3.2, 1200 x 4096 8.8 / 7.9, 600 x
  // 2048 2.8 / 3.1, 2400 x 2048 7.9 / 7.6.) Four vectors a thread are slower
  // than one up to there (8 x 4096 3.4 and 2.2, 400 x 2048 3.6 and 2.5, 1200 x
  // 1024 3.8 and 2.8) and are left for more rows than run at once where the
  // stream kernel does not fit.
  const int at_once = (a.H > 5120 ? 1 : p.per_sm > 0 ? p.per_sm : 2) * sm_count();
  cudaError_t e;
  if (!vec) {
    // Short rows an element at a time (16384 x 333: 24 us, 33 by granules;
    // x 1001: 68 and 52).
    if (a.H <= 512) e = launch<1, 4>(a, s);
    else if (p.per_sm > 0) e = p.n == 1 ? launch_shift<1>(a, p, s) : launch_shift<2>(a, p, s);
    else e = launch<1, 16>(a, s);
  } else if (p.per_sm > 0 && a.T > at_once) {
    e = p.n == 1 ? launch_vectors<1>(a, p, s) : launch_vectors<2>(a, p, s);
  } else if (a.H <= 8192 && a.T <= at_once) {
    e = launch<8, 1>(a, s);   // as many threads per row as it has vectors
  } else {
    e = launch<8, 4>(a, s);
  }
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

}  // namespace moe
