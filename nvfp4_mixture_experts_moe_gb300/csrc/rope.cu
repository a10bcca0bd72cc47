// Rotary positions of queries and keys, in place or on the way into the cache.
//
// Mathematics. Pair p of a token turns by pos * inv_freq_p. In turns the angle
// is the fraction of pos * (inv_freq_p / 2 pi), so with the factor as a 64-bit
// fixed-point fraction a product modulo 2^64 is that fraction to 2^-62 turns
// per position, whatever the position. It is reduced to the nearest quarter
// turn exactly, and sine and cosine of the rest (at most pi / 4) are Taylor
// polynomials in fp32, whose terms end below 2^-28.
//
// A thread has eight pairs of a token for as many heads as it is given: their
// sines and cosines (some 30 instructions a pair) are worked out once.
//
// What bounds it: bytes where there are many tokens (16384 of 32 + 8 heads x
// 128: 52.7 us, 6.4 TB/s of the 6.7 that a copy reaches), the launch where there
// are few (8 tokens: 2.3 us). Rows that vectors cannot move (rotary_dim no
// multiple of 16, or not 16-byte aligned) go a pair a thread in 2-byte accesses,
// at half of that rate (4096 tokens of 40 heads x 72: 15.0 us, 3.1 TB/s; x 128, 40
// elements turned or at an odd address: 25.5, 3.3; in vectors 14.2, 5.9). On the way into the cache (8191 tokens of 32
// query heads, 8 key/value heads x 128, adjacent pairs: 35 us, 26 by the
// bytes) a load's latency: three kinds of rows leave 24 warps an SM.
#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Heads whose rows a thread has asked for, of a rotation and of an append (1,
// 2, 3, 4 of the case above, with the read that follows it: 48.8, 44.2, 45.0, 54 us).
constexpr int kAhead = 4, kAppendAhead = 2;

// (cos, sin) of a pair's angle, times the plan's scale.
__device__ __forceinline__ float2 rotation(uint64_t turns, int pos, float scale) {
  const uint64_t frac = (turns & ~3ull) * (uint64_t)(int64_t)pos;
  const uint64_t quarter = (frac + (1ull << 61)) >> 62;
  const int rest = (int)((int64_t)(frac - (quarter << 62)) >> 30);        // in 2^-34 turns, [-2^31, 2^31)
  const float r = (float)rest * 3.6572952e-10f, x = r * r;               // 2 pi / 2^34
  const float s = fmaf(r * x, fmaf(x, fmaf(x, fmaf(x, 1.0f / 362880.0f, -1.0f / 5040.0f), 1.0f / 120.0f), -1.0f / 6.0f), r);
  const float c = fmaf(x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, -1.0f / 3628800.0f, 1.0f / 40320.0f), -1.0f / 720.0f),
                                       1.0f / 24.0f), -0.5f), 1.0f);
  const bool swap = quarter & 1, neg_c = (quarter + 1) & 2, neg_s = quarter & 2;
  const float cq = swap ? s : c, sq = swap ? c : s;
  return make_float2(scale * (neg_c ? -cq : cq), scale * (neg_s ? -sq : sq));
}

__device__ __forceinline__ float2 rotation_of(const moe_rope_plan& plan, int pair, const int32_t* positions, int tokens, int t) {
  const uint64_t turns = __ldg(reinterpret_cast<const unsigned long long*>(plan.turns) + pair);
  const int axis = min((int)(turns & 3), plan.axes - 1);
  return rotation(turns, __ldg(positions + (size_t)axis * tokens + t), plan.scale);
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(float2_to_bf16x2_bits(x[0], x[1]), float2_to_bf16x2_bits(x[2], x[3]),
                    float2_to_bf16x2_bits(x[4], x[5]), float2_to_bf16x2_bits(x[6], x[7]));
}

__device__ __forceinline__ void turn(float2 cs, float& a, float& b) {
  const float x = a;
  a = fmaf(x, cs.x, -b * cs.y);
  b = fmaf(x, cs.y, b * cs.x);
}

// Eight pairs: x and y are the first and second elements (halves), or sixteen
// neighbouring elements (adjacent).
__device__ __forceinline__ void turn8(const float2 (&cs)[8], bool adjacent, float (&x)[8], float (&y)[8]) {
  if (adjacent) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn(cs[i], x[2 * i], x[2 * i + 1]);
      turn(cs[4 + i], y[2 * i], y[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(cs[i], x[i], y[i]);
  }
}

// A thread's two runs of eight elements. One sector (kWide: 32-byte aligned,
// the second run behind the first) in one load or store: halves of it in two
// are two trips for the same bytes.
__device__ __forceinline__ void load_runs(const uint16_t* p, int lo, int hi, bool wide, uint4 (&w)[2]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0].x), "=r"(w[0].y), "=r"(w[0].z), "=r"(w[0].w), "=r"(w[1].x), "=r"(w[1].y), "=r"(w[1].z),
                   "=r"(w[1].w)
                 : "l"(p + lo));
  } else {
    w[0] = *reinterpret_cast<const uint4*>(p + lo);
    w[1] = *reinterpret_cast<const uint4*>(p + hi);
  }
}

__device__ __forceinline__ void store_runs(uint16_t* p, int lo, int hi, bool wide, const uint4 (&w)[2]) {
  if (wide) {
    const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
    stg_v8(p + lo, v);
  } else {
    *reinterpret_cast<uint4*>(p + lo) = w[0];
    *reinterpret_cast<uint4*>(p + hi) = w[1];
  }
}

struct RopeRows {
  moe_rope_args a;
  int splits, units, turning;   // threads of a token and unit; units of a head, the first `turning` of them with pairs
};

// Rows of 16-byte alignment, rotary_dim a multiple of 16: a unit is eight pairs
// or sixteen elements to copy, two 16-byte loads and stores a head (kWide: one of 32).
template <bool kWide>
__global__ void __launch_bounds__(kThreads) rope_vector_kernel(const __grid_constant__ RopeRows p) {
  const moe_rope_args& a = p.a;
  pdl_wait();
  const unsigned idx = blockIdx.x * kThreads + threadIdx.x;
  const int u = idx % p.units;
  const unsigned rest = idx / p.units;
  const int first = rest % p.splits, t = rest / p.splits;
  if (t >= a.tokens) return;
  const int R = a.plan.rotary_dim, heads = a.q_heads + a.k_heads;
  const bool turns = u < p.turning;
  int lo, hi;   // the unit's two runs of eight elements
  float2 cs[8];
  if (turns) {
    lo = a.plan.adjacent ? 16 * u : 8 * u;
    hi = a.plan.adjacent ? lo + 8 : lo + R / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = rotation_of(a.plan, 8 * u + i, a.positions, a.tokens, t);
      if (a.inverse) cs[i].y = -cs[i].y;
    }
  } else {
    lo = R + 16 * (u - p.turning);
    hi = lo + 8;
  }
  const bool second = hi < a.head_dim;
  const uint16_t* const q = a.q + (size_t)t * a.q_stride;
  const uint16_t* const k = a.k + (size_t)t * a.k_stride;
  uint16_t* const qo = a.q_out + (size_t)t * a.q_out_stride;
  uint16_t* const ko = a.k_out + (size_t)t * a.k_out_stride;
  for (int h0 = first; h0 < heads; h0 += kAhead * p.splits) {
    uint4 w[kAhead][2];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = h0 + j * p.splits;
      if (h >= heads) break;
      const uint16_t* src = h < a.q_heads ? q + (size_t)h * a.head_dim : k + (size_t)(h - a.q_heads) * a.head_dim;
      if (second) load_runs(src, lo, hi, kWide, w[j]);
      else w[j][0] = *reinterpret_cast<const uint4*>(src + lo);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = h0 + j * p.splits;
      if (h >= heads) break;
      uint16_t* dst = h < a.q_heads ? qo + (size_t)h * a.head_dim : ko + (size_t)(h - a.q_heads) * a.head_dim;
      if (turns) {
        float x[8], y[8];
        unpack8(w[j][0], x);
        unpack8(w[j][1], y);
        turn8(cs, a.plan.adjacent, x, y);
        w[j][0] = pack8(x);
        w[j][1] = pack8(y);
      }
      if (second) store_runs(dst, lo, hi, kWide, w[j]);
      else *reinterpret_cast<uint4*>(dst + lo) = w[j][0];
    }
  }
}

// Any alignment and even rotary_dim: a unit is one pair or two elements to copy.
__global__ void __launch_bounds__(kThreads) rope_pair_kernel(const __grid_constant__ RopeRows p) {
  const moe_rope_args& a = p.a;
  pdl_wait();
  const unsigned idx = blockIdx.x * kThreads + threadIdx.x;
  const int u = idx % p.units;
  const unsigned rest = idx / p.units;
  const int first = rest % p.splits, t = rest / p.splits;
  if (t >= a.tokens) return;
  const int R = a.plan.rotary_dim, heads = a.q_heads + a.k_heads;
  const bool turns = u < p.turning;
  const int lo = !turns ? R + 2 * (u - p.turning) : a.plan.adjacent ? 2 * u : u;
  const int hi = turns && !a.plan.adjacent ? u + R / 2 : lo + 1;
  const bool second = hi < a.head_dim;
  float2 cs = make_float2(1.0f, 0.0f);
  if (turns) {
    cs = rotation_of(a.plan, u, a.positions, a.tokens, t);
    if (a.inverse) cs.y = -cs.y;
  }
  for (int h = first; h < heads; h += p.splits) {
    const bool is_q = h < a.q_heads;
    const uint16_t* src = is_q ? a.q + (size_t)t * a.q_stride + (size_t)h * a.head_dim
                               : a.k + (size_t)t * a.k_stride + (size_t)(h - a.q_heads) * a.head_dim;
    uint16_t* dst = is_q ? a.q_out + (size_t)t * a.q_out_stride + (size_t)h * a.head_dim
                         : a.k_out + (size_t)t * a.k_out_stride + (size_t)(h - a.q_heads) * a.head_dim;
    uint16_t x = src[lo], y = second ? src[hi] : (uint16_t)0;
    if (turns) {
      float fx = bf16_bits_to_float(x), fy = bf16_bits_to_float(y);
      turn(cs, fx, fy);
      x = float_to_bf16_bits(fx);
      y = float_to_bf16_bits(fy);
    }
    dst[lo] = x;
    if (second) dst[hi] = y;
  }
}

// ------------------------------------------------ on the way into the cache

struct AppendRope {
  moe_kv4_append_rope_args a;
  int splits;     // warps of a run of tokens
  int page_log;
  bool wide_in, wide_out;   // rows are 32-byte aligned; and queries' runs neighbours
};

// Largest magnitude of eight values; NaN if there is one.
__device__ __forceinline__ float amax8(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x[i])));
  return m;
}

__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float r) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= kv_codes2(x[2 * i], x[2 * i + 1], r) << (8 * i);
  return r > 0.0f ? w : 0u;
}

__device__ __forceinline__ void no_nan(float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (x[i] != x[i]) x[i] = 0.0f;
}

// A CTA has 512 / D consecutive tokens, whose sines and cosines it works out
// once; a warp (a lane: sixteen elements of a token) takes every splits-th of
// their rows: query heads, key heads, value heads.
template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_rope_kernel(const __grid_constant__ AppendRope p) {
  using L = Kv4Block<D>;
  constexpr int kUnits = D / 16, kTokens = 32 / kUnits;
  __shared__ alignas(16) float2 table[kTokens][D / 2];
  const moe_kv4_append_rope_args& a = p.a;
  pdl_wait();
  const int lane = threadIdx.x & 31, u = lane % kUnits, first = blockIdx.y * (blockDim.x / 32) + (threadIdx.x >> 5);
  const int t0 = blockIdx.x * kTokens, R = a.plan.rotary_dim, Hq = a.q_heads, Hk = a.cache.kv_heads;
  for (int i = threadIdx.x; i < kTokens * (R / 2); i += blockDim.x) {
    const int token = i / (R / 2), pair = i - token * (R / 2);
    table[token][pair] = rotation_of(a.plan, pair, a.positions, a.tokens, min(t0 + token, a.tokens - 1));
  }
  const bool real = t0 + lane / kUnits < a.tokens;
  const int t = real ? t0 + lane / kUnits : a.tokens - 1;   // lanes past the end follow, and store nothing
  const bool turns = u < R / 16;
  const int lo = turns && !a.plan.adjacent ? 8 * u : 16 * u, hi = turns && !a.plan.adjacent ? lo + R / 2 : lo + 8;
  const int slot = real ? __ldg(a.slots + t) : -1;
  const long long limit = (long long)a.cache.num_pages << p.page_log;
  const bool keep = slot >= 0 && slot < limit;
  if (slot >= limit && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
  __syncthreads();
  float2 cs[8];
  if (turns)
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float4 two = *reinterpret_cast<const float4*>(&table[lane / kUnits][8 * u + i]);
      cs[i] = make_float2(two.x, two.y);
      cs[i + 1] = make_float2(two.z, two.w);
    }
  const int row = slot % kKvBlock;
  uint8_t* const pool = static_cast<uint8_t*>(a.cache.pool);
  auto block_of = [&](int h) {
    return pool + kv4_block_offset(slot >> p.page_log, h, Hk, (1 << p.page_log) / kKvBlock,
                                   (slot & ((1 << p.page_log) - 1)) / kKvBlock, L::kBytes);
  };
  const int rows = Hq + 2 * Hk;
  const uint16_t *const q = a.q + (size_t)t * a.q_stride, *const k = a.k + (size_t)t * a.k_stride,
                 *const v = a.v + (size_t)t * a.v_stride;
  for (int r0 = first; r0 < rows; r0 += kAppendAhead * p.splits) {
    uint4 w[kAppendAhead][2];
#pragma unroll
    for (int i = 0; i < kAppendAhead; ++i) {
      const int r = r0 + i * p.splits;
      if (r >= rows) break;
      const uint16_t* src = r < Hq ? q + r * D : r < Hq + Hk ? k + (r - Hq) * D : v + (r - Hq - Hk) * D;
      const bool value = r >= Hq + Hk;
      load_runs(src, value ? 16 * u : lo, value ? 16 * u + 8 : hi, p.wide_in && (value || a.plan.adjacent), w[i]);
    }
#pragma unroll
    for (int i = 0; i < kAppendAhead; ++i) {
      const int r = r0 + i * p.splits;
      if (r >= rows) break;
      float x[8], y[8];
      if (r < Hq) {
        if (turns) {
          unpack8(w[i][0], x);
          unpack8(w[i][1], y);
          turn8(cs, a.plan.adjacent, x, y);
          w[i][0] = pack8(x);
          w[i][1] = pack8(y);
        }
        if (real) {
          uint16_t* dst = a.q_out + (size_t)t * a.q_out_stride + r * D;
          store_runs(dst, lo, hi, p.wide_out, w[i]);
        }
        continue;
      }
      const bool key = r < Hq + Hk;
      const int h = r - Hq - (key ? 0 : Hk), at0 = key ? lo : 16 * u, at1 = key ? hi : 16 * u + 8;
      unpack8(w[i][0], x);
      unpack8(w[i][1], y);
      if (key && turns) turn8(cs, a.plan.adjacent, x, y);
      const float gs = key ? a.cache.k_gs : a.cache.v_gs;
      float mx = amax8(x), my = amax8(y);
      if (mx != mx || my != my) {   // a NaN has no code: stored as 0
        no_nan(x);
        no_nan(y);
        mx = amax8(x);
        my = amax8(y);
      }
      // Halves: two neighbouring lanes have the two runs of a group of sixteen.
      const float ox = __shfl_xor_sync(0xffffffffu, mx, 1), oy = __shfl_xor_sync(0xffffffffu, my, 1);
      const bool split = key && turns && !a.plan.adjacent;
      if (split) {
        mx = fmaxf(mx, ox);
        my = fmaxf(my, oy);
      } else {
        mx = my = fmaxf(mx, my);
      }
      if (!keep) continue;
      const KvScale sx = kv_scale(mx, gs), sy = split ? kv_scale(my, gs) : sx;
      uint8_t* const blk = block_of(h) + (key ? 0 : L::kValueCodes);
      *reinterpret_cast<uint32_t*>(blk + row * L::kCodeRow + at0 / 2) = codes8(x, sx.r);
      *reinterpret_cast<uint32_t*>(blk + row * L::kCodeRow + at1 / 2) = codes8(y, sy.r);
      uint8_t* const scales = blk + L::kKeyScales + row * L::kScaleRow;
      if (!split) {
        scales[u] = (uint8_t)sx.code;
      } else if (u % 2 == 0) {
        scales[at0 / 16] = (uint8_t)sx.code;
        scales[at1 / 16] = (uint8_t)sy.code;
      }
    }
  }
}

}  // namespace

// How many threads share a token's heads: as many as keep the GPU busy, one
// for every eight heads at least.
static int head_splits(long long tokens_units, int heads) {
  const long long want = (long long)sm_count() * 2048 / (tokens_units > 0 ? tokens_units : 1) + 1;
  const long long least = (heads + 7) / 8;
  return (int)(want < least ? least : want > heads ? heads : want);
}

moe_status launch_rope(const moe_rope_args& args, cudaStream_t s) {
  moe_rope_args a = args;
  const bool in_place = a.q_out == a.q && (a.k_heads == 0 || a.k_out == a.k);
  if (a.k_heads == 0) {   // never used
    a.k = a.q;
    a.k_stride = a.q_stride;
    a.k_out = a.q_out;
    a.k_out_stride = a.q_out_stride;
  }
  auto wide = [](const void* x, long long stride) { return reinterpret_cast<uintptr_t>(x) % 16 == 0 && stride % 8 == 0; };
  const bool vectors = a.head_dim % 8 == 0 && a.plan.rotary_dim % 16 == 0 && wide(a.q, a.q_stride) &&
                       wide(a.k, a.k_stride) && wide(a.q_out, a.q_out_stride) && wide(a.k_out, a.k_out_stride);
  const int per = vectors ? 16 : 2, rest = a.head_dim - a.plan.rotary_dim;
  RopeRows p;
  p.a = a;
  p.turning = a.plan.rotary_dim / per;
  p.units = p.turning + (in_place ? 0 : (rest + per - 1) / per);
  auto sectors = [](const void* x, long long stride) { return reinterpret_cast<uintptr_t>(x) % 32 == 0 && stride % 16 == 0; };
  const bool wide_units = vectors && a.plan.adjacent && a.head_dim % 16 == 0 && sectors(a.q, a.q_stride) &&
                          sectors(a.k, a.k_stride) && sectors(a.q_out, a.q_out_stride) && sectors(a.k_out, a.k_out_stride);
  const int heads = a.q_heads + a.k_heads;
  p.splits = head_splits((long long)a.tokens * p.units, heads);
  const long long per_token = (long long)p.splits * p.units;
  if (a.tokens > ((1ll << 32) - kThreads) / per_token) return MOE_ERR_UNSUPPORTED;   // threads are counted in 32 bits
  const unsigned grid = (unsigned)((a.tokens * per_token + kThreads - 1) / kThreads);
  const auto k = !vectors ? rope_pair_kernel : wide_units ? rope_vector_kernel<true> : rope_vector_kernel<false>;
  const cudaError_t e = launch_ex(true, k, dim3(grid), dim3(kThreads), 0, s, p);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

moe_status launch_kv4_append_rope(const moe_kv4_append_rope_args& a, cudaStream_t s) {
  AppendRope p;
  p.a = a;
  p.page_log = __builtin_ctz(a.cache.page_tokens);
  const int D = a.cache.head_dim, rows = a.q_heads + 2 * a.cache.kv_heads, tokens = 512 / D;
  const long long runs = ((long long)a.tokens + tokens - 1) / tokens;
  // A warp for each few rows, at least a CTA's eight where there are that many rows.
  constexpr int kWarps = kThreads / 32;
  const int least = rows < kWarps ? rows : kWarps, want = head_splits(runs * 32, rows);
  p.splits = want < least ? least : want;
  const int warps = p.splits < kWarps ? p.splits : kWarps, ctas = (p.splits + warps - 1) / warps;
  p.splits = warps * ctas;
  auto sectors = [](const void* x, long long stride) { return reinterpret_cast<uintptr_t>(x) % 32 == 0 && stride % 16 == 0; };
  p.wide_in = sectors(a.q, a.q_stride) && sectors(a.k, a.k_stride) && sectors(a.v, a.v_stride);
  p.wide_out = a.plan.adjacent && sectors(a.q_out, a.q_out_stride);
  const cudaError_t e = launch_ex(true, D == 64 ? kv4_append_rope_kernel<64> : kv4_append_rope_kernel<128>,
                                  dim3((unsigned)runs, ctas), dim3(warps * 32), 0, s, p);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

}  // namespace moe
