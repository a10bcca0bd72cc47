// The cached blocks that each query picks: scores against the blocks' mean
// keys, and the best of them.
//
// Mathematics. u, the group's queries on a grid of whole numbers, has elements
// of up to 64 * 16 = 2^10, a mean up to 2^7 times a power of two of its row,
// 128 products a score: whole numbers of at most 2^24 of that power, so fp32
// sums are exact in any order. A score becomes a 32-bit key of the same order;
// the pick is all keys above the one of rank `need` and the first of its equals.
#include "kernels.cuh"
#include "kv4.cuh"
#include "kv_lookup.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSelectMax = 64;

// A float's bits in the order of its value (0 is below every key of a number).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u);
}

struct SelectArgs {
  moe_kv4_select_args a;
  int block_log;
};

// Which blocks a query at `pos` takes without asking and which it ranks.
struct Visible {
  int seen;        // blocks it sees
  int c0, c1;      // the ranked ones
  int need;        // how many of them
};

__device__ __forceinline__ Visible visible(const moe_kv4_select_args& a, int block_log, int pos) {
  Visible v;
  v.seen = pos < 0 ? 0 : (pos >> block_log) + 1;
  v.c0 = a.sink;
  v.c1 = v.seen - a.local;
  v.need = v.seen > a.top ? a.top - a.sink - a.local : 0;
  return v;
}

// Where the mean of block j of a request lies; -1: its page is not in the pool.
__device__ __forceinline__ long long entry_of(const moe_kv4_index& x, int block_log, const int32_t* table, int j) {
  const int P = x.cache.page_tokens, tok = j << block_log;
  const int page = __ldg(table + tok / P);
  if (page < 0 || page >= x.cache.num_pages) return -1;
  return P > x.block_tokens ? (long long)page * (P >> block_log) + ((tok & (P - 1)) >> block_log) : page;
}

// Elements of the group's queries on their grid: 2^(5 - E), E from the largest
// magnitude's bits (finite ones only).
__device__ __forceinline__ uint32_t finite_bits(uint16_t x) {
  const uint32_t m = x & 0x7fffu;
  return m < 0x7f80u ? m : 0u;
}
__device__ __forceinline__ float grid_scale(uint32_t top_bits) {
  const int e = max((int)(top_bits >> 7), 27);   // the exponent, at least -100
  return __int_as_float((127 + 5 + 127 - e) << 23);
}
__device__ __forceinline__ float on_grid(uint16_t x, float scale) {
  return finite_bits(x) == 0 ? 0.0f : rintf(bf16_bits_to_float(x) * scale);
}

// ---------------------------------------------------------- few queries
// A CTA has one (query, head): its threads score the ranked blocks (D / 16
// lanes a block), then find the key of rank `need` bit by bit.
constexpr int kThreads = 512, kWarps = kThreads / 32, kKeys = 8192, kPer = kKeys / kThreads + 1;

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_select_kernel(const __grid_constant__ SelectArgs p) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  __shared__ uint32_t keys[kKeys + kSelectMax];
  __shared__ float u[D];
  __shared__ int best[2][kSelectMax];     // blocks that earlier chunks left
  __shared__ uint32_t best_key[2][kSelectMax];
  __shared__ int counts[33], above[kWarps], equal[kWarps];
  __shared__ uint32_t group_top;
  const moe_kv4_select_args& a = p.a;
  const moe_kv4_cache& c = a.index.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hk = c.kv_heads, heads = a.q_heads / Hk;
  pdl_wait();
  const int t = blockIdx.x / Hk, h = blockIdx.x - t * Hk;
  const RowOwner own = row_owner(a.cu_q, a.kv_len, a.batch, a.total_q, a.max_q, a.max_pages * c.page_tokens, t);
  if (own.bad && tid == 0 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
  if (own.b < 0) return;
  const int pos = own.kv - own.n + t - own.c0;
  const Visible v = visible(a, p.block_log, pos);
  int32_t* const out = a.blocks + ((size_t)t * Hk + h) * a.top;
  if (v.seen <= a.top) {
    if (tid < a.top) out[tid] = tid < v.seen ? tid : -1;
    return;
  }
  if (tid < a.sink) out[tid] = tid;
  if (tid < a.local) out[a.top - a.local + tid] = v.c1 + tid;
  if (v.need == 0) return;

  if (tid == 0) group_top = 0;
  __syncthreads();
  const uint16_t* const q = a.q + (size_t)t * a.q_stride + (size_t)h * heads * D;
  uint32_t top = 0;
  for (int i = tid; i < heads * D; i += kThreads) top = max(top, finite_bits(q[i]));
  top = __reduce_max_sync(kFull, top);
  if (lane == 0) atomicMax(&group_top, top);
  __syncthreads();
  if (tid < D) {
    const float scale = grid_scale(group_top);
    float s = 0.0f;
    for (int i = 0; i < heads; ++i) s += on_grid(q[i * D + tid], scale);
    u[tid] = s;
  }
  __syncthreads();
  float mine[16];   // this lane's elements of u
#pragma unroll
  for (int i = 0; i < 16; ++i) mine[i] = u[(lane % kLanes) * 16 + i];

  const int32_t* const table = a.block_table + (size_t)own.b * a.max_pages;
  int carried = 0, side = 0;
  for (int from = v.c0; from < v.c1; from += kKeys) {
    const int n = min(kKeys, v.c1 - from);
    const bool last = from + n == v.c1;
    for (int j0 = warp * kRows; j0 < n; j0 += kWarps * kRows) {
      const int j = j0 + lane / kLanes;
      const long long entry = j < n ? entry_of(a.index, p.block_log, table, from + j) : -1;
      float s = 0.0f;
      if (entry >= 0) {
        const uint4* m = reinterpret_cast<const uint4*>(a.index.means + ((size_t)entry * Hk + h) * D) + lane % kLanes * 2;
        const uint4 w[2] = {__ldg(m), __ldg(m + 1)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
            s = fmaf(f.x, mine[8 * k + 2 * i], s);
            s = fmaf(f.y, mine[8 * k + 2 * i + 1], s);
          }
        }
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) s += __shfl_xor_sync(kFull, s, o);
      if (lane % kLanes == 0 && j < n) keys[carried + j] = entry >= 0 ? order_key(s) : 0u;
      if (entry < 0 && j < n && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
    }
    if (tid < carried) keys[tid] = best_key[side][tid];
    if (tid < 33) counts[tid] = 0;
    __syncthreads();

    // The largest T with at least `need` keys >= T.
    const int total = carried + n, seg = (total + kThreads - 1) / kThreads * 32;   // keys of a warp, neighbours
    const int at = warp * seg + lane;
    uint32_t reg[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) reg[i] = i * 32 < seg && at + i * 32 < total ? keys[at + i * 32] : 0u;
    uint32_t T = 0;
    if (total > v.need) {
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t trial = T | 1u << bit;
        int cnt = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) cnt += reg[i] >= trial;
        cnt = __reduce_add_sync(kFull, cnt);
        if (lane == 0 && cnt) atomicAdd(&counts[bit], cnt);
        __syncthreads();
        cnt = counts[bit];
        if (cnt >= v.need) T = trial;
        if (cnt == v.need) break;
      }
    }
    // Those above T, and the first of its equals, in order.
    int gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool in = i * 32 < seg && at + i * 32 < total;
      gt += in && reg[i] > T;
      eq += in && reg[i] == T;
    }
    gt = __reduce_add_sync(kFull, gt);
    eq = __reduce_add_sync(kFull, eq);
    if (lane == 0) above[warp] = gt, equal[warp] = eq;
    __syncthreads();
    int all_gt = 0, gt0 = 0, eq0 = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) gt0 += above[w], eq0 += equal[w];
      all_gt += above[w];
    }
    const int eq_max = min(total, v.need) - all_gt;    // equals that are taken
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool in = i * 32 < seg && at + i * 32 < total;
      const unsigned g = __ballot_sync(kFull, in && reg[i] > T), e = __ballot_sync(kFull, in && reg[i] == T);
      const unsigned below = (1u << lane) - 1;
      const int my_eq = eq0 + __popc(e & below);
      if (in && (reg[i] > T || (reg[i] == T && my_eq < eq_max))) {
        const int where = gt0 + __popc(g & below) + min(my_eq, eq_max), key = at + i * 32;
        const int blk = key < carried ? best[side][key] : from + key - carried;
        if (last) {
          out[a.sink + where] = blk;
        } else {
          best[side ^ 1][where] = blk;
          best_key[side ^ 1][where] = reg[i];
        }
      }
      gt0 += __popc(g);
      eq0 += __popc(e);
    }
    carried = min(total, v.need);
    side ^= 1;
    __syncthreads();
  }
}

}  // namespace

moe_status launch_kv4_select(const moe_kv4_select_args& a, cudaStream_t s) {
  SelectArgs p;
  p.a = a;
  p.block_log = __builtin_ctz(a.index.block_tokens);
  const int D = a.index.cache.head_dim;
  const cudaError_t e = launch_ex(true, D == 64 ? kv4_select_kernel<64> : kv4_select_kernel<128>,
                                  dim3((unsigned)(a.total_q * a.index.cache.kv_heads)), dim3(kThreads), 0, s, p);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

}  // namespace moe
