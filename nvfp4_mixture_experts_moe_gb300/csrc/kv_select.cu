// The cached blocks that each query picks: scores against the blocks' mean
// keys, and the best of them.
//
// Mathematics. u, the group's queries on a grid of whole numbers, has elements
// of up to 64 * 16 = 2^10, a mean up to 2^7 times a power of two of its row,
// 128 products a score: whole numbers of at most 2^24 of that power, so fp32
// sums are exact in any order. A score becomes a 32-bit key of the same order;
// the pick is all keys above the one of rank `need` and the first of its
// equals. That key is found by halving: of the interval of values and of the
// interval of keys in turn, the first quick where scores lie close together,
// the second bounded whatever they are.
//
// Two kernels. Requests of up to kFewRows rows: a CTA (or a cluster) for a
// (query, head) scores the blocks on the FMA pipe, for the means' bytes are
// what a single query costs. More rows: 128 queries of a head a CTA, a thread
// each, scores by tcgen05 from tensor memory; the thread keeps a list of the
// blocks above the lowest score that can still win.
#include <cooperative_groups.h>

#include <cfloat>

#include "kernels.cuh"
#include "kv4.cuh"
#include "kv_lookup.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;
namespace cg = cooperative_groups;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kFewRows = 8;

// A float's bits in the order of its value (0 is below every key of a number).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k ^ ((int)k < 0 ? 0x80000000u : 0xffffffffu)); }

// A key between lo and hi (hi > lo + 1): half way between the values, or (odd
// steps, and where that is no key between) between the keys.
__device__ __forceinline__ uint32_t middle(uint32_t lo, uint32_t hi, int step) {
  const uint32_t k = order_key(0.5f * key_value(lo) + 0.5f * key_value(hi));
  return (step & 1) || k <= lo || k >= hi ? lo + (hi - lo) / 2 : k;
}

// What a block whose page is not in the pool scores (one whose mean is NaN too): below every sum.
constexpr float kBadScore = -FLT_MAX;

struct SelectArgs {
  moe_kv4_select_args a;
  int block_log;
  int rows;      // CTAs of a request (few queries); 0: of any row
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
__device__ __forceinline__ int entry_of(const moe_kv4_index& x, int page_log, int block_log, const int32_t* table, int j) {
  const int tok = j << block_log, page = __ldg(table + (tok >> page_log));
  if (page < 0 || page >= x.cache.num_pages) return -1;
  return page_log > block_log ? (page << (page_log - block_log)) + ((tok & ((1 << page_log) - 1)) >> block_log) : page;
}

// Elements of the group's queries on their grid: 2^(5 - E), E from the largest
// magnitude's bits (finite ones only).
__device__ __forceinline__ uint32_t finite_bits(uint32_t x) {
  const uint32_t m = x & 0x7fffu;
  return m < 0x7f80u ? m : 0u;
}
__device__ __forceinline__ float grid_scale(uint32_t top_bits) {
  const int e = max((int)(top_bits >> 7), 27);   // the exponent, at least -100
  return __int_as_float((127 + 5 + 127 - e) << 23);
}
__device__ __forceinline__ float on_grid(uint32_t x, float scale) {
  return finite_bits(x) == 0 ? 0.0f : rintf(__uint_as_float(x << 16) * scale);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// ---------------------------------------------------------- few queries
// D / 16 lanes score a block, kAhead blocks at a time (the trips to memory for
// the table and the means are what takes long); the CTAs of a cluster send
// their keys to the first. There a warp cuts each run of keys to its best, and
// one warp cuts what is left of all runs: halving within a warp needs no
// barriers, with them a step took 860 cycles.
constexpr int kThreads = 512, kWarps = kThreads / 32, kKeys = 4096, kAhead = 4;
constexpr int kPer = (kKeys + kSparseTop + kThreads - 1) / kThreads;      // keys a lane of the first cut
constexpr int kPer2 = kWarps * kSparseTop / 32;                           // and of the second

struct FewSmem {
  uint32_t keys[kPer * kThreads];
  alignas(16) float u[128];
  int best[2][kSparseTop];               // blocks that earlier chunks left
  uint32_t best_key[2][kSparseTop];
  uint32_t run_key[kWarps * kSparseTop];
  int run_blk[kWarps * kSparseTop];
  uint32_t group_top;
};

// The `need` largest of `total` keys (reg[i]: key 32 i + lane, 0 past the end), the first of equal ones, to put(where,
// i) in order; all where there are no more. By a whole warp.
template <int N, class Put>
__device__ __forceinline__ void warp_cut(const uint32_t (&reg)[N], int total, int need, Put put) {
  const int lane = threadIdx.x & 31, groups = (total + 31) / 32;
  uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (32 * i + lane < total) {
      lo = min(lo, reg[i]);
      hi = max(hi, reg[i]);
    }
  lo = __reduce_min_sync(kFull, lo);
  hi = __reduce_max_sync(kFull, hi) + 1;
  int at_least = total, above = 0;   // keys >= lo, >= hi
  for (int step = 0; at_least > need && hi - lo > 1; ++step) {
    // three keys in between at once
    const uint32_t m1 = middle(lo, hi, step), m0 = m1 - lo > 1 ? middle(lo, m1, step) : lo,
                   m2 = hi - m1 > 1 ? middle(m1, hi, step) : hi;
    int c0 = 0, c1 = 0, c2 = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= groups) break;
      c0 += reg[i] >= m0;
      c1 += reg[i] >= m1;
      c2 += reg[i] >= m2;
    }
    // at most 32 * 32 keys: two counts a word
    const unsigned two = __reduce_add_sync(kFull, (unsigned)(c0 | c1 << 16));
    c2 = m2 == hi ? above : __reduce_add_sync(kFull, c2);
    c0 = m0 == lo ? at_least : (int)(two & 0xffffu);
    c1 = (int)(two >> 16);
    if (c2 >= need && m2 != hi) lo = m2, at_least = c2;
    else if (c1 >= need) lo = m1, at_least = c1, hi = m2, above = c2;
    else if (c0 >= need) lo = m0, at_least = c0, hi = m1, above = c1;
    else hi = m0, above = c0;
  }
  int equals = at_least > need ? need - above : total;   // too many of one key: the first of them
  int w = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i >= groups) break;
    const bool in = 32 * i + lane < total;
    const unsigned below = (1u << lane) - 1, e = __ballot_sync(kFull, in && reg[i] == lo);
    const bool take = in && (reg[i] > lo || (reg[i] == lo && __popc(e & below) < equals));
    const unsigned t = __ballot_sync(kFull, take);
    if (take) put(w + __popc(t & below), i);
    w += __popc(t);
    equals -= __popc(e);
  }
}

// One query and head, by a whole cluster.
template <int D>
__device__ __forceinline__ void select_row(const SelectArgs& p, const RowOwner& own, int t, int h, FewSmem& sm, int rank,
                                           int ranks) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  constexpr int kStep = kWarps * kRows;   // blocks that a CTA's warps take at once
  const moe_kv4_select_args& a = p.a;
  const moe_kv4_cache& c = a.index.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hk = c.kv_heads, heads = a.q_heads / Hk, page_log = __ffs(c.page_tokens) - 1;
  const Visible v = visible(a, p.block_log, own.kv - own.n + t - own.c0);
  int32_t* const out = a.blocks + ((size_t)t * Hk + h) * a.top;
  if (v.seen <= a.top) {
    if (tid < a.top && rank == 0) out[tid] = tid < v.seen ? tid : -1;
    return;
  }
  if (rank == 0) {
    if (tid < a.sink) out[tid] = tid;
    if (tid < a.local) out[a.top - a.local + tid] = v.c1 + tid;
  }
  if (v.need == 0) return;

  const int32_t* const table = a.block_table + (size_t)own.b * a.max_pages;
  int entry[kAhead];
  uint4 w[kAhead][2];
  // The means of this thread's blocks of a round, asked for before what multiplies them is there.
  auto load = [&](int from, int n, int j0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = j0 + i * kStep + lane / kLanes;
      entry[i] = j < n ? entry_of(a.index, page_log, p.block_log, table, from + j) : -2;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (entry[i] >= 0) {
        const uint4* m = reinterpret_cast<const uint4*>(a.index.means + ((size_t)entry[i] * Hk + h) * D) + lane % kLanes * 2;
        w[i][0] = __ldg(m);
        w[i][1] = __ldg(m + 1);
      }
    }
  };
  const int first = rank * kStep * kAhead + warp * kRows;
  if (tid == 0) sm.group_top = 0;
  uint32_t x[kSparseGroup];   // element tid of the group's queries
  if (tid < D) {
    const uint16_t* const q = a.q + (size_t)t * a.q_stride + (size_t)h * heads * D + tid;
#pragma unroll
    for (int i = 0; i < kSparseGroup; ++i) x[i] = i < heads ? q[i * D] : 0u;
  }
  load(v.c0, min(kKeys, v.c1 - v.c0), first);
  __syncthreads();
  if (tid < D) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kSparseGroup; ++i) top = max(top, finite_bits(x[i]));
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) atomicMax(&sm.group_top, top);
  }
  __syncthreads();
  if (tid < D) {
    const float scale = grid_scale(sm.group_top);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSparseGroup; ++i) s += on_grid(x[i], scale);
    sm.u[tid] = s;
  }
  __syncthreads();

  uint32_t* const keys = ranks > 1 ? cg::this_cluster().map_shared_rank(sm.keys, 0) : sm.keys;
  int carried = 0, side = 0;
  for (int from = v.c0; from < v.c1; from += kKeys) {
    const int n = min(kKeys, v.c1 - from);
    const bool last = from + n == v.c1;
    for (int j0 = first; j0 < n; j0 += ranks * kStep * kAhead) {
      if (from > v.c0 || j0 > first) load(from, n, j0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = j0 + i * kStep + lane / kLanes;
        if (j - lane / kLanes >= n) break;   // the same for a whole warp
        const float4* const u4 = reinterpret_cast<const float4*>(sm.u + lane % kLanes * 16);
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t m0 = k % 2 ? w[i][k / 2].z : w[i][k / 2].x, m1 = k % 2 ? w[i][k / 2].w : w[i][k / 2].y;
          const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&m0));
          const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&m1));
          const float4 uk = u4[k];
          s = fmaf(f0.x, uk.x, s);
          s = fmaf(f0.y, uk.y, s);
          s = fmaf(f1.x, uk.z, s);
          s = fmaf(f1.y, uk.w, s);
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) s += __shfl_xor_sync(kFull, s, o);
        if (lane % kLanes == 0 && j < n) {
          keys[carried + j] = order_key(entry[i] >= 0 ? fmaxf(s, kBadScore) : kBadScore);
          if (entry[i] < 0 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
        }
      }
    }
    if (rank == 0 && tid < carried) sm.keys[tid] = sm.best_key[side][tid];
    if (ranks > 1) cg::this_cluster().sync();
    else __syncthreads();

    if (rank == 0) {
      // A warp's run of neighbouring keys; what the runs before it keep is known beforehand.
      const int total = carried + n, seg = (total + kThreads - 1) / kThreads * 32, at = warp * seg;
      {
        const int mine = max(0, min(seg, total - at));
        int before = 0;
        for (int k = 0; k < warp; ++k) before += min(max(0, min(seg, total - k * seg)), v.need);
        uint32_t reg[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) reg[i] = 32 * i + lane < mine ? sm.keys[at + 32 * i + lane] : 0u;
        if (mine > 0)
          warp_cut(reg, mine, v.need, [&](int where, int i) {
            const int key = at + 32 * i + lane;
            sm.run_key[before + where] = reg[i];
            sm.run_blk[before + where] = key < carried ? sm.best[side][key] : from + key - carried;
          });
      }
      __syncthreads();
      if (warp == 0) {
        int left = 0;
        for (int k = 0; k < kWarps; ++k) left += min(max(0, min(seg, total - k * seg)), v.need);
        uint32_t reg[kPer2];
#pragma unroll
        for (int i = 0; i < kPer2; ++i) reg[i] = 32 * i + lane < left ? sm.run_key[32 * i + lane] : 0u;
        warp_cut(reg, left, v.need, [&](int where, int i) {
          const int blk = sm.run_blk[32 * i + lane];
          if (last) {
            out[a.sink + where] = blk;
          } else {
            sm.best[side ^ 1][where] = blk;
            sm.best_key[side ^ 1][where] = reg[i];
          }
        });
      }
    }
    carried = min(carried + n, v.need);
    side ^= 1;
    if (ranks > 1) cg::this_cluster().sync();   // the first has read what the others wrote
    else __syncthreads();
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_select_few_kernel(const __grid_constant__ SelectArgs p) {
  __shared__ FewSmem sm;
  const moe_kv4_select_args& a = p.a;
  const int Hk = a.index.cache.kv_heads, cap = a.max_pages * a.index.cache.page_tokens;
  const int ranks = (int)cg::this_cluster().num_blocks(), rank = (int)cg::this_cluster().block_rank();
  const int item = blockIdx.x / ranks, h = item % Hk;
  // All CTAs of a cluster run before one writes to another: they meet while the lengths come.
  if (ranks > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  pdl_wait();
  const RowOwner own = p.rows == 0 ? row_owner(a.cu_q, a.kv_len, a.batch, a.total_q, a.max_q, cap, item / Hk)
                                   : request_of(a.cu_q, a.kv_len, a.total_q, a.max_q, cap, item / Hk / p.rows);
  if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (own.bad && threadIdx.x == 0 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
  if (own.b < 0) return;
  if (p.rows == 0) {
    select_row<D>(p, own, item / Hk, h, sm, rank, ranks);
    return;
  }
  // A request's rows, dealt out to `rows` CTAs.
  if (own.n > kFewRows) return;
  for (int i = item / Hk % p.rows; i < own.n; i += p.rows) select_row<D>(p, own, own.c0 + i, h, sm, rank, ranks);
}

// --------------------------------------------------------- many queries
// Warps 0 to 3: a thread a query. It puts u into tensor memory (the A operand),
// then reads its row of each score tile and appends what lies above its bound
// to its list; a list of more than kKeep is cut at a key that leaves at least
// `need`. Warps 4 to 7 bring the means of 64 blocks a stage (cp.async into
// 128-byte-swizzled rows); one thread of warp 8 issues the products.
constexpr int kTile = 128, kCols = 64, kStages = 2, kGroup = 32, kKeep = 64, kList = kKeep + kGroup;
constexpr int kManyThreads = 288, kTmem = 256;
constexpr int kMostBlocks = 65536;   // list entries name blocks in 16 bits
constexpr long long kWaitLimit = 2ll * 1000 * 1000 * 1000;   // cycles (about 1 s)

struct Segment {
  int b, end;     // request; the last row's c1
};

template <int D>
struct ManySmem {
  alignas(1024) uint8_t ring[kStages][kCols * D * 2];
  uint32_t key[kList][kTile];
  uint16_t blk[kList][kTile];
  Segment seg[kTile];
  int owner[kTile + 2];          // of rows -1 .. kTile
  int segments, abort;
  uint32_t tmem;
  uint64_t full[kStages], empty[kStages], scored[2], read[2], rows_in, drained;
};

// A thread's list: cnt entries in the order of their blocks.
template <class Sm>
struct List {
  Sm& sm;
  int row, cnt;
  float bound;         // at least `need` entries reach it: what comes later and is not above cannot win
  __device__ __forceinline__ uint32_t key(int i) const { return sm.key[i][row]; }

  // Cuts the list to at least `need` and at most `most` (>= need) entries, if it has more. Whole warps, in step up to
  // the longest list: what a thread has past its own is read and not counted.
  __device__ __forceinline__ void cut(int need, int most) {
    const bool wanted = cnt > most && need > 0;
    const int longest = __reduce_max_sync(kFull, wanted ? cnt : 0);
    uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll 8
    for (int i = 0; i < longest; ++i) {
      const uint32_t k = key(i);
      if (i < cnt) {
        lo = min(lo, k);
        hi = max(hi, k);
      }
    }
    hi += 1;
    int at_least = cnt, above = 0;     // entries >= lo, >= hi
    for (int step = 0;; ++step) {
      const bool go = wanted && at_least > most && hi - lo > 1;
      if (!__any_sync(kFull, go)) break;
      const uint32_t mid = go ? middle(lo, hi, step) : 0xffffffffu;
      int c = 0;
#pragma unroll 8
      for (int i = 0; i < longest; ++i) c += key(i) >= mid && i < cnt;
      if (go) {
        if (c >= need) lo = mid, at_least = c;
        else hi = mid, above = c;
      }
    }
    int equals = at_least > most ? need - above : cnt;   // too many of one key: the first of them
    int w = wanted ? 0 : cnt;
#pragma unroll 4
    for (int i = 0; i < longest; ++i) {
      const uint32_t k = key(i);
      if (wanted && i < cnt && (k > lo || (k == lo && equals-- > 0))) {
        sm.key[w][row] = k;
        sm.blk[w][row] = sm.blk[i][row];
        ++w;
      }
    }
    cnt = w;
    if (wanted) bound = key_value(lo);
  }
};

template <int D>
__global__ void __launch_bounds__(kManyThreads, 2) kv4_select_many_kernel(const __grid_constant__ SelectArgs p) {
  using Sm = ManySmem<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const moe_kv4_select_args& a = p.a;
  const moe_kv4_cache& c = a.index.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hk = c.kv_heads, heads = a.q_heads / Hk, page_log = __ffs(c.page_tokens) - 1;
  const int t0 = blockIdx.x / Hk * kTile, h = blockIdx.x % Hk;
  pdl_wait();
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 128);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.scored[i], 1);
      mbar_init(&sm.read[i], kTile);
    }
    mbar_init(&sm.rows_in, kTile);
    mbar_init(&sm.drained, 1);
    sm.segments = 0;
    sm.abort = 0;
    fence_barrier_init();
  }
  // ------------------------------------------------- whose rows these are
  RowOwner own = {-1, 0, 0, 0, false};
  Visible v = {0, 0, 0, 0};
  const int t = t0 + tid;
  if (tid < kTile) {
    if (t < a.total_q) own = row_owner_thread(a.cu_q, a.kv_len, a.batch, a.total_q, a.max_q, a.max_pages * c.page_tokens, t);
    if (own.bad && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
    if (own.b >= 0 && own.n <= kFewRows) own.b = -1;   // the other kernel's
    int32_t* const out = a.blocks + ((size_t)t * Hk + h) * a.top;
    if (own.b >= 0) {
      v = visible(a, p.block_log, own.kv - own.n + t - own.c0);
      if (v.seen <= a.top) {
        for (int i = 0; i < a.top; ++i) out[i] = i < v.seen ? i : -1;
      } else {
        for (int i = 0; i < a.sink; ++i) out[i] = i;
        for (int i = 0; i < a.local; ++i) out[a.top - a.local + i] = v.c1 + i;
      }
    }
    sm.owner[tid + 1] = v.need > 0 ? own.b : -1;
    if (tid == 0) sm.owner[0] = -1, sm.owner[kTile + 1] = -1;
  }
  __syncthreads();
  // Rows that rank blocks, as runs of one request; a later row of a run ends later.
  if (tid < kTile && v.need > 0 && sm.owner[tid + 2] != own.b) {
    int k = 0;   // runs that end before this one
    for (int i = 0; i < tid; ++i) k += sm.owner[i + 1] >= 0 && sm.owner[i + 2] != sm.owner[i + 1];
    sm.seg[k] = {own.b, v.c1};
    atomicAdd(&sm.segments, 1);
  }
  if (warp == 8) tmem_alloc(&sm.tmem, kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;               // scores in columns 0..127 (two tiles), u in the D / 2 after 128
  volatile int* const abort = &sm.abort;
  const int segments = sm.segments;

  if (segments > 0 && warp < 4) {
    // ------------------------------------------------------------- queries
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    {
      const uint16_t* const q = a.q + (size_t)min(t, a.total_q - 1) * a.q_stride + (size_t)h * heads * D;
      const bool real = v.need > 0;
      uint32_t pair = 0;
      if (real)
        for (int i = 0; i < heads * D / 8; ++i) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(q) + i);
          pair = max_u16x2(max_u16x2(pair, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
          pair = max_u16x2(max_u16x2(pair, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
        }
      uint32_t top = max(pair & 0xffffu, pair >> 16);
      const bool finite = top < 0x7f80u;
      if (!finite) {   // again without what counts as 0
        top = 0;
        for (int i = 0; i < heads * D; ++i) top = max(top, finite_bits(q[i]));
      }
      const float scale = grid_scale(top);
      const uint32_t scale2 = __float_as_uint(scale) >> 16 | (__float_as_uint(scale) & 0xffff0000u);
#pragma unroll 1
      for (int d0 = 0; d0 < D; d0 += 32) {
        // x scale + 192 in bf16 is 192 and the rounded product (at most 64), whose bits are 0x4300 + 64 + that
        uint32_t r[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = 0;
        if (real)
          for (int g = 0; g < heads; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 x = __ldg(reinterpret_cast<const uint4*>(q + g * D + d0) + i);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t y = w[j];
                if (!finite) y = (finite_bits(y) ? y & 0xffffu : 0u) | (finite_bits(y >> 16) ? y & 0xffff0000u : 0u);
                r[4 * i + j] += fma_bf16x2(y, scale2, 0x43404340u) - 0x43004300u;
              }
            }
        const float zero = real ? 64.0f * heads : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const __half2 x = __floats2half2_rn((float)(r[i] & 0xffffu) - zero, (float)(r[i] >> 16) - zero);
          r[i] = *reinterpret_cast<const uint32_t*>(&x);
        }
        tmem_st16(tmem + lanes + 128 + d0 / 2, r);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sm.rows_in);
    }
    List<Sm> list = {sm, tid, 0, -INFINITY};
    int tile = 0;
    bool ok = true;
    for (int sg = 0; sg < segments && ok; ++sg) {
      const Segment seg = sm.seg[sg];
      const int c1 = v.need > 0 && own.b == seg.b ? v.c1 : 0;
      for (int j0 = a.sink; j0 < seg.end; j0 += kCols, ++tile) {
        const int buf = tile & 1;
        ok = __all_sync(kFull, mbar_wait(&sm.scored[buf], tile >> 1 & 1, abort, kWaitLimit));
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int g = 0; g < kCols / kGroup; ++g) {
          uint32_t r[kGroup];
          tmem_ld32(tmem + lanes + buf * kCols + g * kGroup, r);
          tmem_ld_wait();
          if (g == kCols / kGroup - 1) {
            tc_fence_before();
            mbar_arrive(&sm.read[buf]);
          }
          const int j = j0 + g * kGroup, n = min(kGroup, c1 - j);   // this row's blocks of the group
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            const float s = fmaxf(__uint_as_float(r[i]), kBadScore);   // which a NaN gives
            if (s > list.bound && i < n) {
              sm.key[list.cnt][tid] = order_key(s);
              sm.blk[list.cnt][tid] = (uint16_t)(j + i);
              ++list.cnt;
            }
          }
          // One list too long: every list is cut that is much longer than it has to be.
          if (__any_sync(kFull, list.cnt > kKeep)) list.cut(v.need, min(kKeep, v.need + 7));
        }
      }
    }
    // ------------------------------------------------- the best, in order
    list.cut(v.need, v.need);
    if (v.need > 0) {
      int32_t* const out = a.blocks + ((size_t)t * Hk + h) * a.top + a.sink;
      for (int i = 0; i < v.need; ++i) out[i] = ok && i < list.cnt ? sm.blk[i][tid] : -1;
    }
  } else if (segments > 0 && warp < 8) {
    // --------------------------------------------------------------- means
    constexpr int kChunks = D / 8, kPerThread = kCols * kChunks / 128;   // 16-byte pieces of a row, of a thread
    int tile = 0, done = 0;
    bool ok = true;
    for (int sg = 0; sg < segments && ok; ++sg) {
      const Segment seg = sm.seg[sg];
      const int32_t* const table = a.block_table + (size_t)seg.b * a.max_pages;
      for (int j0 = a.sink; j0 < seg.end; j0 += kCols, ++tile) {
        const int stage = tile % kStages;
        // the table's entries first: they do not wait for the stage
        int entry[kPerThread];
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
          const int j = j0 + ((tid - 128) + 128 * i) / kChunks;
          entry[i] = j < seg.end ? entry_of(a.index, page_log, p.block_log, table, j) : -2;
        }
        ok = __all_sync(kFull, mbar_wait(&sm.empty[stage], (tile / kStages & 1) ^ 1, abort, kWaitLimit));
        if (!ok) break;
        const uint32_t dst = smem_u32(sm.ring[stage]);
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
          const int idx = tid - 128 + 128 * i, row = idx / kChunks, ch = idx % kChunks;
          // K halves of 64 elements one after the other, rows of 128 bytes
          const uint32_t at = (uint32_t)(ch / 8 * (kCols * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
          if (entry[i] == -1) {   // a page that is not in the pool: a row of NaN, which no mean is
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + at), "r"(0x7e007e00u) : "memory");
            if (a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
          } else {
            const uint16_t* src = a.index.means + ((size_t)max(entry[i], 0) * Hk + h) * D + ch * 8;
            cp_async_16(dst + at, src, entry[i] >= 0 ? 16u : 0u);
          }
        }
        cp_async_commit();
        if (tile > done) {     // the stage before this one is in
          cp_async_wait<1>();
          fence_proxy_async_smem();
          mbar_arrive(&sm.full[done % kStages]);
          ++done;
        }
      }
    }
    cp_async_wait_all();
    if (done < tile) {
      fence_proxy_async_smem();
      mbar_arrive(&sm.full[done % kStages]);
    }
  } else if (segments > 0 && lane == 0) {
    // ------------------------------------------------------------ products
    constexpr uint32_t idesc = idesc_f16(kTile, kCols, 0);
    int tile = 0;
    bool ok = mbar_wait(&sm.rows_in, 0, abort, kWaitLimit);
    tc_fence_after();
    for (int sg = 0; sg < segments && ok; ++sg) {
      const Segment seg = sm.seg[sg];
      for (int j0 = a.sink; j0 < seg.end; j0 += kCols, ++tile) {
        const int buf = tile & 1, stage = tile % kStages;
        ok = mbar_wait(&sm.full[stage], tile / kStages & 1, abort, kWaitLimit) &&
             mbar_wait(&sm.read[buf], (tile >> 1 & 1) ^ 1, abort, kWaitLimit);
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = smem_u32(sm.ring[stage]);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_f16_tmem_a(tmem + buf * kCols, tmem + 128 + k * 8,
                         smem_desc(src + k / 4 * (kCols * 128) + k % 4 * 32, 16, 1024, kSwizzle128B), idesc, k != 0);
        tc_commit(&sm.empty[stage]);
        tc_commit(&sm.scored[buf]);
      }
    }
    // What was issued is complete before tensor memory is given back (also after a wait that gave up).
    tc_commit(&sm.drained);
    const long long c0 = clock64();
    while (!mbar_try_wait(&sm.drained, 0) && clock64() - c0 < kWaitLimit) {
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, kTmem);
  if (tid == 0 && sm.abort && a.device_status != nullptr) set_status(a.device_status, MOE_ERR_TIMEOUT);
}

template <int D>
cudaError_t launch_few(const SelectArgs& p, long long items, cudaStream_t s) {
  // CTAs for a query: as many as fit the GPU at once and have a round of blocks each where the table is full.
  const long long most = (long long)p.a.max_pages * p.a.index.cache.page_tokens >> p.block_log;
  const int step = kWarps * (512 / D) * kAhead;
  int ranks = 1;
  while (ranks < 8 && items * ranks * 2 <= sm_count() && most > (long long)step * ranks) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)ranks, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kv4_select_few_kernel<D>, p);
}

template <int D>
cudaError_t launch_many(const SelectArgs& p, cudaStream_t s) {
  constexpr size_t smem = sizeof(ManySmem<D>) + 1024;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(kv4_select_many_kernel<D>, smem, done);
  if (e != cudaSuccess) return e;
  const unsigned tiles = (unsigned)(((long long)p.a.total_q + kTile - 1) / kTile);
  return launch_ex(true, kv4_select_many_kernel<D>, dim3(tiles * p.a.index.cache.kv_heads), dim3(kManyThreads), smem, s, p);
}

}  // namespace

moe_status launch_kv4_select(const moe_kv4_select_args& a, cudaStream_t s) {
  SelectArgs p;
  p.a = a;
  p.block_log = __builtin_ctz(a.index.block_tokens);
  const int D = a.index.cache.head_dim, Hk = a.index.cache.kv_heads;
  // Lengths are on the device: a call that allows requests of more than
  // kFewRows rows launches both kernels, each skipping the other's. A CTA of
  // the first then has all rows of a request, as most requests will have one.
  const bool long_lists = ((long long)a.max_pages * a.index.cache.page_tokens >> p.block_log) > kMostBlocks;
  const bool many = a.max_q > kFewRows && !long_lists;
  p.rows = long_lists && a.max_q > kFewRows ? 0 : many ? 1 : a.max_q;
  const long long items = (p.rows == 0 ? (long long)a.total_q : (long long)a.batch * p.rows) * Hk;
  cudaError_t e = D == 64 ? launch_few<64>(p, items, s) : launch_few<128>(p, items, s);
  if (e == cudaSuccess && many) e = D == 64 ? launch_many<64>(p, s) : launch_many<128>(p, s);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(many ? 2 : 1);
  return MOE_OK;
}

}  // namespace moe
