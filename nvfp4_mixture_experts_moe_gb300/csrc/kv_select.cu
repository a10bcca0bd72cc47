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

// ---------------------------------------------------------- few queries
// D / 16 lanes score a block, kAhead blocks at a time (the trips to memory for
// the table and the means are what takes long); then the CTA's threads find
// the key of rank `need`, the CTAs of a cluster sending theirs to the first.
constexpr int kThreads = 512, kWarps = kThreads / 32, kKeys = 8192, kPer = kKeys / kThreads + 1, kAhead = 4;

struct FewSmem {
  uint32_t keys[kKeys + kSparseTop];
  float u[128];
  int best[2][kSparseTop];               // blocks that earlier chunks left
  uint32_t best_key[2][kSparseTop];
  int counts[3], above[kWarps], equal[kWarps];
  uint32_t lowest, highest, group_top;
};

// One query and head, by a whole cluster.
template <int D>
__device__ __forceinline__ void select_row(const SelectArgs& p, const RowOwner& own, int t, int h, FewSmem& sm, int rank,
                                           int ranks) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
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

  if (tid == 0) sm.group_top = 0;
  __syncthreads();
  const uint16_t* const q = a.q + (size_t)t * a.q_stride + (size_t)h * heads * D;
  uint32_t top = 0;
  for (int i = tid; i < heads * D; i += kThreads) top = max(top, finite_bits(q[i]));
  top = __reduce_max_sync(kFull, top);
  if (lane == 0) atomicMax(&sm.group_top, top);
  __syncthreads();
  if (tid < D) {
    const float scale = grid_scale(sm.group_top);
    float s = 0.0f;
    for (int i = 0; i < heads; ++i) s += on_grid(q[i * D + tid], scale);
    sm.u[tid] = s;
  }
  __syncthreads();
  float mine[16];   // this lane's elements of u
#pragma unroll
  for (int i = 0; i < 16; ++i) mine[i] = sm.u[(lane % kLanes) * 16 + i];

  const int32_t* const table = a.block_table + (size_t)own.b * a.max_pages;
  uint32_t* const keys = ranks > 1 ? cg::this_cluster().map_shared_rank(sm.keys, 0) : sm.keys;
  int carried = 0, side = 0;
  for (int from = v.c0; from < v.c1; from += kKeys) {
    const int n = min(kKeys, v.c1 - from);
    const bool last = from + n == v.c1;
    constexpr int kStep = kWarps * kRows;   // blocks that a CTA's warps take at once
    for (int j0 = rank * kStep * kAhead + warp * kRows; j0 < n; j0 += ranks * kStep * kAhead) {
      int entry[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = j0 + i * kStep + lane / kLanes;
        entry[i] = j < n ? entry_of(a.index, page_log, p.block_log, table, from + j) : -2;
      }
      uint4 w[kAhead][2];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (entry[i] >= 0) {
          const uint4* m = reinterpret_cast<const uint4*>(a.index.means + ((size_t)entry[i] * Hk + h) * D) + lane % kLanes * 2;
          w[i][0] = __ldg(m);
          w[i][1] = __ldg(m + 1);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t x[4] = {w[i][k].x, w[i][k].y, w[i][k].z, w[i][k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[e]));
            s = fmaf(f.x, mine[8 * k + 2 * e], s);
            s = fmaf(f.y, mine[8 * k + 2 * e + 1], s);
          }
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) s += __shfl_xor_sync(kFull, s, o);
        const int j = j0 + i * kStep + lane / kLanes;
        if (lane % kLanes == 0 && j < n) {
          keys[carried + j] = order_key(entry[i] >= 0 ? fmaxf(s, kBadScore) : kBadScore);
          if (entry[i] < 0 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
        }
      }
    }
    if (rank == 0) {
      if (tid < carried) sm.keys[tid] = sm.best_key[side][tid];
      if (tid < 3) sm.counts[tid] = 0;
      if (tid == 0) sm.lowest = 0xffffffffu, sm.highest = 0;
    }
    if (ranks > 1) cg::this_cluster().sync();
    else __syncthreads();

    if (rank == 0) {
      // lo and hi: at least `need` keys are >= lo, fewer >= hi.
      const int total = carried + n, seg = (total + kThreads - 1) / kThreads * 32;   // keys of a warp, neighbours
      const int at = warp * seg + lane;
      uint32_t reg[kPer], lowest = 0xffffffffu, highest = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        reg[i] = 0;
        if (i * 32 < seg && at + i * 32 < total) {
          reg[i] = sm.keys[at + i * 32];
          lowest = min(lowest, reg[i]);
          highest = max(highest, reg[i]);
        }
      }
      lowest = __reduce_min_sync(kFull, lowest);
      highest = __reduce_max_sync(kFull, highest);
      if (lane == 0) {
        atomicMin(&sm.lowest, lowest);
        atomicMax(&sm.highest, highest);
      }
      __syncthreads();
      uint32_t lo = sm.lowest, hi = sm.highest + 1;
      int at_least = total;   // keys >= lo
      for (int step = 0; at_least > v.need && hi - lo > 1; ++step) {
        const uint32_t mid = middle(lo, hi, step);
        int cnt = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (i * 32 >= seg) break;
          cnt += reg[i] >= mid;
        }
        cnt = __reduce_add_sync(kFull, cnt);
        if (lane == 0 && cnt) atomicAdd(&sm.counts[step % 3], cnt);
        if (tid == 0) sm.counts[(step + 1) % 3] = 0;   // read two steps ago
        __syncthreads();
        cnt = sm.counts[step % 3];
        if (cnt >= v.need) lo = mid, at_least = cnt;
        else hi = mid;
      }
      // Those above lo, and the first of its equals, in order.
      int gt = 0, eq = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (i * 32 >= seg) break;
        const bool in = at + i * 32 < total;
        gt += in && reg[i] > lo;
        eq += in && reg[i] == lo;
      }
      gt = __reduce_add_sync(kFull, gt);
      eq = __reduce_add_sync(kFull, eq);
      if (lane == 0) sm.above[warp] = gt, sm.equal[warp] = eq;
      __syncthreads();
      int all_gt = 0, gt0 = 0, eq0 = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) gt0 += sm.above[w], eq0 += sm.equal[w];
        all_gt += sm.above[w];
      }
      const int eq_max = min(total, v.need) - all_gt;    // equals that are taken
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (i * 32 >= seg) break;
        const bool in = at + i * 32 < total;
        const unsigned g = __ballot_sync(kFull, in && reg[i] > lo), e = __ballot_sync(kFull, in && reg[i] == lo);
        const unsigned below = (1u << lane) - 1;
        const int my_eq = eq0 + __popc(e & below);
        if (in && (reg[i] > lo || (reg[i] == lo && my_eq < eq_max))) {
          const int where = gt0 + __popc(g & below) + min(my_eq, eq_max), key = at + i * 32;
          const int blk = key < carried ? sm.best[side][key] : from + key - carried;
          if (last) {
            out[a.sink + where] = blk;
          } else {
            sm.best[side ^ 1][where] = blk;
            sm.best_key[side ^ 1][where] = reg[i];
          }
        }
        gt0 += __popc(g);
        eq0 += __popc(e);
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
  if (ranks > 1) cg::this_cluster().sync();     // all of them run before one writes to another
  pdl_wait();
  if (p.rows == 0) {
    const int t = item / Hk;
    const RowOwner own = row_owner(a.cu_q, a.kv_len, a.batch, a.total_q, a.max_q, cap, t);
    if (own.bad && threadIdx.x == 0 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
    if (own.b >= 0) select_row<D>(p, own, t, h, sm, rank, ranks);
    return;
  }
  // A request's rows, dealt out to `rows` CTAs.
  const RowOwner own = request_of(a.cu_q, a.kv_len, a.total_q, a.max_q, cap, item / Hk / p.rows);
  if (own.bad && threadIdx.x == 0 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
  if (own.b < 0 || own.n > kFewRows) return;
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

  // Cuts the list to at least `need` and at most `most` (>= need) entries, if it has more. Whole warps.
  __device__ __forceinline__ void cut(int need, int most) {
    uint32_t lo = 0xffffffffu, hi = 0;
    for (int i = 0; i < cnt; ++i) {
      const uint32_t k = key(i);
      lo = min(lo, k);
      hi = max(hi, k);
    }
    hi += 1;
    int at_least = cnt, above = 0;     // entries >= lo, >= hi
    const bool wanted = cnt > most && need > 0;
    for (int step = 0;; ++step) {
      const bool go = wanted && at_least > most && hi - lo > 1;
      if (!__any_sync(kFull, go)) break;
      const uint32_t mid = go ? middle(lo, hi, step) : 0xffffffffu;
      int c = 0;
#pragma unroll 8
      for (int i = 0; i < cnt; ++i) c += key(i) >= mid;
      if (go) {
        if (c >= need) lo = mid, at_least = c;
        else hi = mid, above = c;
      }
    }
    if (wanted) {
      int equals = at_least > most ? need - above : cnt;   // too many of one key: the first of them
      int w = 0;
      for (int i = 0; i < cnt; ++i) {
        const uint32_t k = key(i);
        if (k > lo || (k == lo && equals-- > 0)) {
          sm.key[w][row] = k;
          sm.blk[w][row] = sm.blk[i][row];
          ++w;
        }
      }
      cnt = w;
      bound = key_value(lo);
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kManyThreads) kv4_select_many_kernel(const __grid_constant__ SelectArgs p) {
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
      uint32_t top = 0;
      if (real)
        for (int i = 0; i < heads * D / 8; ++i) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(q) + i);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max(top, max(finite_bits(w[j]), finite_bits(w[j] >> 16)));
        }
      const float scale = grid_scale(top);
#pragma unroll 1
      for (int d0 = 0; d0 < D; d0 += 32) {
        float s[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = 0.0f;
        if (real)
          for (int g = 0; g < heads; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 x = __ldg(reinterpret_cast<const uint4*>(q + g * D + d0) + i);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                s[8 * i + 2 * j] += on_grid(w[j] & 0xffffu, scale);
                s[8 * i + 2 * j + 1] += on_grid(w[j] >> 16, scale);
              }
            }
        uint32_t r[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const __half2 x = __floats2half2_rn(s[2 * i], s[2 * i + 1]);
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
          if (__any_sync(kFull, list.cnt > kKeep)) list.cut(v.need, list.cnt > kKeep ? min(kKeep, v.need + 7) : kList);
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
  // CTAs for a query: as many as leave each a round of its warps' blocks at the longest, and the GPU not twice full.
  const long long most = (long long)p.a.max_pages * p.a.index.cache.page_tokens >> p.block_log;
  const int step = kWarps * (512 / D) * kAhead;
  int ranks = 1;
  while (ranks < 8 && items * ranks * 2 <= 2ll * sm_count() && most > (long long)step * ranks) ranks *= 2;
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
