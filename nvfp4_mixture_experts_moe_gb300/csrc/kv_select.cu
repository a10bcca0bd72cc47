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
// (query, head), bound by the latency of its steps (4 single tokens over 2048
// blocks, 8 heads x 128: 11.7 us, 2.5 by the means' bytes). More rows: 128
// queries of a head a CTA, a thread each, scores by tcgen05 in tensor memory
// (4096 rows over 1024 blocks, 32/8 heads x 128: 50 us, 5.6 by the queries'
// bytes): of a CTA's 75,000 cycles the queries take 11,000, a tile of 64 means
// some 1500 the first time it goes by (the hand-overs between its warps) and
// 2200 the second (the lists), the picks 4500.
#include <cooperative_groups.h>

#include <cfloat>
#include <type_traits>

#include "kernels.cuh"
#include "kv4.cuh"
#include "kv_lookup.cuh"
#include "kv_math.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;
using kv::kFull;
using kv::max_u16x2;
namespace cg = cooperative_groups;

constexpr int kFewRows = 8, kManyRows = 608, kManyRowsNarrow = 640;

// A float's bits in the order of its value (0 is below every key of a number).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k ^ ((int)k < 0 ? 0x80000000u : 0xffffffffu)); }

// The largest number that is less.
__device__ __forceinline__ float key_below(float x) {
  const uint32_t k = order_key(x) - 1;
  return key_value(k - (k == 0x7fffffffu));   // -0 is not less than 0
}

// A key between lo and hi (hi > lo + 1): half way between the values, or (odd
// steps, and where that is no key between) between the keys.
__device__ __forceinline__ uint32_t middle(uint32_t lo, uint32_t hi, int step) {
  const uint32_t k = order_key(0.5f * key_value(lo) + 0.5f * key_value(hi));
  return (step & 1) || k <= lo || k >= hi ? lo + (hi - lo) / 2 : k;
}

// What a block whose page is not in the pool scores (one whose mean is NaN too): below every sum.
constexpr float kBadScore = -FLT_MAX;
__device__ __forceinline__ float finite_score(float s) { return fminf(fmaxf(s, kBadScore), FLT_MAX); }

struct SelectArgs {
  moe_kv4_select_args a;
  int block_log;
  int rows;      // CTAs of a request (few queries); 0: of any row
  long long wait_limit;
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

// The page whose rows a block of several pages has: its first one's unless another block owns those; -1: one of the two
// is not in the pool.
__device__ __forceinline__ int row_page(int first, int last, int owner, int num_pages) {
  if (first < 0 || first >= num_pages || last < 0 || last >= num_pages) return -1;
  return owner < 0 || owner == last ? first : last;
}
__device__ __forceinline__ int owner_of(const moe_kv4_index& x, int page) {
  return page >= 0 && page < x.cache.num_pages ? __ldg(x.owners + page) : -1;
}

// Where the mean of block j of a request lies; -1: its page is not in the pool.
__device__ __forceinline__ int entry_of(const moe_kv4_index& x, int page_log, int block_log, const int32_t* table, int j) {
  const int tok = j << block_log, page = __ldg(table + (tok >> page_log));
  if (page_log < block_log)
    return row_page(page, __ldg(table + ((tok + (1 << block_log) - 1) >> page_log)), owner_of(x, page), x.cache.num_pages);
  if (page < 0 || page >= x.cache.num_pages) return -1;
  return (page << (page_log - block_log)) + ((tok & ((1 << page_log) - 1)) >> block_log);
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

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// ---------------------------------------------------------- few queries
// A warp scores 16 blocks with one chain of matrix products, the means coming
// straight from memory as A fragments and u being the only column of B; the
// CTAs of a cluster send their scores to the first. There a histogram of the
// scores' range finds how far down the best go, its few candidates are ranked
// by counting who is above them. All of it is short code: what is run once
// waits for its instructions as much as for its data.
constexpr int kThreads = 512, kWarps = kThreads / 32, kScores = 4096, kAhead = 1, kBins = 256, kCandidates = 256;

struct FewSmem {
  alignas(16) float score[kScores + kSparseTop];
  alignas(16) __half u[128];
  alignas(16) float cand[kCandidates];
  int cand_blk[kCandidates];
  int hist[kBins];
  int best[kSparseTop];                  // blocks that earlier chunks left, and their scores
  float best_score[kSparseTop];
  int taken[kCandidates], found;
  int bin, above;                        // the histogram's answer
  unsigned lowest, highest, group_top;
};

// The `need` largest of sm.score[0 .. total) to put(where, block, score), in the
// order of the blocks, the first of equal ones; all where there are no more. By
// a whole CTA.
template <class BlockOf, class Put>
__device__ __forceinline__ void best_scores(FewSmem& sm, int total, int need, BlockOf block_of, Put put) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // What counts: scores in [lo, hi], `above` more lie over hi and are in.
  float lo = -INFINITY, hi = INFINITY, from = 0.0f, scale = 0.0f;
  int above = 0, bin = 0;
  if (total > need) {
#pragma unroll 1
    while (true) {
      // the range of what counts: of the whole, then of one bin of it
      unsigned low = 0xffffffffu, high = 0;
      for (int i = tid; i < total; i += kThreads) {
        const float x = sm.score[i];
        if (x >= lo && x <= hi && (scale == 0.0f || min((int)((0.5f * x - from) * scale), kBins - 1) == bin)) {
          low = min(low, order_key(x));
          high = max(high, order_key(x));
        }
      }
      low = __reduce_min_sync(kFull, low);
      high = __reduce_max_sync(kFull, high);
      if (lane == 0) {
        atomicMin(&sm.lowest, low);
        atomicMax(&sm.highest, high);
      }
      if (tid < kBins) sm.hist[tid] = 0;
      __syncthreads();
      lo = key_value(sm.lowest);
      hi = key_value(sm.highest);
      if (lo == hi) break;   // all equal: the first of them
      from = 0.5f * lo;
      scale = (kBins - 1) / (0.5f * hi - from);
      for (int i = tid; i < total; i += kThreads) {
        const float x = sm.score[i];
        if (x >= lo && x <= hi) atomicAdd(&sm.hist[min((int)((0.5f * x - from) * scale), kBins - 1)], 1);
      }
      __syncthreads();
      if (tid == 0) sm.lowest = 0xffffffffu, sm.highest = 0;
      if (warp == 0) {
        // the highest bin with at least `need` scores in it and over it; a lane has eight bins, from the top
        int mine[kBins / 32], sum = 0;
#pragma unroll
        for (int i = 0; i < kBins / 32; ++i) {
          mine[i] = sm.hist[kBins - 1 - lane * (kBins / 32) - i];
          sum += mine[i];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(kFull, incl, o);
          if (lane >= o) incl += v;
        }
        int over = above + incl - sum;
        const unsigned reached = __ballot_sync(kFull, above + incl >= need);
        if (lane == __ffs(reached) - 1) {
          int i = 0;
#pragma unroll
          for (int k = 0; k < kBins / 32 - 1; ++k)
            if (i == k && over + mine[k] < need) over += mine[k], ++i;
          sm.bin = kBins - 1 - lane * (kBins / 32) - i;
          sm.above = over;
        }
      }
      __syncthreads();
      bin = sm.bin;
      above = sm.above;
      if (above + sm.hist[bin] <= kCandidates) break;
      __syncthreads();
    }
  }
  // The candidates, in any order: what is over the bin or in it; of many equal scores the first that are needed.
  const bool ties = total > need && lo == hi;
  if (tid == 0) sm.found = 0;
  __syncthreads();
  for (int i = tid; i < total; i += kThreads) {
    const float x = sm.score[i];
    bool in = total <= need || x > hi;
    if (!in && !ties && x >= lo) in = min((int)((0.5f * x - from) * scale), kBins - 1) >= bin;
    if (in) {
      const int at = atomicAdd(&sm.found, 1);
      sm.cand[at] = x;
      sm.cand_blk[at] = block_of(i);
    }
  }
  if (ties) {
    __syncthreads();
    if (warp == 0) {
      int at = sm.found;
#pragma unroll 1
      for (int i0 = 0; i0 < total && at < need; i0 += 32) {
        const bool equal = i0 + lane < total && sm.score[i0 + lane] == lo;
        const unsigned e = __ballot_sync(kFull, equal);
        const int mine = at + __popc(e & ((1u << lane) - 1));
        if (equal && mine < need) {
          sm.cand[mine] = lo;
          sm.cand_blk[mine] = block_of(i0 + lane);
        }
        at += __popc(e);
      }
      __syncwarp();
      if (lane == 0) sm.found = min(at, need);
    }
  }
  __syncthreads();
  // Who is among the best, and then how many of those are blocks before one's own.
  const int n = sm.found;
  bool in = false;
  int blk = 0;
  if (tid < n) {
    const float x = sm.cand[tid];
    blk = sm.cand_blk[tid];
    int over = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float y = sm.cand[j];
      over += y > x || (y == x && sm.cand_blk[j] < blk);
    }
    in = over < need;
    sm.taken[tid] = in ? blk : 0x7fffffff;
  }
  __syncthreads();
  if (in) {
    int where = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) where += sm.taken[j] < blk;
    put(where, blk, sm.cand[tid]);
  }
}

// One query and head, by a whole cluster.
template <int D>
__device__ __forceinline__ void select_row(const SelectArgs& p, const RowOwner& own, int t, int h, FewSmem& sm, int rank,
                                           int ranks) {
  constexpr int kStep = kWarps * 16 * kAhead;   // blocks that a CTA's warps take at once
  constexpr int kLoads = D / 32;                // 16-byte pieces of a lane's part of a row
  const moe_kv4_select_args& a = p.a;
  const moe_kv4_cache& c = a.index.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
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
  int entry[kAhead][2];
  uint4 w[kAhead][2][kLoads];
  // The means of the warp's blocks of a round, asked for before what multiplies them is there: rows g8 and g8 + 8 of each
  // 16 blocks, elements D / 4 t4 and on.
  auto load = [&](int from, int n, int j0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int j = j0 + i * kWarps * 16 + r * 8 + g8;
        entry[i][r] = j < n ? entry_of(a.index, page_log, p.block_log, table, from + j) : -2;
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4* m = reinterpret_cast<const uint4*>(a.index.means + ((size_t)max(entry[i][r], 0) * Hk + h) * D) + t4 * kLoads;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) w[i][r][k] = entry[i][r] >= 0 ? __ldg(m + k) : make_uint4(0u, 0u, 0u, 0u);
      }
  };
  const int first = rank * kStep + warp * 16;
  uint32_t x[kSparseGroup / 2];   // element tid of the group's queries, two a word
  if (tid < D) {
    const uint16_t* const q = a.q + (size_t)t * a.q_stride + (size_t)h * heads * D + tid;
#pragma unroll
    for (int i = 0; i < kSparseGroup / 2; ++i)
      x[i] = (2 * i < heads ? (uint32_t)q[2 * i * D] : 0u) | (2 * i + 1 < heads ? (uint32_t)q[(2 * i + 1) * D] << 16 : 0u);
  }
  load(v.c0, min(kScores, v.c1 - v.c0), first);
  if (tid == 0) sm.group_top = 0, sm.lowest = 0xffffffffu, sm.highest = 0;
  __syncthreads();
  if (tid < D) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kSparseGroup / 2; ++i) top = max(top, max(finite_bits(x[i]), finite_bits(x[i] >> 16)));
    top = __reduce_max_sync(kFull, top);
    if (lane == 0) atomicMax(&sm.group_top, top);
  }
  __syncthreads();
  if (tid < D) {
    const float scale = grid_scale(sm.group_top);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSparseGroup / 2; ++i) s += on_grid(x[i] & 0xffffu, scale) + on_grid(x[i] >> 16, scale);
    sm.u[tid] = __float2half_rn(s);
  }
  __syncthreads();
  int carried = 0;
  for (int from = v.c0; from < v.c1; from += kScores) {
    const int n = min(kScores, v.c1 - from);
    const bool last = from + n == v.c1;
#pragma unroll 1
    for (int j0 = first; j0 < n; j0 += ranks * kStep) {
      if (from > v.c0 || j0 > first) load(from, n, j0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const uint4 &x0 = w[i][0][k], &x1 = w[i][1][k];
          // u as the first column of B, the others 0; elements in the order the A fragments have them
          uint4 u = *reinterpret_cast<const uint4*>(sm.u + t4 * (D / 4) + k * 8);
          if (g8 > 0) u = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t lo[4] = {x0.x, x1.x, x0.y, x1.y}, hi[4] = {x0.z, x1.z, x0.w, x1.w};
          mma_f16_16816(s, lo, u.x, u.y);
          mma_f16_16816(s, hi, u.z, u.w);
        }
        if (t4 == 0)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int j = j0 + i * kWarps * 16 + r * 8 + g8;
            if (j < n) sm.score[carried + j] = entry[i][r] >= 0 ? finite_score(s[2 * r]) : kBadScore;
            if (entry[i][r] == -1 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
          }
      }
    }
    if (rank == 0 && tid < carried) sm.score[tid] = sm.best_score[tid];
    __syncthreads();
    if (ranks > 1) {
      if (rank > 0) {   // whole lines to the first CTA
        float* const to = cg::this_cluster().map_shared_rank(sm.score, 0) + carried;
        for (int j0 = rank * kStep; j0 < n; j0 += ranks * kStep)
          for (int j = j0 + tid; j < min(n, j0 + kStep); j += kThreads) to[j] = sm.score[carried + j];
      }
      cg::this_cluster().sync();
    }
    if (rank == 0)
      best_scores(sm, carried + n, v.need,
                  [&](int i) { return i < carried ? sm.best[i] : from + i - carried; },
                  [&](int where, int blk, float score) {
                    if (last) out[a.sink + where] = blk;
                    else sm.best[where] = blk, sm.best_score[where] = score;
                  });
    carried = min(carried + n, v.need);
    if (tid == 0) sm.lowest = 0xffffffffu, sm.highest = 0;
    if (ranks > 1) cg::this_cluster().sync();   // the first has read what the others wrote
    else __syncthreads();
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) kv4_select_few_kernel(const __grid_constant__ SelectArgs p) {
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
// Warps 0 to 3: a thread a query. Once u is in tensor memory (the A operand;
// warps 0 to 7 work it out, a row a warp, and hand it over in the lists'
// memory) the thread reads its row of each score tile. Warps 4 to 7 bring the
// means of 64 blocks a stage (cp.async into 128-byte-swizzled rows); one thread
// of warp 8 issues the products.
//
// The blocks go by twice. First only the maximum of each of 32 groups (every
// 32nd block) is kept, in registers: at least `need` blocks reach the need-th
// largest maximum, so only blocks that do can be among the best; of 1024 blocks
// and 13 picks about 17. The second time those go to a list. Going by once,
// with a bound that rises as lists of more than kKeep are cut, takes 79 us
// where this took 54 (over 64 blocks 34 and 23). For more than kSampled picks
// 64 groups are kept, in the lists' memory, if there are more blocks than
// kTwiceLong (once and twice, 48 picks of 1024: 244 and 179 us, of 300 100 and
// 91; 30 of 200 58 and 60); lists can still fill up then, and are cut at a
// value that leaves at least `need`.
//
// Runs of 256 rows (one CTA an SM, four stages) are slower by a tenth, though
// they load half as much; two threads a row with half a list each were slower
// by half.
constexpr int kRows = 128, kCols = 64, kStages = 2, kGroup = 32, kKeep = 64, kList = kKeep + kGroup;
constexpr int kLists = kRows / 32, kManyThreads = kRows + 160, kTmem = 256;
static_assert(kList % 16 == 0, "lists are read 16 entries at a time");
// Picks for which 32 groups will do; blocks that are worth a first pass for more of them.
constexpr int kSampled = 24, kTwiceLong = 256;
constexpr int kMostBlocks = 65536;   // list entries name blocks in 16 bits

template <int D>
struct ManySmem {
  alignas(1024) uint8_t ring[kStages][kCols * D * 2];
  float score[kList + 1][kRows];   // one place more: what is written there does not stay
  uint16_t blk[kList + 1][kRows];
  int warp_sum[kManyThreads / 32];
  int request, tile;             // what this CTA has: request, run of kRows of its rows
  int abort;
  uint32_t tmem;
  uint64_t full[kStages], empty[kStages], scored[2], read[2], rows_in, drained;
};

// The largest first: a bitonic network.
__device__ __forceinline__ void sort(float (&x)[kGroup]) {
#pragma unroll
  for (int lk = 1; lk <= 5; ++lk)
#pragma unroll
    for (int ld = 4; ld >= 0; --ld)
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
        if (ld < lk && !(i >> ld & 1)) {
          const float a = x[i], b = x[i | 1 << ld];
          const bool up = i >> lk & 1;
          x[i] = up ? fminf(a, b) : fmaxf(a, b);
          x[i | 1 << ld] = up ? fmaxf(a, b) : fminf(a, b);
        }
}

// A thread's list: cnt entries in the order of their blocks; what is past them
// is not above the bound.
template <class Sm>
struct List {
  Sm& sm;
  int row, cnt;
  float bound;     // at least `need` entries reach it: what comes later and is not above cannot win
  float top;       // no entry is above

  // Cuts a list of more than `most` entries to at least `need` and at most `most` (>= need). Whole warps, in step up to
  // the longest list.
  __device__ __forceinline__ void cut(int need, int most) {
    const bool wanted = cnt > most && need > 0;
    const int longest = (__reduce_max_sync(kFull, wanted ? cnt : 0) + 15) & ~15;
    uint32_t lo = order_key(fmaxf(bound, kBadScore)), hi = order_key(top) + 1;
    int at_least = cnt, above = 0;     // entries >= lo, >= hi
#pragma unroll 1
    for (int step = 0;; ++step) {
      const bool go = wanted && at_least > most && hi - lo > 1;
      if (!__any_sync(kFull, go)) break;
      const uint32_t key = go ? middle(lo, hi, step) : hi;
      const float mid = key_value(key);
      int c[2] = {0, 0};
#pragma unroll 1
      for (int i = 0; i < longest; i += 16) {
        float x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = sm.score[i + j][row];
#pragma unroll
        for (int j = 0; j < 16; ++j) c[j & 1] += x[j] >= mid;
      }
      if (go) {
        if (c[0] + c[1] >= need) lo = key, at_least = c[0] + c[1];
        else hi = key, above = c[0] + c[1];
      }
    }
    keep(wanted, longest, key_value(lo), at_least > most ? need - above : kList);   // too many of one score: the first of them
  }

  // Exactly `need` entries where there are more, of lists of up to kGroup: their order instead of a search.
  __device__ __forceinline__ void cut_short(int need) {
    const bool wanted = cnt > need && need > 0;
    float x[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) x[i] = sm.score[i][row];
    sort(x);
    float from = -INFINITY;
    int above = 0;
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (i < need) from = x[i];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) above += x[i] > from;
    keep(wanted, kGroup, from, need - above);
  }

  // What is above `from`, and the first `equals` entries equal to it.
  __device__ __forceinline__ void keep(bool wanted, int longest, float from, int equals) {
    int w = 0;
#pragma unroll 1
    for (int i = 0; i < longest; i += 16) {   // read ahead of what is written: w <= i
      float x[16];
      uint16_t blk[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        x[j] = sm.score[i + j][row];
        blk[j] = sm.blk[i + j][row];
      }
      if (wanted) {
#pragma unroll
        for (int j = 0; j < 16; ++j) sm.score[i + j][row] = -INFINITY;   // what is moved down is written again
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const bool equal = x[j] == from && i + j < cnt;
          if (x[j] > from || (equal && equals > 0)) {
            sm.score[w][row] = x[j];
            sm.blk[w][row] = blk[j];
            ++w;
          }
          equals -= equal;
        }
      }
    }
    if (wanted) {
      cnt = w;
      bound = from;
    }
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
  const int h = blockIdx.x % Hk, cap = a.max_pages * c.page_tokens;
  pdl_wait();
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 128);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.scored[i], 1);
      mbar_init(&sm.read[i], kRows);
    }
    mbar_init(&sm.rows_in, kRows);
    mbar_init(&sm.drained, 1);
    sm.request = -1;
    sm.abort = 0;
    fence_barrier_init();
  }
  // ------------------------------------------------- whose rows these are
  // The CTA's place among the runs of all requests that are this kernel's, by a scan over the lengths.
  int carry = blockIdx.x / Hk;   // runs before the CTA's, of this request and the ones after it
  for (int b0 = 0; b0 < a.batch && carry >= 0; b0 += kManyThreads) {
    int runs = 0;
    if (b0 + tid < a.batch) {
      const RowOwner r = request_of(a.cu_q, a.kv_len, a.total_q, a.max_q, cap, b0 + tid);
      if (r.bad && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
      if (r.b >= 0 && r.n > kFewRows) runs = (r.n + kRows - 1) / kRows;
    }
    int incl = runs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < kManyThreads / 32; ++w) {
      const int x = sm.warp_sum[w];
      if (w < warp) incl += x;
      all += x;
    }
    if (incl > carry && incl - runs <= carry) {
      sm.request = b0 + tid;
      sm.tile = carry - (incl - runs);
    }
    carry -= all;
    __syncthreads();
  }
  if (sm.request < 0) return;
  const RowOwner own = request_of(a.cu_q, a.kv_len, a.total_q, a.max_q, cap, sm.request);
  const int t0 = own.c0 + sm.tile * kRows, rows = min(kRows, own.c0 + own.n - t0);
  const int pos0 = own.kv - own.n + t0 - own.c0;       // the first row's position
  const int32_t* const table = a.block_table + (size_t)own.b * a.max_pages;
  // The last row ranks most blocks; where it ranks none, no row does.
  const Visible last = visible(a, p.block_log, pos0 + rows - 1);
  const int end = last.need > 0 ? last.c1 : 0;
  // whether the blocks go by twice
  const bool twice = last.need <= kSampled || end - a.sink > kTwiceLong;
  auto ranks = [&](int r) { return r < rows && visible(a, p.block_log, pos0 + r).need > 0; };
  Visible v = {0, 0, 0, 0};
  const int t = t0 + tid;
  if (tid < rows) {
    int32_t* const out = a.blocks + ((size_t)t * Hk + h) * a.top;
    v = visible(a, p.block_log, pos0 + tid);
    if (v.seen <= a.top) {
      for (int i = 0; i < a.top; ++i) out[i] = i < v.seen ? i : -1;
    } else {
      for (int i = 0; i < a.sink; ++i) out[i] = i;
      for (int i = 0; i < a.local; ++i) out[a.top - a.local + i] = v.c1 + i;
    }
  }
  if (last.need == 0) return;
  if (warp == kLists + 4) tmem_alloc(&sm.tmem, kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;   // two tiles of scores, then u
  constexpr int kU = 2 * kCols;
  volatile int* const abort = &sm.abort;

  // ----------------------------------------------- the rows of u, a row a warp
  constexpr int kRowLanes = D / 8, kPasses = 32 / kRowLanes;   // lanes of a head's row, heads at once
  constexpr int kPad = D * 2 + 16;                              // bytes of a row of u on its way to tensor memory
  static_assert(kPad * kRows <= (int)sizeof(sm.score), "u passes through the lists");
  uint8_t* const rows_of_u = reinterpret_cast<uint8_t*>(sm.score);
  if (warp < 8) {
    // kHeads of a lane at most, kRowsAtOnce rows asked for together
    auto work_out = [&](auto heads_of_lane, auto rows_at_once) {
      constexpr int kHeads = decltype(heads_of_lane)::value, kAtOnce = decltype(rows_at_once)::value;
      const int part = lane % kRowLanes, g0 = lane / kRowLanes;
#pragma unroll 1
      for (int r0 = warp * (kRows / 8); r0 < (warp + 1) * (kRows / 8); r0 += kAtOnce) {
        uint4 x[kAtOnce][kHeads];
#pragma unroll
        for (int b = 0; b < kAtOnce; ++b)
#pragma unroll
          for (int i = 0; i < kHeads; ++i) {
            const int g = g0 + i * kPasses;
            x[b][i] = g < heads && ranks(r0 + b)
                          ? __ldg(reinterpret_cast<const uint4*>(a.q + (size_t)(t0 + r0 + b) * a.q_stride +
                                                                 (size_t)(h * heads + g) * D + part * 8))
                          : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
        for (int b = 0; b < kAtOnce; ++b) {
          uint32_t pair = 0;
#pragma unroll
          for (int i = 0; i < kHeads; ++i) {
            pair = max_u16x2(max_u16x2(pair, x[b][i].x & 0x7fff7fffu), x[b][i].y & 0x7fff7fffu);
            pair = max_u16x2(max_u16x2(pair, x[b][i].z & 0x7fff7fffu), x[b][i].w & 0x7fff7fffu);
          }
          uint32_t top = __reduce_max_sync(kFull, max(pair & 0xffffu, pair >> 16));
          if (top >= 0x7f80u) {   // something counts as 0: the same for a whole warp
            pair = 0;
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
              uint32_t* const w = &x[b][i].x;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                w[j] = (finite_bits(w[j]) ? w[j] & 0xffffu : 0u) | (finite_bits(w[j] >> 16) ? w[j] & 0xffff0000u : 0u);
                pair = max_u16x2(pair, w[j] & 0x7fff7fffu);
              }
            }
            top = __reduce_max_sync(kFull, max(pair & 0xffffu, pair >> 16));
          }
          const uint32_t scale = __float_as_uint(grid_scale(top)) >> 16, scale2 = scale | scale << 16;
          // x scale + 192 in bf16 is 192 and the rounded product (at most 64), whose bits are 0x4300 + 64 + that; a
          // lane's missing heads add 64 as well
          uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < kHeads; ++i) {
            sum[0] += fma_bf16x2(x[b][i].x, scale2, 0x43404340u) - 0x43004300u;
            sum[1] += fma_bf16x2(x[b][i].y, scale2, 0x43404340u) - 0x43004300u;
            sum[2] += fma_bf16x2(x[b][i].z, scale2, 0x43404340u) - 0x43004300u;
            sum[3] += fma_bf16x2(x[b][i].w, scale2, 0x43404340u) - 0x43004300u;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int o = kRowLanes; o < 32; o <<= 1) sum[j] += __shfl_xor_sync(kFull, sum[j], o);
            constexpr float kZero = 64.0f * kHeads * kPasses;
            const __half2 y = __floats2half2_rn((float)(sum[j] & 0xffffu) - kZero, (float)(sum[j] >> 16) - kZero);
            sum[j] = *reinterpret_cast<const uint32_t*>(&y);
          }
          if (g0 == 0)
            *reinterpret_cast<uint4*>(rows_of_u + (r0 + b) * kPad + part * 16) = make_uint4(sum[0], sum[1], sum[2], sum[3]);
        }
      }
    };
    // as many rows as 32 registers hold
    if (heads <= 2 * kPasses) work_out(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
    else work_out(std::integral_constant<int, kSparseGroup / kPasses>{}, std::integral_constant<int, kPasses / 2>{});
  }
  __syncthreads();

  if (warp < kLists) {
    // ------------------------------------------------------------- queries
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += 32) {
      uint32_t r[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(rows_of_u + tid * kPad + d0 * 2 + i * 16);
        r[4 * i] = x.x, r[4 * i + 1] = x.y, r[4 * i + 2] = x.z, r[4 * i + 3] = x.w;
      }
      tmem_st16(tmem + lanes + kU + d0 / 2, r);
    }
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&sm.rows_in);
    // the lists' memory is the lists' once every query has its row
    asm volatile("bar.sync 1, %0;" ::"n"(kRows) : "memory");
    for (int i = 0; i < kList; ++i) sm.score[i][tid] = -INFINITY;
    List<Sm> list = {sm, tid, 0, -INFINITY, -INFINITY};
    int tile = 0;
    bool ok = true;
    const int c1 = v.need > 0 ? v.c1 : 0;
    // take(j, n, r): this row's scores of kGroup blocks from j on, of which it ranks n.
    auto every_score = [&](auto take) {
      for (int j0 = a.sink; j0 < end && ok; j0 += kCols, ++tile) {
        const int buf = tile & 1;
        ok = __all_sync(kFull, mbar_wait(&sm.scored[buf], tile >> 1 & 1, abort, p.wait_limit));
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
          const int j = j0 + g * kGroup;
          take(j, min(kGroup, c1 - j), r);
        }
      }
    };
    if (twice && last.need <= kSampled) {
      float best[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) best[i] = -INFINITY;
      every_score([&](int, int n, uint32_t (&r)[kGroup]) {
        if (__all_sync(kFull, n >= kGroup)) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i) best[i] = fmaxf(best[i], __uint_as_float(r[i]));
        } else {
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
            if (i < n) best[i] = fmaxf(best[i], __uint_as_float(r[i]));
        }
      });
      sort(best);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) sm.score[kKeep + i][tid] = best[i];
      float least = fminf(sm.score[kKeep + max(v.need, 1) - 1][tid], FLT_MAX);
      every_score([&](int j, int n, uint32_t (&r)[kGroup]) {
        uint32_t part[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          sm.score[kKeep + i][tid] = __uint_as_float(r[i]);
          if (__uint_as_float(r[i]) >= least) part[i & 3] |= 1u << i;
        }
        uint32_t reach = part[0] | part[1] | part[2] | part[3];
        if (least == -INFINITY) reach = ~0u;
        if (n < kGroup) reach &= n <= 0 ? 0u : (1u << n) - 1u;
        if (__any_sync(kFull, list.cnt + __popc(reach) > kKeep)) {
          const int before = list.cnt;
          list.cut(v.need, kKeep - kGroup);
          if (before > kKeep - kGroup) least = key_value(order_key(list.bound) + 1);
        }
        for (; reach; reach &= reach - 1) {
          const int i = __ffs((int)reach) - 1;
          const float s = finite_score(sm.score[kKeep + i][tid]);
          if (s >= least) {
            sm.score[list.cnt][tid] = s;
            sm.blk[list.cnt][tid] = (uint16_t)(j + i);
            ++list.cnt;
            list.top = fmaxf(list.top, s);
          }
        }
        __syncwarp();
      });
    } else {
      if (twice) {   // 64 groups
        every_score([&](int j, int n, uint32_t (&r)[kGroup]) {
          float(*const best)[kRows] = sm.score + ((j - a.sink) & kGroup);
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
            if (i < n) best[i][tid] = fmaxf(best[i][tid], __uint_as_float(r[i]));
        });
        list.cnt = 2 * kGroup;
        list.top = FLT_MAX;
        list.cut(v.need, v.need);
        // (NaN for a row that ranks nothing: nothing is above it)
        list.bound = key_below(fminf(list.bound, FLT_MAX));
        list.cnt = 0;
        list.top = -INFINITY;
        for (int i = 0; i < 2 * kGroup; ++i) sm.score[i][tid] = -INFINITY;
      }
      every_score([&](int j, int n, uint32_t (&r)[kGroup]) {
        // Every score is written behind the list, and stays if it is above: a branch for each column costs six times
        // as much.
        const bool whole = __all_sync(kFull, n >= kGroup);
        if (!whole)
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
            if (i >= n) r[i] = 0xff800000u;   // below every bound
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          const float s = finite_score(__uint_as_float(r[i]));
          sm.score[list.cnt][tid] = s;
          sm.blk[list.cnt][tid] = (uint16_t)(j + i);
          list.cnt += s > list.bound && (whole || i < n);
          list.top = fmaxf(list.top, s);
        }
        // One list too long: every list is cut that is much longer than it has to be.
        if (__any_sync(kFull, list.cnt > kKeep)) list.cut(v.need, min(kKeep, v.need + v.need / 2 + 8));
      });
    }
    // ------------------------------------------------- the best, in order
    if (__all_sync(kFull, list.cnt <= kGroup)) list.cut_short(v.need);
    else list.cut(v.need, v.need);
    if (v.need > 0) {
      int32_t* const out = a.blocks + ((size_t)t * Hk + h) * a.top + a.sink;
      for (int i = 0; i < v.need; ++i) out[i] = ok && i < list.cnt ? sm.blk[i][tid] : -1;
    }
  } else if (warp < kLists + 4) {
    // --------------------------------------------------------------- means
    // A thread has one 16-byte piece of kPieces rows, kEvery rows apart; the first 16 lanes look a warp's rows up, a tile
    // ahead.
    constexpr int kChunks = D / 8, kEvery = 128 / kChunks, kPieces = kCols / kEvery, kBeside = 32 / kChunks;
    const int me = tid - kRows, tiles = (end - a.sink + kCols - 1) / kCols, total = tiles << twice;
    const int ch = lane % kChunks, row0 = me / kChunks;
    const int looked_up = (me >> 5) * kBeside + lane % 16 % kBeside + lane % 16 / kBeside * kEvery;
    // K halves of 64 elements one after the other, rows of 128 bytes; kEvery is a multiple of a swizzle's 8 rows
    const uint32_t at = smem_u32(sm.ring[0]) + (uint32_t)(ch / 8 * (kCols * 128) + row0 * 128 + (((ch & 7) ^ (row0 & 7)) << 4));
    const uint16_t* const means = a.index.means + (size_t)h * D + ch * 8;
    const int per_page_log = max(page_log - p.block_log, 0);
    int tile = 0, done = 0;
    auto block_of = [&](int tile) { return a.sink + (tile < tiles ? tile : tile - tiles) * kCols + looked_up; };
    auto page_of = [&](int tile) {
      const int j = block_of(tile);
      return tile < total && j < end ? __ldg(table + ((j << p.block_log) >> page_log)) : 0;
    };
    // Blocks of several pages: their last pages, and who has the rows of the first ones, which are looked up a tile earlier.
    const bool spans = page_log < p.block_log;
    auto last_of = [&](int tile) {
      const int j = block_of(tile);
      return tile < total && j < end ? __ldg(table + ((((j + 1) << p.block_log) - 1) >> page_log)) : 0;
    };
    int page = page_of(0), last_page = 0, owner = 0, page1 = 0, last_page1 = 0;
    if (spans) {
      last_page = last_of(0);
      owner = owner_of(a.index, page);
      page1 = page_of(1);
      last_page1 = last_of(1);
    }
    for (; tile < total; ++tile) {
      const int stage = tile % kStages, j = block_of(tile);
      if (spans) page = row_page(page, last_page, owner, c.num_pages);
      const int mine = j >= end ? -2
                       : page < 0 || page >= c.num_pages ? -1
                                                         : (page << per_page_log) + (j & ((1 << per_page_log) - 1));
      if (spans) {
        page = page1;
        last_page = last_page1;
        owner = owner_of(a.index, page);
        page1 = page_of(tile + 2);
        last_page1 = last_of(tile + 2);
      } else {
        page = page_of(tile + 1);
      }
      if (!__all_sync(kFull, mbar_wait(&sm.empty[stage], (tile / kStages & 1) ^ 1, abort, p.wait_limit))) break;
      const uint32_t dst = at + stage * (uint32_t)sizeof(sm.ring[0]);
      int entry[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) entry[i] = __shfl_sync(kFull, mine, i * kBeside + lane / kChunks);
      if (!__any_sync(kFull, mine < 0)) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) cp_async_16(dst + i * kEvery * 128, means + (size_t)entry[i] * (Hk * D), 16u);
      } else {
#pragma unroll 1
        for (int i = 0; i < kPieces; ++i) {
          const int e = __shfl_sync(kFull, mine, i * kBeside + lane / kChunks);
          if (e == -1) {   // a page that is not in the pool: a row of NaN, which no mean is
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + i * kEvery * 128), "r"(0x7e007e00u) : "memory");
            if (a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
          } else {
            cp_async_16(dst + i * kEvery * 128, means + (size_t)max(e, 0) * (Hk * D), e >= 0 ? 16u : 0u);
          }
        }
      }
      cp_async_commit();
      if (tile - done == kStages - 1) {     // the first of the stages on their way is in
        cp_async_wait<kStages - 1>();
        fence_proxy_async_smem();
        mbar_arrive(&sm.full[done % kStages]);
        ++done;
      }
    }
    cp_async_wait_all();
    fence_proxy_async_smem();
    for (; done < tile; ++done) mbar_arrive(&sm.full[done % kStages]);
  } else {
    // ------------------------------------------------------------ products
    // The warp runs together, one lane issues (one lane on its own: 53 us); stages and tiles of scores by constants.
    const bool one = elect_one();
    static_assert(kStages == 2, "a stage a tile of scores");
    constexpr uint32_t idesc = idesc_f16(128, kCols, 0);
    const uint64_t ring = smem_desc(smem_u32(sm.ring[0]), 16, 1024, kSwizzle128B);
    const int total = (end - a.sink + kCols - 1) / kCols << twice;
    bool ok = __all_sync(kFull, mbar_wait(&sm.rows_in, 0, abort, p.wait_limit));
    tc_fence_after();
#pragma unroll 1
    for (int first = 0; first < total && ok; first += 2) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (first + b >= total || !ok) break;
        const uint32_t parity = first >> 1 & 1;
        ok = __all_sync(kFull, mbar_wait(&sm.full[b], parity, abort, p.wait_limit) &&
                                   mbar_wait(&sm.read[b], parity ^ 1, abort, p.wait_limit));
        if (!ok) break;
        tc_fence_after();
        if (one) {
          const uint64_t src = ring + (uint64_t)(b * (sizeof(sm.ring[0]) >> 4));
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_f16_tmem_a(tmem + b * kCols, tmem + kU + k * 8, src + (uint64_t)((k / 4 * (kCols * 128) + k % 4 * 32) >> 4),
                           idesc, k != 0);
          tc_commit(&sm.empty[b]);
          tc_commit(&sm.scored[b]);
        }
        __syncwarp();
      }
    }
    // What was issued is complete before tensor memory is given back (also after a wait that gave up).
    if (one) tc_commit(&sm.drained);
    const long long c0 = clock64();
    while (!mbar_try_wait(&sm.drained, 0) && clock64() - c0 < 4000000000ll) {
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kLists + 4) tmem_dealloc(tmem, kTmem);
  if (tid == 0 && sm.abort && a.device_status != nullptr) set_status(a.device_status, MOE_ERR_TIMEOUT);
}

template <int D>
cudaError_t launch_few(const SelectArgs& p, long long items, cudaStream_t s) {
  // CTAs for a query: as many as fit the GPU at once and have a round of blocks each where the table is full.
  const long long most = (long long)p.a.max_pages * p.a.index.cache.page_tokens >> p.block_log;
  constexpr int step = kWarps * 16 * kAhead;
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
  static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs an SM");
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(kv4_select_many_kernel<D>, smem, done);
  if (e != cudaSuccess) return e;
  // as many runs of kRows rows as the requests can have: each but its last is full, and holds more than kFewRows
  const long long full = p.a.total_q / kRows, part = p.a.total_q / (kFewRows + 1);
  const unsigned tiles = (unsigned)(full + (part < p.a.batch ? part : p.a.batch));
  return launch_ex(true, kv4_select_many_kernel<D>, dim3(tiles * p.a.index.cache.kv_heads),
                   dim3(kManyThreads), smem, s, p);
}

}  // namespace

moe_status launch_kv4_select(const moe_kv4_select_args& a, cudaStream_t s) {
  SelectArgs p;
  p.a = a;
  p.block_log = __builtin_ctz(a.index.block_tokens);
  p.wait_limit = debug_wait_limit();
  const int D = a.index.cache.head_dim, Hk = a.index.cache.kv_heads;
  // Lengths are on the device: a call that allows requests of more than
  // kFewRows rows launches both kernels, each skipping the other's. A CTA of
  // the first then has all rows of a request, as most requests will have one.
  const bool long_lists = ((long long)a.max_pages * a.index.cache.page_tokens >> p.block_log) > kMostBlocks;
  // Few rows go faster without it: two CTAs of the first kernel run on an SM, 608 are two waves of 152 SMs, more a third
  // (us of the first and the second for 76 and 80 rows of 8 heads x 128 over 151 blocks: 14.6 and 16.6, 18.2 and 16.9;
  // over 512 blocks 23.1 and 23.3, 28.8 and 23.5; x 64 over 151 blocks 12.3 and 16.1, 15.5 and 16.2, so that a third wave
  // begins before it does). Over tables of 2048 blocks and more the second is ahead from some 48 rows on (64 rows: 60 and
  // 52), but a table may be far from full.
  const bool many = a.max_q > kFewRows && (long long)a.total_q * Hk > (D == 64 ? kManyRowsNarrow : kManyRows) && !long_lists;
  p.rows = many ? 1 : a.max_q > kFewRows ? 0 : a.max_q;
  const long long items = (p.rows == 0 ? (long long)a.total_q : (long long)a.batch * p.rows) * Hk;
  cudaError_t e = D == 64 ? launch_few<64>(p, items, s) : launch_few<128>(p, items, s);
  if (e == cudaSuccess && many) e = D == 64 ? launch_many<64>(p, s) : launch_many<128>(p, s);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(many ? 2 : 1);
  return MOE_OK;
}

}  // namespace moe
