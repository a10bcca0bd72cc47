// Attention over the NVFP4 cache for many query rows (prompts, prompt chunks,
// long drafts): tcgen05 tiles of 2 x 128 query rows against 128 cached tokens.
//
// A row is one (token, query head) pair of a key/value head's group, so the
// heads of a group share every dequantised key and value. Mathematics as in
// kv_attention_decode.cu: rows as f16 times a power of two (exact), keys and
// values as e2m1 * e4m3 in f16 (exact), fp32 scores, p = 2^(s - m) rounded to
// f16, m 7 to 15 below the running maximum (log2), fp32 sums and output.
//
// Per CTA (one per SM):
// * four dequant warps, each two 16-token blocks of the tile: codes and scales
//   by plain loads a tile ahead, converted into 128-byte-swizzled shared-memory
//   tiles, keys K-major, values with d contiguous (MN-major); a scout warp has
//   looked up the pages and sent the blocks on their way into L2 before;
// * two threads issue S_i = Q_i K^T and O_i += P_i V, each for one of the two row
//   tiles i, in halves of 64 tokens, so that the softmax of one half runs under
//   the MMAs of the other; P_i (f16, read from tensor memory) lies in the
//   columns of the half of S_i it came from;
// * eight softmax warps, one row per thread: a half of S is read once; a half
//   whose maximum is more than 15 above m rescales O and the sum first, when
//   the halves before have gone into O (rare after the first).
//
// What bounds it: per 128 tokens and 256 rows at D = 128 the MMAs take 2048
// cycles at their rate (2560 with S in halves: Q is read twice), the
// exponentials 1024, and the softmax and dequant warps issue some 2000
// instructions per scheduler. A KV tile takes 4300: the tensor pipe is active in
// 62 % of the cycles (45 % at D = 64, where the MMAs are half) and instructions
// issue in 50 %, so neither is the limit but the chain between them: the two
// softmax warps of a scheduler each go through wait, load from tensor memory,
// maximum, vote, exponentials, store and arrive for a half of S, and what they
// leave uncovered the MMAs, which wait for P, do not fill. A 16384-token prompt
// of 32 heads over 8 runs at 1127 TFLOP/s (58 % of the measured matrix rate),
// one of 4096 tokens at 838: there each CTA enters and leaves three to five row
// tiles, 4-5 us each.
//
// Work is dealt out by KV tiles: all (request, head, row tile, KV tile) in
// order, one equal range per CTA. A row tile that two or more CTAs cut leaves
// fp32 partials and a note of them (at most one per CTA); a second, small
// launch joins them in order. (The last CTA to arrive doing it alone took 5 us
// per partial: 133 KB through one SM.)
//
// Short calls: lengths, the CTA's place in the work, pages, tiles and the
// join are one trip to memory after the other, 13 to 15 us in all.
#include "kernels.cuh"
#include "kv4.cuh"
#include "kv_tiles.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;
using namespace tiles;

constexpr int kTok = 128;              // cached tokens of a tile
constexpr int kHalfTok = kTok / 2;     // and of a half: what softmax and MMA warps hand each other
constexpr int kRowTile = 256;          // query rows of an item: two M = 128 tiles
constexpr int kChunk = 1024;           // requests of one launch
constexpr int kSoftWarps = 8, kDeqWarps = 4;
constexpr int kWarpBlocks = kTok / kKvBlock / kDeqWarps;
static_assert(kWarpBlocks == 2, "blocks of a dequant warp");
constexpr int kMmaWarp = kSoftWarps + kDeqWarps;   // and the one after it
constexpr int kScoutWarp = kMmaWarp + 2;
constexpr int kThreads = (kScoutWarp + 1) * 32;
// What starting and ending a row tile costs, in KV tiles. (us with 0, 1, 2, 3
// and 5, 32 heads over 8: a 4096-token prompt 211, 184, 163, 161, 165; four of
// 512 50, 41, 41, 39, 41; 16 requests of 1 to 181 new tokens on 3000 141, 139,
// 139, 140, 141.)
constexpr int kSetup = 2;
// Row tiles of up to this many rows are split over their KV tiles. (us split
// and not: 8 x 8 tokens over 16384, 32 rows, 103 and 117; 16 tokens over 16000,
// 64 rows, 26.6 and 28.7.)
constexpr int kSplitRows = 64;
constexpr int kTmemCols = 512;

// The row tile that begins in a CTA's range and goes on past it.
struct Cut {
  int row0, rows, h, q;   // first query row of the request, rows of the tile, head, index
  int n;                  // CTAs that hold a piece of it; 0: there is none
  int pad[3];
};

struct PromptArgs {
  moe_kv4_attn_args a;
  int b0, nb;
  int min_rows;        // requests with at most this many rows belong to another kernel
  int* status;
  Cut* cuts;           // [kKvMaxCtas]
  float* partials;     // [kKvMaxCtas][2][kRowTile x D, then (m, l) per row]
  long long wait_limit;
  // Launched right behind the few-row kernel of the same call: that one lets
  // this one start once everything before itself is done, and the two share
  // no memory, so this one waits for it only at its own end (whoever waits
  // for this kernel waits for both). A call of long and short requests then
  // uses the SMs that the first leaves idle.
  int overlap;
};

template <int D>
constexpr int kSlotFloats = kRowTile * (D + 2);
constexpr size_t kCutFloats = (size_t)kKvMaxCtas * sizeof(Cut) / sizeof(float);
static_assert(sizeof(Cut) == 32, "sectors");

struct Request {
  int row0, n, kv;
  bool bad;
};

__device__ __forceinline__ Request load_request(const moe_kv4_attn_args& a, int b) {
  Request r;
  const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), kv = __ldg(a.kv_len + b);
  r.row0 = c0;
  r.n = c1 - c0;
  r.kv = max(0, min(kv, a.max_pages * a.cache.page_tokens));
  r.bad = kv != r.kv;
  if (c0 < 0 || r.n < 0 || c1 > a.total_q || r.n > a.max_q) {
    r.n = 0;
    r.bad = true;
  }
  return r;
}

// First token that a request's row tile sees and number of its KV tiles (the
// first holds that token); at least one tile, so that rows that see nothing are
// written (as zeros) like any other.
__device__ __forceinline__ int row_tile_tiles(const moe_kv4_attn_args& a, const Request& r, int group, int q,
                                              int& seen) {
  const int rows = r.n * group;
  const int i0 = q * kRowTile / group, i1 = (min(rows, (q + 1) * kRowTile) - 1) / group;
  const int hi = a.causal ? max(0, r.kv - r.n + i1 + 1) : r.kv;
  seen = a.window > 0 ? max(0, r.kv - r.n + i0 - a.window + 1) : 0;
  return max(1, (hi + kTok - 1) / kTok - seen / kTok);
}

// Where a warp stands in its CTA's range, one (request, head, row tile) after
// another. The range counts units: a row tile's kSetup first units stand for
// its set-up and its end, then one unit per KV tile; a piece that holds only
// set-up units is passed over. Every warp walks the range for itself, in its
// own copy in shared memory, through two functions that are not inlined: the
// kernel's loops have to stay small, its warps run different code and share
// one instruction cache.
struct Walk {
  int row0, n, kv;  // the request
  int b, h, q;      // request (within the launch), head, row tile
  int x;            // linear index of the row tile's first unit
  int seen;         // first token that the row tile sees
  int tiles;        // KV tiles of the row tile
  int t0, t1;       // this piece's
  int more;         // 0 past the last piece
};

struct Range {
  const PromptArgs* p;
  const int* pre;   // units before each request
  int C0, C1;       // the CTA's
};

__device__ __noinline__ void walk_next(const Range& rg, Walk* w) {
  const moe_kv4_attn_args& a = rg.p->a;
  const int group = a.q_heads / a.cache.kv_heads;
  Request r = {w->row0, w->n, w->kv, false};
  int x = w->x, tiles = w->tiles, q = w->q, seen = 0, t1;
  do {
    x += tiles + kSetup;
    if (x >= rg.C1) {
      w->more = 0;
      return;
    }
    if ((long long)(++q) * kRowTile >= (long long)r.n * group) {
      q = 0;
      if (++w->h == a.cache.kv_heads) {
        w->h = 0;
        do ++w->b;
        while (rg.pre[w->b + 1] == rg.pre[w->b]);
        r = load_request(a, rg.p->b0 + w->b);
        w->row0 = r.row0;
        w->n = r.n;
        w->kv = r.kv;
      }
    }
    tiles = row_tile_tiles(a, r, group, q, seen);
    t1 = min(tiles, rg.C1 - x - kSetup);
  } while (t1 <= 0);
  w->x = x;
  w->q = q;
  w->seen = seen;
  w->tiles = tiles;
  w->t0 = 0;
  w->t1 = t1;
}

// All lanes together.
__device__ __noinline__ void walk_begin(const Range& rg, Walk* w) {
  const moe_kv4_attn_args& a = rg.p->a;
  const int lane = threadIdx.x & 31, group = a.q_heads / a.cache.kv_heads;
  int lo = 0, hi = rg.p->nb - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (rg.pre[mid] <= rg.C0) lo = mid;
    else hi = mid - 1;
  }
  const Request r = load_request(a, rg.p->b0 + lo);
  const int per_head = (rg.pre[lo + 1] - rg.pre[lo]) / a.cache.kv_heads;
  int rem = rg.C0 - rg.pre[lo];
  const int h = rem / per_head;
  rem -= h * per_head;
  int q = 0, f = 0, tiles;
  for (;; q += 32) {   // 32 row tiles at a time until the one that holds the unit
    const int v = (long long)(q + lane) * kRowTile < (long long)r.n * group
                      ? row_tile_tiles(a, r, group, q + lane, f) + kSetup
                      : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += u;
    }
    const unsigned past = __ballot_sync(kFull, incl > rem);
    if (past) {
      const int at = __ffs(past) - 1;
      rem -= __shfl_sync(kFull, incl - v, at);
      tiles = __shfl_sync(kFull, v, at) - kSetup;
      f = __shfl_sync(kFull, f, at);
      q += at;
      break;
    }
    rem -= __shfl_sync(kFull, incl, 31);
  }
  if (lane == 0) {
    const int x = rg.C0 - rem, t0 = max(0, rem - kSetup), t1 = min(tiles, rg.C1 - x - kSetup);
    *w = {r.row0, r.n, r.kv, lo, h, q, x, f, tiles, t0, t1, 1};
    if (t1 <= t0) walk_next(rg, w);
  }
  __syncwarp();
}

// A 16-token block of a tile to come: where it lies, its tokens that may be
// used. The others enter as zeros; a key before `from` enters as it is, its
// score is not used.
struct Place {
  const uint8_t* src;
  int from, to;     // to < 0: the block's page is bad
};
constexpr int kPlaces = 8;             // tiles looked up ahead

template <int D>
struct Smem {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * 128 * 128;   // 128 rows x D f16
  alignas(1024) uint8_t q[2][kTile];
  alignas(1024) uint8_t kv[2][2][kTile];   // keys, values: two stages each
  uint64_t q_full[2], q_split;         // rows of the streams' row tiles, of a split one
  uint64_t s_full[2][2], p_full[2][2];   // [stream][half]
  uint64_t pv_done[2], o_full[2];      // a half of a stream has gone into O, the last one of a row tile
  uint64_t kv_full[2][2], kv_empty[2][2];   // [keys or values][stage]
  uint64_t x_full, x_empty;            // the second warpgroup's half of a split row tile
  uint64_t drain;
  float2 x_ml[kSplitRows];             // (m, l) of its rows; its output lies in q[1]
  alignas(8) uint8_t hole[4][8];       // blocks of a tile whose page is bad
  int pre[kChunk + 1];                 // units (over all heads and row tiles) before each request
  Walk walk[kThreads / 32];
  alignas(16) Place place[kPlaces][kTok / kKvBlock];
  int place_more[kPlaces];             // 0: the range ends before this tile
  uint64_t place_full[kPlaces], place_empty[kPlaces];
  uint32_t tmem_base;
  int abort;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_prompt_kernel(const __grid_constant__ PromptArgs p) {
  using L = Kv4Block<D>;
  using Sm = Smem<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Sm* sm = reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const moe_kv4_attn_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hk = a.cache.kv_heads, group = a.q_heads / Hk;

  // ------------------------------------------------ units before each request
  if (tid == 0) {
    sm->abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->q_full[i], 4);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sm->s_full[i][h], 1);
        mbar_init(&sm->p_full[i][h], 4);
      }
      mbar_init(&sm->pv_done[i], 1);
      mbar_init(&sm->o_full[i], 1);
      mbar_init(&sm->kv_full[0][i], kDeqWarps);
      mbar_init(&sm->kv_full[1][i], kDeqWarps);
      mbar_init(&sm->kv_empty[0][i], 2);
      mbar_init(&sm->kv_empty[1][i], 2);
    }
    for (int i = 0; i < kPlaces; ++i) {
      mbar_init(&sm->place_full[i], 1);
      mbar_init(&sm->place_empty[i], kDeqWarps);
    }
    mbar_init(&sm->q_split, 4);
    mbar_init(&sm->x_full, 4);
    mbar_init(&sm->x_empty, 4);
    mbar_init(&sm->drain, 2);
    fence_barrier_init();
  }
  if (!p.overlap) pdl_wait();
  pdl_trigger();
  for (int b = warp; b < p.nb; b += kThreads / 32) {   // a warp per request
    const Request r = load_request(a, p.b0 + b);
    const long long rows = (long long)r.n * group;
    int sum = 0;
    if (rows > p.min_rows)
      for (int q = lane; (long long)q * kRowTile < rows; q += 32) {
        int f;
        sum += row_tile_tiles(a, r, group, q, f) + kSetup;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) {
      sm->pre[b + 1] = sum * Hk;
      if (r.bad && blockIdx.x == 0) set_status(p.status, MOE_ERR_DEVICE);
    }
  }
  __syncthreads();
  if (warp == 0) {
    long long carry = 0;
    for (int base = 0; base < p.nb; base += 32) {
      const int i = base + lane;
      long long v = i < p.nb ? sm->pre[i + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
      }
      if (i < p.nb) sm->pre[i + 1] = (int)(v + carry);
      carry += __shfl_sync(kFull, v, 31);
    }
    if (lane == 0) {
      sm->pre[0] = 0;
      // Past what the host checked: requests that share rows. None is served.
      if (carry > 0x7fffffff) {
        sm->pre[p.nb] = 0;
        set_status(p.status, MOE_ERR_DEVICE);
      }
    }
  }
  __syncthreads();
  const int total = sm->pre[p.nb];
  const int G = min((int)gridDim.x, total), cta = blockIdx.x;
  if (cta >= G) {
    if (tid == 0) p.cuts[cta].n = 0;
    if (p.overlap) pdl_wait();
    return;
  }
  const Range rg = {&p, sm->pre, mul_div(total, cta, G), mul_div(total, cta + 1, G)};
  if (warp == kMmaWarp) tmem_alloc(&sm->tmem_base, kTmemCols);
  Walk* const w = &sm->walk[warp];
  walk_begin(rg, w);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  volatile int* abort = &sm->abort;
  auto slot = [&](int c, int which) { return p.partials + ((size_t)c * 2 + which) * kSlotFloats<D>; };
  auto wait = [&](uint64_t* bar, int phase) {   // all lanes: the warp's common answer
    return __all_sync(kFull, mbar_wait(bar, (uint32_t)(phase & 1), abort, p.wait_limit)) != 0;
  };
  auto next = [&]() {                           // the warp's next piece
    __syncwarp();
    if (lane == 0) walk_next(rg, w);
    __syncwarp();
  };
  auto cta_of = [&](int unit) { return mul_div(unit + 1, G, total, -1); };

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------- softmax
    const int i = warp >> 2;                       // row tile of this warpgroup
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + lanes + 128 * i, o_t = tmem + lanes + 256 + 128 * i;
    int js = 0, jo = 0, jx = 0;                    // S tiles, items, split items this warpgroup has seen
    int jt = 0;                                    // tiles of the CTA before the next piece
    struct Item {
      // A row tile of few rows is split: both warpgroups hold all its rows and
      // take every other KV tile, joined at the end.
      bool split, real, active, whole;             // real: this thread's row exists, active: one of the warp's does
      int r, t0, nt, jt0, tok0, hi_tok, lo_tok;    // row within the tile; its KV tiles here; first token; what it sees
      size_t at;                                   // (token, head) of the row
      float c;                                     // from S to scores in powers of two
    };
    // The warpgroup's next row tile: its rows as f16 into shared memory, the
    // largest element in [2^14, 2^15) (smaller only below 2^-112).
    bool moved = true;                             // the walk stands behind the row tile entered last
    auto move_on = [&]() {
      if (!moved) next();
      moved = true;
    };
    auto enter = [&](Item& it) {
      for (move_on(); w->more; next()) {
        const int q0 = w->q * kRowTile, rows = min(kRowTile, w->n * group - q0), h = w->h, kv = w->kv;
        it.split = rows <= kSplitRows;
        it.jt0 = jt;
        it.t0 = w->t0;
        it.nt = w->t1 - w->t0;
        jt += it.nt;
        if (!it.split && i * 128 >= rows) continue;
        it.whole = it.nt == w->tiles;
        it.r = (it.split ? 0 : i * 128) + (warp & 3) * 32 + lane;
        it.real = it.r < rows;
        it.active = it.r - lane < rows;
        const int rr = q0 + (it.real ? it.r : 0), token = rr / group, qh = h * group + rr - token * group;
        it.at = (size_t)(w->row0 + token) * a.q_heads + qh;
        it.hi_tok = a.causal ? kv - w->n + token : kv - 1;
        it.lo_tok = a.window > 0 ? it.hi_tok - a.window + 1 : 0;
        it.tok0 = w->seen / kTok * kTok + it.t0 * kTok;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (size_t)(w->row0 + token) * a.q_stride + qh * D);
        // A row's 16-byte chunks come by neighbouring lanes (a row per thread
        // would fetch every sector twice and took 5 us a tile), each thread
        // then works on its own row in shared memory. The second warpgroup of
        // a split tile needs its rows' factors only.
        constexpr int kChunks = D / 8, kRows = 32 / kChunks;
        uint8_t* tile = &sm->q[i][0];
        const uint32_t dst = smem_u32(tile);
        const bool keep = !it.split || i == 0;
        // (With no tile of its own it goes straight to its empty half, which it
        // writes over these rows: nothing to fetch.)
        if (keep || it.nt > 1) {
          uint4 raw[kChunks];
#pragma unroll
          for (int v = 0; v < kChunks; ++v)
            raw[v] = __ldg(reinterpret_cast<const uint4*>(__shfl_sync(
                               kFull, reinterpret_cast<unsigned long long>(src), v * kRows + lane / kChunks)) + lane % kChunks);
#pragma unroll
          for (int v = 0; v < kChunks; ++v)
            sts16(dst + tile_chunk<>((warp & 3) * 32 + v * kRows + lane / kChunks, lane % kChunks), raw[v]);
          __syncwarp();
        }
        uint32_t mx = 0;
#pragma unroll
        for (int v = 0; v < kChunks; ++v) {
          const uint4 x = *reinterpret_cast<const uint4*>(tile + tile_chunk<>(it.r & 127, v));
          mx = max_u16x2(max_u16x2(mx, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
          mx = max_u16x2(max_u16x2(mx, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
        }
        const uint32_t big = max(mx & 0xffffu, mx >> 16);
        const int ex = min(max((int)(big >> 7), 15), 254);
        // never 0, so that a hidden score stays -inf
        it.c = fmaxf(fabsf(a.scale) * kLog2e / a.cache.k_gs * pow2(ex - 141), 1e-37f);
        // a larger score is a larger product; a row with a NaN or an infinity has no softmax whatever it sees: all NaN
        const float up = big >= 0x7f80u ? __int_as_float(0x7fffffff) : a.scale < 0.0f ? -pow2(141 - ex) : pow2(141 - ex);
        if (keep) {
#pragma unroll 4
          for (int v = 0; v < D / 8; ++v) {
            uint4* chunk = reinterpret_cast<uint4*>(tile + tile_chunk<>(it.r & 127, v));
            uint4 x = *chunk;
            uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              xw[j] = pack_f16x2(__uint_as_float(xw[j] << 16) * up, __uint_as_float(xw[j] & 0xffff0000u) * up);
            *chunk = x;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(it.split ? &sm->q_split : &sm->q_full[i]);
        }
        moved = false;
        return true;
      }
      return false;
    };
    Item it, done;
    done.split = false;
    bool pending = false, have = false, ok = true;
    float m = 0.0f, l = 0.0f;
    for (;;) {
      // Write out the row tile that is done and enter the next one: the next
      // one first, so that its first S runs under the writing, unless the rows
      // of the one that is done are still in use (a split one's by the other
      // stream).
#pragma unroll 1
      for (int pass = 0; pass < 2 && ok; ++pass) {
        if ((pass == 0) != done.split) {
          have = enter(it);
          continue;
        }
        if (!pending) continue;
        const int begin = done.split ? i : 0;
        const bool any = begin < done.nt;            // the second half of a split tile may be empty
        if (any && !(ok = wait(&sm->o_full[i], jo++))) break;
        tc_fence_after();
        float* xo = reinterpret_cast<float*>(&sm->q[1][0]);   // a split tile's second half goes through here
        float own = 1.0f, other = 0.0f;              // factors of this half and of the other
        if (done.split && i == 0) {
          if (!(ok = wait(&sm->x_full, jx++))) break;
          if (done.active) {
            const float2 x = sm->x_ml[done.r];
            const float mn = fmaxf(m, x.x), mu = mn == -INFINITY ? 0.0f : mn;
            own = ex2(m - mu);
            other = ex2(x.x - mu);
            l = l * own + x.y * other;
            m = mn;
          }
        }
        if (done.active) {
          const bool give = done.split && i == 1, final = !give && done.whole;
          if (final) {
            // 0: a row that sees nothing; NaN: a bad query's row, which stays NaN
            const float inv = l == 0.0f ? 0.0f : 1.0f / (l * a.cache.v_gs);
            own *= inv;
            other *= inv;
          }
          const bool blank = give ? !any : final && l == 0.0f;   // O holds nothing to read
          const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
          const int which = done.t0 > 0 ? 0 : 1, swz = give ? done.r & (D / 4 - 1) : 0;
          float* dst = give ? xo + done.r * D : slot(cta, which) + (size_t)done.r * D;
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t o[32];
            tmem_ld32(o_t + cc, o);
            ld_wait(o);
            float f[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = blank ? 0.0f : __uint_as_float(o[e]) * own;
            if (done.split && i == 0) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {   // 16-byte chunks swizzled by the row
                const float4 x = *reinterpret_cast<const float4*>(
                    xo + done.r * D + (((cc + e) / 4) ^ (done.r & (D / 4 - 1))) * 4);
                f[e] += x.x * other;
                f[e + 1] += x.y * other;
                f[e + 2] += x.z * other;
                f[e + 3] += x.w * other;
              }
            }
            if (!give && !done.real) continue;
            if (final) {
              uint16_t* out = a.out + done.at * D + cc;
#pragma unroll
              for (int e = 0; e < 32; e += 16) {
                uint32_t b[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) b[k] = float2_to_bf16x2_bits(f[e + 2 * k], f[e + 2 * k + 1]);
                if (wide) {   // a whole sector per thread
                  stg_v8(out + e, b);
                } else {
                  reinterpret_cast<uint4*>(out + e)[0] = make_uint4(b[0], b[1], b[2], b[3]);
                  reinterpret_cast<uint4*>(out + e)[1] = make_uint4(b[4], b[5], b[6], b[7]);
                }
              }
            } else if (give) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(dst + (((cc + e) / 4) ^ swz) * 4) =
                    make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t b[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) b[k] = __float_as_uint(f[e + k]);
                stg_v8(dst + cc + e, b);
              }
            }
          }
          if (give) sm->x_ml[done.r] = make_float2(m, l);
          else if (done.real && !final)
            *reinterpret_cast<float2*>(slot(cta, which) + kRowTile * D + 2 * done.r) = make_float2(m, l);
          else if (done.real && a.lse != nullptr) a.lse[done.at] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
        }
        tc_fence_before();
        if (done.split) {
          __syncwarp();
          if (lane == 0) mbar_arrive(i == 1 ? &sm->x_full : &sm->x_empty);
          if (i == 1 && !(ok = wait(&sm->x_empty, jx++))) break;
        }
      }
      if (!ok || !have) break;
      const int nt = it.nt, hi_tok = it.hi_tok, lo_tok = it.lo_tok;
      const float c = it.c;
      const bool active = it.active;
      m = -INFINITY;
      uint64_t l2 = pack2(0.0f, 0.0f);
      const uint64_t c2 = pack2(c, c);
      const int step = it.split ? 2 : 1, begin = it.split ? i : 0;
      for (int t = begin; t < nt && ok; t += step, ++js) {
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (!(ok = wait(&sm->s_full[i][half], js))) break;
          tc_fence_after();
          const int tok0 = it.tok0 + t * kTok + half * kHalfTok;
          const uint32_t hole = *reinterpret_cast<const volatile uint32_t*>(&sm->hole[(it.jt0 + t) & 3][4 * half]);
          const bool masked = __any_sync(kFull, tok0 + kHalfTok - 1 > hi_tok || tok0 < lo_tok) || hole != 0;
          if (active) {
            const uint32_t s_h = s_t + kHalfTok * half;
            uint32_t s0[32], s1[32];
            tmem_ld32(s_h, s0);
            tmem_ld32(s_h + 32, s1);
            ld_wait(s0);
            ld_wait(s1);
            // 32 columns: those that are not seen go to -inf; the largest score
            auto peak = [&](uint32_t (&sr)[32], int piece) {
              if (masked) {   // bit e: column e is seen
                const int hi = hi_tok - tok0 - 32 * piece, lo = lo_tok - tok0 - 32 * piece;
                uint32_t see = hi >= 31 ? ~0u : hi < 0 ? 0u : (2u << hi) - 1u;
                see &= lo <= 0 ? ~0u : lo > 31 ? 0u : ~0u << lo;
                const uint32_t bad = hole >> (16 * piece);
                if (bad & 0xffu) see &= 0xffff0000u;
                if (bad & 0xff00u) see &= 0x0000ffffu;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(see >> e & 1u)) sr[e] = 0xff800000u;
              }
              float u0 = __uint_as_float(sr[0]), u1 = __uint_as_float(sr[1]);
#pragma unroll
              for (int e = 2; e < 30; e += 4) {
                u0 = max3(u0, __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]));
                u1 = max3(u1, __uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3]));
              }
              return max3(u0, u1, fmaxf(__uint_as_float(sr[30]), __uint_as_float(sr[31])));
            };
            const float p0 = peak(s0, 0), p1 = peak(s1, 1), top = fmaxf(p0, p1) * c;
            if (__any_sync(kFull, top > m + kSlack)) {
              const float mn = fmaxf(m, top - kLead), f = mn == -INFINITY ? 1.0f : ex2(m - mn);
              m = mn;
              const float2 l = unpack2(l2);
              l2 = pack2(l.x * f, l.y * f);
              if (t > begin || half > 0) {   // O holds the halves before, once the last of them has gone in
                if (!(ok = wait(&sm->pv_done[i], 2 * js + half - 1))) break;
                tc_fence_after();
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 16) {
                  uint32_t o[16];
                  tmem_ld16(o_t + cc, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st16(o_t + cc, o);
                }
              }
            }
            const float mu = m == -INFINITY ? 0.0f : m;
            const uint64_t m2 = pack2(-mu, -mu);
            auto exps = [&](const uint32_t (&sr)[32], int piece) {
              uint32_t pk[16];
              uint64_t sum = pack2(0.0f, 0.0f);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 y = unpack2(fma2(pack2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), c2, m2));
                const float p0 = ex2(y.x), p1 = ex2(y.y);
                sum = add2(sum, pack2(p0, p1));
                pk[e] = pack_f16x2(p0, p1);
              }
              l2 = add2(l2, sum);
              tmem_st16(s_h + 16 * piece, pk);   // P takes the columns of S, read by then
            };
            exps(s0, 0);
            exps(s1, 1);
            tmem_st_wait();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->p_full[i][half]);
          move_on();                               // while S is under way
        }
        if (!ok) break;
      }
      if (!ok) break;
      l = unpack2(l2).x + unpack2(l2).y;
      done = it;
      pending = true;
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------- dequant
    const int blk0 = (warp - kSoftWarps) * kWarpBlocks;   // this warp's 16-token blocks of every tile
    constexpr int kLoads = D / 64;                 // 16-byte code loads per lane for a block's keys
    // This lane's 16-byte chunk of a row's codes (32 elements) and its row
    // within a load. Eight neighbouring lanes take two neighbouring chunks of
    // four rows: their 16-byte stores to the swizzled tile hit different banks.
    const int cl = (lane & 1) + (D == 128 ? lane >> 4 << 1 : 0), tl = D == 128 ? lane >> 1 & 7 : lane >> 1;
    constexpr int kRowsPerLoad = D == 128 ? 8 : 16;
    uint32_t off[4];                               // of this lane's four 16-byte stores, in a tile
#pragma unroll
    for (int j = 0; j < 4; ++j) off[j] = tile_chunk<>(tl, 4 * cl + j);
    struct Raw {
      uint4 codes[kWarpBlocks][kLoads];
      uint32_t sf[kWarpBlocks][kLoads];            // two scale bytes each
    } rk, rv;
    auto load = [&](Raw& r, int j, int at) {       // keys (at 0) or values of tile j
      const int cat = at + tl * L::kCodeRow + 16 * cl, sat = at + L::kKeyScales + tl * L::kScaleRow + 2 * cl;
#pragma unroll
      for (int x = 0; x < kWarpBlocks; ++x) {
        const Place pl = sm->place[j & (kPlaces - 1)][blk0 + x];
#pragma unroll
        for (int y = 0; y < kLoads; ++y) {
          r.codes[x][y] = make_uint4(0u, 0u, 0u, 0u);   // what may not have been appended enters as zeros
          r.sf[x][y] = 0u;
          if (y * kRowsPerLoad + tl < pl.to && (at == 0 || y * kRowsPerLoad + tl >= pl.from)) {
            r.codes[x][y] = __ldg(reinterpret_cast<const uint4*>(pl.src + cat + y * kRowsPerLoad * L::kCodeRow));
            r.sf[x][y] = __ldg(reinterpret_cast<const uint16_t*>(pl.src + sat + y * kRowsPerLoad * L::kScaleRow));
          }
        }
      }
    };
    auto store = [&](uint32_t tile, const Raw& r) {
#pragma unroll
      for (int x = 0; x < kWarpBlocks; ++x)
#pragma unroll
        for (int y = 0; y < kLoads; ++y) {
          const uint32_t at = tile + ((blk0 + x) * kKvBlock + y * kRowsPerLoad) * 128;
          const uint32_t two = cvt_e4m3x2_f16x2(r.sf[x][y]);
          const uint32_t sc0 = __byte_perm(two, 0, 0x1010), sc1 = __byte_perm(two, 0, 0x3232);
          const uint32_t wd[4] = {r.codes[x][y].x, r.codes[x][y].y, r.codes[x][y].z, r.codes[x][y].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t f[4];
            cvt_e2m1x8_f16(wd[j], f);
            const uint32_t sc = j < 2 ? sc0 : sc1;
            sts16(at + off[j],
                  make_uint4(hmul2_u32(f[0], sc), hmul2_u32(f[1], sc), hmul2_u32(f[2], sc), hmul2_u32(f[3], sc)));
          }
        }
    };
    // A tile's data are read one tile before they are converted, and the keys
    // go one tile ahead of the values: a stage of values is free only after
    // the softmax of the tile two before, a stage of keys already before it.
    auto place = [&](int j) {                      // whether there is a tile j
      return wait(&sm->place_full[j & (kPlaces - 1)], j / kPlaces) && sm->place_more[j & (kPlaces - 1)] != 0;
    };
    auto keys = [&](int j) {
      if (!wait(&sm->kv_empty[0][j & 1], (j >> 1) ^ 1)) return false;
      if (lane < kWarpBlocks)
        sm->hole[j & 3][blk0 + lane] = sm->place[j & (kPlaces - 1)][blk0 + lane].to < 0 ? 0xff : 0;
      store(smem_u32(&sm->kv[0][j & 1][0]), rk);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->kv_full[0][j & 1]);
      return true;
    };
    bool have = place(0), ahead = false, ok = true;   // tiles j and j + 1 exist
    if (have) {
      load(rk, 0, 0);
      load(rv, 0, L::kValueCodes);
    }
    for (int j = -1; have && ok; ++j) {
      if ((j < 0 || ahead) && !(ok = keys(j + 1))) break;
      const bool more = (j < 0 || ahead) && place(j + 2);
      if (more) load(rk, j + 2, 0);
      if (j >= 0) {
        const int s = j & 1;
        if (!wait(&sm->kv_empty[1][s], (j >> 1) ^ 1)) break;
        store(smem_u32(&sm->kv[1][s][0]), rv);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->kv_full[1][s]);
        have = ahead;
        if (have) load(rv, j + 1, L::kValueCodes);
      }
      if (have) {   // tile j + 1 is converted or in registers
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->place_empty[(j + 1) & (kPlaces - 1)]);
      }
      ahead = more;
    }
  } else if (warp == kScoutWarp) {
    // --------------------------------------------------------------- scout
    // Walks up to kPlaces tiles ahead of the conversion: a lane per block reads
    // the page ids and starts the blocks' way into L2, so that the dequant
    // warps' loads wait neither for the tables nor for memory.
    const int P = a.cache.page_tokens, p_log = __ffs(P) - 1;
    for (int j = 0, lt = w->t0;; ++j) {
      const int here = j & (kPlaces - 1), more = w->more;
      if (!wait(&sm->place_empty[here], (j / kPlaces) ^ 1)) break;
      if (more && lane < kTok / kKvBlock) {
        const int tok = w->seen / kTok * kTok + lt * kTok + lane * kKvBlock;
        // not past the end, nor before every row's window: pages there may have been given back
        Place pl = {nullptr, w->seen - tok, w->kv - tok};
        if (pl.from >= kKvBlock || pl.to < 0) pl.to = 0;
        if (pl.to > 0) {
          const int page = __ldg(a.block_table + (size_t)(p.b0 + w->b) * a.max_pages + (tok >> p_log));
          if (page >= 0 && page < a.cache.num_pages) {
            pl.src = static_cast<const uint8_t*>(a.cache.pool) +
                     kv4_block_offset(page, w->h, Hk, P / kKvBlock, (tok & (P - 1)) / kKvBlock, L::kBytes);
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(pl.src), "r"((uint32_t)L::kBytes) : "memory");
          } else {
            pl.to = -1;
            set_status(p.status, MOE_ERR_DEVICE);
          }
        }
        sm->place[here][lane] = pl;
      }
      if (lane == 0) sm->place_more[here] = more;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->place_full[here]);
      if (!more) break;
      if (++lt == w->t1) {
        next();
        lt = 0;
        if (w->more) {   // the next row tile's queries
          const int r0 = w->q * kRowTile, r1 = min(r0 + kRowTile, w->n * group);
          for (int token = r0 / group + lane; token * group < r1; token += 32)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             a.q + (size_t)(w->row0 + token) * a.q_stride + (size_t)w->h * group * D),
                         "r"((uint32_t)(group * D * 2))
                         : "memory");
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ MMA
    const uint32_t id_s = idesc_f16(128, kHalfTok, 0);
    const uint32_t id_o = idesc_f16(128, D, 0) | (1u << 16);   // values: N (d) contiguous
    constexpr int kHalf = 128 * 128;
    const uint64_t qd = smem_desc(smem_u32(&sm->q[0][0]), 16, 1024, kSwizzle128B);
    const uint64_t kd = smem_desc(smem_u32(&sm->kv[0][0][0]), 16, 1024, kSwizzle128B);
    // MN-major: leading offset between 64-column halves, stride between 8-token groups
    const uint64_t vd = smem_desc(smem_u32(&sm->kv[1][0][0]), kHalf, 1024, kSwizzle128B);
    // Two streams of (S, softmax, O), a warp each: the item's row tiles, or a
    // split tile's even and odd KV tiles. Both walk every KV tile and give its
    // shared memory back, used or not. A stream's two halves of S take turns:
    // while the softmax works on one, P V of the other and the S that follows
    // in its columns are under way (whole tiles of S left either the softmax
    // or the MMAs waiting: 8 % more time at D = 64, the same at 128, where
    // S with N = 64 reads as much of Q as with N = 128).
    const int i = warp - kMmaWarp;
    int j0 = 0, n_q = 0, n_qs = 0, n_p = 0;
    bool ok = true;
    Cut cut = {0, 0, 0, 0, 0, {0, 0, 0}};
    while (w->more && ok) {
      const int nt = w->t1 - w->t0, rows = min(kRowTile, w->n * group - w->q * kRowTile);
      if (w->t0 == 0 && w->t1 < w->tiles) {   // only a range's last piece can be one
        const int lo = cta_of(w->x + kSetup), hi = cta_of(w->x + kSetup + w->tiles - 1);
        cut = {w->row0, rows, w->h, w->q, hi - lo + 1, {0, 0, 0}};
      }
      const bool split = rows <= kSplitRows, idle = i == 1 && !split && rows <= 128;
      const int ahead = split ? 2 : 1;
      if (split) ok = wait(&sm->q_split, n_qs++);
      else if (!idle) ok = wait(&sm->q_full[i], n_q++);
      if (!ok) break;
      const uint64_t qa = qd + (uint64_t)((split ? 0 : i * Sm::kTile) >> 4);
      for (int t = -ahead; t < nt; ++t) {
        const bool mine = split ? (t & 1) == i : !idle, more = t + ahead < nt;
        const int jv = j0 + t, sv = jv & 1, jk = jv + ahead, sk = jk & 1;
        if (t >= 0 && !(ok = wait(&sm->kv_full[1][sv], jv >> 1))) break;
        if (more && !(ok = wait(&sm->kv_full[0][sk], jk >> 1))) break;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (t >= 0 && mine && !(ok = wait(&sm->p_full[i][half], n_p))) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t s_h = tmem + 128 * i + kHalfTok * half;
            if (t >= 0) {
              if (mine) {
                const uint64_t vb = vd + (uint64_t)((sv * Sm::kTile + half * (kHalfTok / 16) * 2048) >> 4);
#pragma unroll
                for (int kk = 0; kk < kHalfTok / 16; ++kk)
                  mma_f16_tmem_a(tmem + 256 + 128 * i, s_h + 8 * kk, vb + kk * (2048 >> 4), id_o,
                                 t >= ahead || half > 0 || kk > 0);
                tc_commit(&sm->pv_done[i]);
                if (half) tc_commit(&sm->kv_empty[1][sv]);
                if (half && !more) tc_commit(&sm->o_full[i]);
              } else if (half) {
                mbar_arrive(&sm->kv_empty[1][sv]);
              }
            }
            if (more) {
              if (mine) {
                const uint64_t kb = kd + (uint64_t)((sk * Sm::kTile + half * kHalfTok * 128) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint64_t off = (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
                  mma_f16(s_h, qa + off, kb + off, id_s, kk != 0);
                }
                tc_commit(&sm->s_full[i][half]);
                if (half) tc_commit(&sm->kv_empty[0][sk]);
              } else if (half) {
                mbar_arrive(&sm->kv_empty[0][sk]);
              }
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        n_p += t >= 0 && mine;
        if (t == -ahead) next();   // the next piece, while there is time
      }
      j0 += nt;
    }
    if (!ok) cut.n = 0;   // timed out: nothing to join
    if (lane == 0 && i == 0) p.cuts[cta] = cut;
    if (lane == 0) {
      tc_commit(&sm->drain);
      const long long t0 = clock64();
      while (!mbar_try_wait(&sm->drain, 0) && clock64() - t0 < 4000000000ll) {
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
  if (tid == 0 && sm->abort) set_status(p.status, MOE_ERR_TIMEOUT);
  if (p.overlap) pdl_wait();
}

// Joins the partials of the row tiles that several CTAs cut: block (c, part)
// takes 1024 elements of the tile that begins in CTA c. Four elements per
// thread, the loads of kJoinParts partials in flight together: a short tile
// over a long context is in up to all CTAs' pieces, one trip to L2 after the
// other (64 rows over 16000 tokens: 53 us the call with two partials and four
// times the elements in flight, 36 so).
constexpr int kJoinThreads = 256, kJoinParts = 4;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv4_prompt_join_kernel(const __grid_constant__ PromptArgs p) {
  pdl_wait();
  const Cut cut = p.cuts[blockIdx.x];
  const int x = blockIdx.y * kJoinThreads + threadIdx.x;
  if (cut.n < 2 || x >= cut.rows * (D / 4)) return;
  const moe_kv4_attn_args& a = p.a;
  const int group = a.q_heads / a.cache.kv_heads;
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int c = 0; c < cut.n; c += kJoinParts) {
    float2 ml[kJoinParts];
    float4 v[kJoinParts];
    float mn = m;
#pragma unroll
    for (int k = 0; k < kJoinParts; ++k) {
      ml[k] = make_float2(-INFINITY, 0.0f);
      v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (c + k < cut.n) {   // the tile's first CTA holds it at its end, the others at their start
        const float* src = p.partials + ((size_t)(blockIdx.x + c + k) * 2 + (c + k == 0 ? 1 : 0)) * kSlotFloats<D>;
        ml[k] = *reinterpret_cast<const float2*>(src + kRowTile * D + 2 * (x / (D / 4)));
        v[k] = reinterpret_cast<const float4*>(src)[x];
      }
    }
#pragma unroll
    for (int k = 0; k < kJoinParts; ++k) mn = fmaxf(mn, ml[k].x);
    const float mu = mn == -INFINITY ? 0.0f : mn, f = ex2(m - mu);   // 0 from -inf
    m = mn;
    l *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int k = 0; k < kJoinParts; ++k) {
      const float g = ex2(ml[k].x - mu);
      l += g * ml[k].y;
      o.x += g * v[k].x;
      o.y += g * v[k].y;
      o.z += g * v[k].z;
      o.w += g * v[k].w;
    }
  }
  const int row = x / (D / 4), d = x % (D / 4) * 4, rr = cut.q * kRowTile + row, token = rr / group;
  const float inv = 1.0f / (l * a.cache.v_gs);
  const size_t at = (size_t)(cut.row0 + token) * a.q_heads + cut.h * group + rr - token * group;
  *reinterpret_cast<uint2*>(a.out + at * D + d) =
      l == 0.0f ? make_uint2(0u, 0u)   // not what a NaN gives
                : make_uint2(float2_to_bf16x2_bits(o.x * inv, o.y * inv), float2_to_bf16x2_bits(o.z * inv, o.w * inv));
  if (d == 0 && a.lse != nullptr) a.lse[at] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
}

template <int D>
cudaError_t launch(const PromptArgs& p, int ctas, cudaStream_t s) {
  auto k = kv4_prompt_kernel<D>;
  constexpr size_t smem = sizeof(Smem<D>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = opt_in_smem(k, smem, done);
  if (e != cudaSuccess) return e;
  e = launch_ex(true, k, dim3(ctas), dim3(kThreads), smem, s, p);
  if (e != cudaSuccess) return e;
  constexpr int rows = kJoinThreads / (D / 4);
  return launch_ex(true, kv4_prompt_join_kernel<D>, dim3(ctas, kRowTile / rows), dim3(kJoinThreads), 0, s, p);
}

}  // namespace

size_t kv4_prompt_ws_floats(int head_dim) {
  return kCutFloats + (size_t)kKvMaxCtas * 2 * (head_dim == 64 ? kSlotFloats<64> : kSlotFloats<128>);
}

long long kv4_prompt_units(const moe_kv4_attn_args& a) {
  const long long rows = (long long)a.total_q * (a.q_heads / a.cache.kv_heads);
  const long long tiles = (long long)a.max_pages * a.cache.page_tokens / kTok + 2 + kSetup;
  return (rows / kRowTile + a.batch) * a.cache.kv_heads * tiles;
}

moe_status launch_kv4_prompt(const moe_kv4_attn_args& a, int min_rows, int* status, float* partials, bool overlap,
                             cudaStream_t s) {
  PromptArgs p;
  p.a = a;
  p.min_rows = min_rows;
  p.status = status;
  p.cuts = reinterpret_cast<Cut*>(partials);
  p.partials = partials + kCutFloats;
  p.wait_limit = debug_wait_limit();
  p.overlap = overlap && a.batch <= kChunk;   // one launch of each
  const int sms = sm_count(), ctas = sms < kKvMaxCtas ? sms : kKvMaxCtas;
  for (int b0 = 0; b0 < a.batch; b0 += kChunk) {
    p.b0 = b0;
    p.nb = a.batch - b0 < kChunk ? a.batch - b0 : kChunk;
    cudaError_t e = a.cache.head_dim == 64 ? launch<64>(p, ctas, s) : launch<128>(p, ctas, s);
    if (e != cudaSuccess) return cuda_ok(e);
    count_launches(2);
  }
  return MOE_OK;
}

}  // namespace moe
