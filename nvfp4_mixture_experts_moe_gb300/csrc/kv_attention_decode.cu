// Attention over the NVFP4 cache for few query rows: single tokens and
// drafted tokens of up to 16 rows per (request, key/value head), a row being
// one (token, query head) pair of the head's group.
//
// Mathematics. For a row q and cached token j: s_j = scale (q . k_j), out =
// sum_j p_j v_j / sum_j p_j with p_j = 2^(s_j log2 e - m), m a running
// maximum. The row enters as f16 times a power of two that puts its largest
// element in [2^14, 2^15) (exact for bf16 down to 2^-24 of that element), the
// keys as e2m1 * e4m3 in f16 (exact: at most six significant bits), so the
// products are exact and summed in fp32. p_j is rounded to f16 for the second
// product, from an m that lies 7 to 15 below the running maximum: the largest
// p_j is 2^7 to 2^15, so one down to 2^-21 of it keeps 2^-11 of itself, and one
// down to 2^-32 is not lost (many of those next to one token that takes nearly
// all, whose value may be small, are the output). The values enter exactly
// like the keys; sums and statistics are fp32.
//
// What bounds it: the cache's bytes, 1.125 D per token and head, where
// contexts are long; the trips to memory one after the other (lengths, pages,
// tiles, partials: 7 us in all) where they are short. The kernel is a list of
// tiles dealt out evenly: a tile is 32 or 64 tokens of one (request, head);
// all tiles in order (request, head, token) are cut into one range per CTA
// and that into one range per warp. Each warp streams its tiles through a
// private ring of shared-memory stages (16-byte asynchronous copies), so there
// is no synchronisation between warps until their ranges end, whatever the
// lengths. Ranges that cut a (request, head) leave partial results (m, sum,
// unnormalised output), joined first by the warps of a CTA, then by the last
// CTA to finish one; every join adds in the order of the ranges, so results
// do not depend on timing. Where every (request, head) is short and there are
// no more of them than SMs, a CTA takes one whole: the join across CTAs costs
// 2 to 4 us (16 requests of 1024 tokens: 15.0 us cut, 11.1 whole).
//
// mma.sync rather than tcgen05: at 1 to 16 rows the tensor work is a few
// per cent of the time, and the dequantised operand never has to leave the
// registers that converted it. A tile of 32 tokens at D = 128 costs a warp
// 590 instructions for 8 rows and 670 for 16 (250 on the ALU pipe, half of them
// conversions, 200 to 220 on the FMA pipe, most of them scales, 32 and 64
// matrix, 48 and 65 of shared memory). With 16 rows the registers leave 12
// warps instead of 16, which issue in 0.48 of the cycles instead of 0.63: these
// run further from the memory rate.
//
// Measured (replayed): 4 requests of 131072 tokens, 8 heads x 128: 108 us,
// 5.6 TB/s (82 % of the measured copy rate), with 12 or 16 query heads to each
// 161 and 163 us; 64 of up to 8192 in pages of 16: 69 us, 4.5 TB/s (9 us until
// the first tiles are there, 8 after the last for uneven ends and joins), with
// 16 query heads to each 118; 16 rows over 84,500 tokens at D = 64: 29.7 us
// (26.3 from L2); one request of 1000 tokens: 9.2 us.
#include <type_traits>

#include "kernels.cuh"
#include "kv4.cuh"
#include "kv_rows.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace rows;
using namespace tc;

constexpr int kChunk = 1024;       // requests of one launch
// Tiles that a CTA works on in the time that a join across CTAs takes, where
// every SM has a range (which then begin and end anywhere); half where not. (us
// with 0, 12, 24, 48 and 96 here: 16 x 1024 tokens of 8 heads 15.0, 11.1, 11.1,
// 11.1, 11.1; 16 x 4096 24.5, 24.4, 22.0, 22.0, 22.0; 8 x 1000 for 16 rows 23.8,
// 23.7, 15.9, 15.9, 15.9; 1 x 1000 8.9, 8.9, 8.9, 8.9, 10.5; 16 of 256 to 2048
// 15.5, 15.6, 15.5, 14.7, 14.7.)
constexpr int kAlone = 24;

struct DecodeArgs {
  moe_kv4_attn_args a;
  int b0, nb;          // the requests of this launch
  int max_rows;        // requests with more query rows belong to another kernel
  int* status;
  int* counters;       // [kKvMaxCtas] zero between launches
  float* partials;     // see Slots
};

// A tile is 4608 bytes of one (request, head): 32 tokens at D = 128, 64 at 64.
template <int D, int NT>
struct Shape {
  static constexpr int kWarps = NT == 1 ? 16 : 12;
  static constexpr int kBlocks = 256 / D;              // 16-token blocks of a tile
  static constexpr int kTile = kBlocks * kKvBlock;
  static constexpr int kStageBytes = kBlocks * Kv4Block<D>::kBytes;
  static constexpr int kStages = NT == 1 ? 3 : 4;
  static constexpr int kThreads = kWarps * 32;
};

struct Ends {
  int b, h, s0, s1;   // request, head, tiles
  int row0, n;
};

template <int D, int NT>
struct Smem {
  using Sh = Shape<D, NT>;
  alignas(128) uint8_t ring[Sh::kWarps][Sh::kStages][Sh::kStageBytes];
  int pre[kChunk + 1];     // tiles (over all heads) before each request
  int warp_sum[Sh::kWarps], warp_top[Sh::kWarps];
  int start[Sh::kWarps + 1];   // the warps' ranges
  int piece[2][Sh::kWarps];    // where a warp's last and first partial lie in the ring, in floats
  Ends ends[Sh::kWarps][2];    // the segments a warp's range begins and ends with
  int last[2];
  static_assert(Sh::kStages * Sh::kStageBytes >= Slots<D, NT>::kFloats * 4, "a warp's ring holds its last partial");
  // A range has at most one partial before its last: a piece of a segment
  // that began earlier. It stays in the stage its last tile came from, the
  // ring going on with one stage less; if it does not fit, it goes to memory.
  static constexpr bool kPark = Sh::kStageBytes >= Slots<D, NT>::kFloats * 4;
};

// Lengths of one request, cut to what the tables can hold.
struct Request {
  int row0, n, kv;   // first query row, query rows, cached tokens
  bool bad;
};

__device__ __forceinline__ Request load_request(const moe_kv4_attn_args& a, int b) {
  Request r;
  const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), kv = __ldg(a.kv_len + b);
  const int cap = a.max_pages * a.cache.page_tokens;
  r.row0 = c0;
  r.n = c1 - c0;
  r.kv = max(0, min(kv, cap));
  r.bad = kv != r.kv;
  if (c0 < 0 || r.n < 0 || c1 > a.total_q || r.n > a.max_q) {
    r.n = 0;
    r.bad = true;
  }
  return r;
}

// First token any of the request's rows sees.
__device__ __forceinline__ int first_seen(const moe_kv4_attn_args& a, const Request& r) {
  return a.window > 0 ? max(0, min(r.kv, r.kv - r.n + 1 - a.window)) : 0;
}

__device__ __forceinline__ int last_at_most(const int* arr, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (arr[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct Segment {
  int b, h;      // request (within the launch), key/value head
  int s0, s1;    // its tiles
};

__device__ __forceinline__ Segment segment_of(const int* pre, int nb, int heads, int tile) {
  Segment s;
  s.b = last_at_most(pre, nb - 1, tile);
  const int per = (pre[s.b + 1] - pre[s.b]) / heads;
  s.h = (tile - pre[s.b]) / per;
  s.s0 = pre[s.b] + s.h * per;
  s.s1 = s.s0 + per;
  return s;
}

// Normalised bf16 and lse of a joined row. One that has seen nothing has l = 0
// and gets zeros and -inf; l is NaN where a score was, and so are the row and
// its lse.
__device__ __forceinline__ void write_joined(const Joined& x, const moe_kv4_attn_args& a, const Request& rq, int h, int group,
                                             int row, int D, int d) {
  const float inv = x.l == 0.0f ? 0.0f : 1.0f / (x.l * a.cache.v_gs);
  const size_t at = (size_t)(rq.row0 + row / group) * a.q_heads + h * group + row % group;
  *reinterpret_cast<uint2*>(a.out + at * D + d) =
      make_uint2(float2_to_bf16x2_bits(x.o.x * inv, x.o.y * inv), float2_to_bf16x2_bits(x.o.z * inv, x.o.w * inv));
  if (d == 0 && a.lse != nullptr) a.lse[at] = x.l == 0.0f ? -INFINITY : x.m * kLn2 + logf(x.l);
}

// Joins n partials that a CTA's warps left in shared memory (one may lie in
// global memory), in their order: warp `mine` of `warps` takes every warps-th
// run of 32 times four neighbouring columns (a row at D = 128), which its
// lanes read without bank conflicts. To the output or, dst given, to a partial.
template <int D, int NT, class Src>
__device__ __forceinline__ void join_warps(const moe_kv4_attn_args& a, const Request& rq, int h, int n, Src src,
                                           int mine, int warps, float* dst) {
  constexpr int kRows = 8 * NT, kBatch = 2;
  const int group = a.q_heads / a.cache.kv_heads, lane = threadIdx.x & 31;
  for (int e = 32 * mine + lane; e < rq.n * group * (D / 4); e += 32 * warps) {
    const int row = e / (D / 4), d = e % (D / 4) * 4;
    Joined x;
#pragma unroll 1
    for (int i = 0; i < n; i += kBatch) {
      float2 ml[kBatch];
      float4 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        ml[j] = make_float2(-INFINITY, 0.0f);
        v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i + j < n) {
          const float* s = src(i + j);
          ml[j] = *reinterpret_cast<const float2*>(s + kRows * D + 2 * row);
          v[j] = *reinterpret_cast<const float4*>(s + row * D + warp_chunk(row, d / 4) * 4);
        }
      }
      x.add(ml, v);
    }
    if (dst != nullptr) {
      *reinterpret_cast<float4*>(dst + row * D + d) = x.o;
      if (d == 0) *reinterpret_cast<float2*>(dst + kRows * D + 2 * row) = make_float2(x.m, x.l);
    } else {
      write_joined(x, a, rq, h, group, row, D, d);
    }
  }
}

// Joins n partials that CTAs left in global memory, up to one per CTA of the
// grid, by a whole CTA: a warp reads whole rows (four neighbouring columns a
// thread), and what threads there are beyond a row tile's columns take every
// kParts-th partial, joined at the end through shared memory.
template <int D, int NT, class Src>
__device__ __forceinline__ void join_ctas(const moe_kv4_attn_args& a, const Request& rq, int h, int n, Src src,
                                          float* shared) {
  constexpr int kRows = 8 * NT, kElems = kRows * D / 4, T = Shape<D, NT>::kThreads, kBatch = 4;
  constexpr int kParts = T >= kElems ? T / kElems : 1, kStep = kParts > 1 ? kElems : T;
  const int group = a.q_heads / a.cache.kv_heads, part = threadIdx.x / kStep;
  for (int e = threadIdx.x - part * kStep; e < (kElems + kStep - 1) / kStep * kStep; e += kStep) {
    const int row = e / (D / 4), d = e % (D / 4) * 4;
    const bool real = e < kElems && part < kParts && row < rq.n * group;
    Joined x;
    if (real)
#pragma unroll 1
      for (int i = part; i < n; i += kBatch * kParts) {
        float2 ml[kBatch];
        float4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          ml[j] = make_float2(-INFINITY, 0.0f);
          v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (i + j * kParts < n) {
            const float* s = src(i + j * kParts);
            ml[j] = __ldcg(reinterpret_cast<const float2*>(s + kRows * D + 2 * row));
            v[j] = __ldcg(reinterpret_cast<const float4*>(s + row * D + d));
          }
        }
        x.add(ml, v);
      }
    if constexpr (kParts > 1) {
      float4* const os = reinterpret_cast<float4*>(shared);
      float2* const mls = reinterpret_cast<float2*>(os + (kParts - 1) * kElems);
      if (real && part > 0) {
        os[(part - 1) * kElems + e] = x.o;
        mls[(part - 1) * kElems + e] = make_float2(x.m, x.l);
      }
      __syncthreads();
      if (real && part == 0) {
        float2 ml[kParts - 1];
        float4 v[kParts - 1];
#pragma unroll
        for (int j = 0; j < kParts - 1; ++j) {
          ml[j] = mls[j * kElems + e];
          v[j] = os[j * kElems + e];
        }
        x.add(ml, v);
      }
      __syncthreads();
    }
    if (real && part == 0) write_joined(x, a, rq, h, group, row, D, d);
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1) kv4_decode_kernel(const __grid_constant__ DecodeArgs p) {
  using Sh = Shape<D, NT>;
  using L = Kv4Block<D>;
  using Sm = Smem<D, NT>;
  constexpr int W = Sh::kWarps, S = Sh::kStages, kRows = 8 * NT, MT = D / 16;
  constexpr int NB = Sh::kBlocks, kTile = Sh::kTile, kPart = NT == 1 ? NB : 2;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Sm* sm = reinterpret_cast<Sm*>(smem_raw);
  const moe_kv4_attn_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;
  const int P = a.cache.page_tokens, p_log = __ffs(P) - 1, Hk = a.cache.kv_heads, group = a.q_heads / Hk;

  // ------------------------------------------------ tiles before each request
  pdl_wait();
  pdl_trigger();   // after the wait: see the many-row kernel
  if (tid == 0) sm->pre[0] = 0;
  int carry = 0, longest = 0;   // tiles of all requests; of one (request, head)
  bool bad = false;
  for (int base = 0; base < p.nb; base += Sh::kThreads) {
    const int b = base + tid;
    int tiles = 0;
    if (b < p.nb) {
      const Request r = load_request(a, p.b0 + b);
      bad |= r.bad;
      const long long rows = (long long)r.n * group;
      if (rows > 0 && rows <= p.max_rows) tiles = (r.kv + kTile - 1) / kTile - first_seen(a, r) / kTile;
    }
    const int top = __reduce_max_sync(kFull, tiles);
    tiles *= Hk;
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) {
      sm->warp_sum[warp] = incl;
      sm->warp_top[warp] = top;
    }
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int v = sm->warp_sum[w];
      if (w < warp) before += v;
      carry += v;
      longest = max(longest, sm->warp_top[w]);
    }
    if (b < p.nb) sm->pre[b + 1] = before + incl;
    __syncthreads();
  }
  if (bad && blockIdx.x == 0) set_status(p.status, MOE_ERR_DEVICE);
  const int total = sm->pre[p.nb];

  // rows that see nothing at all: zeros
  for (int b = blockIdx.x; b < p.nb; b += gridDim.x) {
    if (sm->pre[b + 1] != sm->pre[b]) continue;
    const Request r = load_request(a, p.b0 + b);
    if (r.n == 0 || (long long)r.n * group > p.max_rows) continue;
    const size_t at = (size_t)r.row0 * a.q_heads;
    for (int i = tid; i < r.n * a.q_heads * D / 8; i += Sh::kThreads)
      reinterpret_cast<uint4*>(a.out + at * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse != nullptr)
      for (int i = tid; i < r.n * a.q_heads; i += Sh::kThreads) a.lse[at + i] = -INFINITY;
  }
  if (total == 0) return;

  // ------------------------------------------------------- this warp's range
  // Equal ranges, or a (request, head) for each CTA where that takes little
  // more of its time than the join across CTAs would.
  // Few tiles go to fewer CTAs, four to each, or eight where a (request, head)
  // has more than 64 and the join of its partials is what takes long. (us with
  // four and eight: 1 x 1000 tokens of one head 7.9 and 8.6, 1 x 4096 at D = 64
  // 8.9 and 9.2; 2 x 4066 of one 10.2 and 9.8, 1 x 4096 of 8 10.1 and 9.9, 1 x
  // 16384 of one 15.5 and 12.2; with sixteen 2 x 4066 takes 11.2.)
  const int least = longest > 16 * kKvTilesPerCta ? 2 * kKvTilesPerCta : kKvTilesPerCta;
  const int cta = blockIdx.x, spread = min((int)gridDim.x, (total + least - 1) / least);
  const int per_cta = (total + spread - 1) / spread, more = spread == (int)gridDim.x ? kAlone : kAlone / 2;
  const bool alone = p.nb * Hk <= (int)gridDim.x && longest <= per_cta + more;
  const int G = alone ? p.nb * Hk : spread;
  if (cta >= G) return;
  int C0 = mul_div(total, cta, G), C1 = mul_div(total, cta + 1, G);
  if (alone) {
    const int b = cta / Hk, per = (sm->pre[b + 1] - sm->pre[b]) / Hk;
    C0 = sm->pre[b] + (cta - b * Hk) * per;
    C1 = C0 + per;
    if (per == 0) return;
  }
  const int wact = min(W, C1 - C0);   // (a CTA's range times W fits 32 bits: it is at most 2^31 / 152 tiles)
  const int r0 = C0 + (int)((unsigned)(C1 - C0) * min(warp, wact) / (unsigned)wact);
  const int r1 = C0 + (int)((unsigned)(C1 - C0) * min(warp + 1, wact) / (unsigned)wact);
  if (lane == 0) {   // read after the barrier that follows the loop
    sm->start[warp + 1] = r1;
  }
  __syncwarp();
  if (tid == 0) sm->start[0] = C0;
  float* const slots = p.partials;
  auto cta_slot = [&](int c, int which) {
    return slots + ((size_t)kKvMaxCtas * W + (size_t)c * 2 + which) * Slots<D, NT>::kFloats;
  };

  if (warp < wact) {
    // Lane i holds where tile base + i comes from: one place per page, of
    // min(P, kTile) tokens. Everything that needs a division or the tables is
    // done here, once in 32 tiles.
    const int run_log = min(p_log - 4, NB == 2 ? 1 : 2);   // log2 of the blocks of a copy
    int d_b = 0, d_h = 0, d_tok = 0, d_valid = 0, d_s0 = 0, d_seg_end = 0, d_row0 = 0, d_n = 0, base = r0;
    const uint8_t* d_src[NB];
    auto describe = [&](int from) {
      base = from;
      const int tile = from + lane;
      d_valid = 0;
#pragma unroll
      for (int i = 0; i < NB; ++i) d_src[i] = nullptr;
      if (tile < r1) {
        const Segment s = segment_of(sm->pre, p.nb, Hk, tile);
        const Request r = load_request(a, p.b0 + s.b);
        d_b = s.b;
        d_h = s.h;
        d_row0 = r.row0;
        d_n = r.n;
        d_s0 = s.s0;
        d_seg_end = s.s1;
        const int seen = first_seen(a, r);
        d_tok = (seen / kTile + (tile - s.s0)) * kTile;
        const int unseen = (seen - d_tok) >> p_log;
        const int32_t* table = a.block_table + (size_t)(p.b0 + s.b) * a.max_pages + (d_tok >> p_log);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int blk = i << run_log;
          if (blk >= NB || d_tok + blk * kKvBlock >= r.kv) break;
          if (i < unseen) continue;   // a page before every row's window may have been given back
          const int page = __ldg(table + i);
          if (page >= 0 && page < a.cache.num_pages) {
            d_valid |= ((1 << (1 << run_log)) - 1) << blk;
            d_src[i] = static_cast<const uint8_t*>(a.cache.pool) +
                       kv4_block_offset(page, s.h, Hk, P / kKvBlock, (d_tok & (P - 1)) / kKvBlock, L::kBytes);
          } else {
            set_status(p.status, MOE_ERR_DEVICE);
          }
        }
      }
    };
    // All lanes copy a described tile into a slot, one group per tile.
    auto issue = [&](int tile, int slot) {
      const int src = tile - base;
      const int valid = __shfl_sync(kFull, d_valid, src);
      const uint32_t dst = smem_u32(&sm->ring[warp][0][0]) + slot * Sh::kStageBytes + lane * 16;
      const uint8_t* from[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        if (i > 0 && (i << run_log) >= NB) break;
        from[i] = reinterpret_cast<const uint8_t*>(
                      __shfl_sync(kFull, reinterpret_cast<unsigned long long>(d_src[i]), src)) + lane * 16;
      }
      if ((1 << run_log) == NB) {
        if (valid) {
#pragma unroll
          for (int c = 0; c < Sh::kStageBytes; c += 512) cp_async_16(dst + c, from[0] + c, 16);
        }
      } else {
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          if (!(valid >> blk & 1)) continue;
          // blocks 0, 1 (and 2, 3) share a page of 32 tokens
          const uint8_t* f = run_log == 0 ? from[blk] : from[blk / 2] + (blk & 1) * L::kBytes;
#pragma unroll
          for (int c = 0; c < L::kBytes; c += 512)
            if (c + 512 <= L::kBytes || lane * 16 < L::kBytes - c)
              cp_async_16(dst + blk * L::kBytes + c, f + c, 16);
        }
      }
    };

    describe(r0);
    // The first segment's rows are asked for before any tile, or they would
    // wait behind all the tiles in flight.
    {
      const char* q = reinterpret_cast<const char*>(
          a.q + (size_t)__shfl_sync(kFull, d_row0, 0) * a.q_stride + (size_t)__shfl_sync(kFull, d_h, 0) * group * D);
      for (int i = __shfl_sync(kFull, d_n, 0); i > 0; --i, q += a.q_stride * 2)
        if (lane * 128 < group * D * 2) asm volatile("prefetch.global.L1 [%0];" ::"l"(q + lane * 128));
    }
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < S; ++i) {
      if (r0 + i < r1) issue(r0 + i, i);
      cp_async_commit();
    }

    RowState<D, NT> st;
    Request rq = {0, 0, 0, false};
    int h = 0, plain0 = 0, plain1 = 0;   // tiles with every token in [plain0, plain1) need no mask
    int seg_end = r0;
    bool from_start = false;             // the segment's first tile is in this range
    int next = r0 + min(S, r1 - r0);     // the next tile to issue

    int slot = 0, parked = -1;
    auto advance = [&](int s) { return s + 1 == S ? 0 : s + 1; };
    for (int tile = r0; tile < r1; ++tile) {
      const int src = tile - base;       // < 32: described before it was issued
      const int tok0 = __shfl_sync(kFull, d_tok, src), valid = __shfl_sync(kFull, d_valid, src);
      if (tile == seg_end || tile == r0) {   // a new (request, head)
        const int b = __shfl_sync(kFull, d_b, src);
        h = __shfl_sync(kFull, d_h, src);
        seg_end = __shfl_sync(kFull, d_seg_end, src);
        const int s0 = __shfl_sync(kFull, d_s0, src);
        from_start = s0 == tile;
        rq = load_request(a, p.b0 + b);
        if (lane == 0) {
          const Ends e = {b, h, s0, seg_end, rq.row0, rq.n};
          if (tile == r0) sm->ends[warp][0] = e;
          if (seg_end >= r1) sm->ends[warp][1] = e;
        }
        const int low = a.causal ? rq.kv - rq.n : rq.kv - 1;   // the first row's last token
        plain1 = low + 1;
        plain0 = a.window > 0 ? rq.kv - a.window : 0;
        start_rows<D, NT>(st, g8, t4, a.scale, a.cache.k_gs, [&](int row) {
          return row < rq.n * group
                     ? a.q + (size_t)(rq.row0 + row / group) * a.q_stride + (h * group + row % group) * D
                     : nullptr;
        });
      }

      if (parked < 0) cp_async_wait<S - 1>();   // this tile's group, on every lane
      else cp_async_wait<S - 2>();
      __syncwarp();
      const uint8_t* stage = &sm->ring[warp][0][0] + slot * Sh::kStageBytes;
      const bool masked = tok0 < plain0 || tok0 + kTile > plain1 || valid != (1 << NB) - 1;

      // Two copies of the work on a tile (on its halves for 16 rows at D = 64:
      // registers), so that tiles every row sees whole (all but a request's
      // last, for a single token) carry no mask.
      auto work = [&](auto with_mask, const uint8_t* part, int tok0, int valid) {
        constexpr bool kMask = decltype(with_mask)::value;
        const int recip = kMask ? (65535 + group) / group : 0;
        attend_blocks<D, NT, kPart, kMask>(st, g8, t4, part, [&](int blk, int nt, int i) {
          const int tok = tok0 + blk * kKvBlock + token_of(g8) + 8 * (i >> 1);
          // the last token its query sees; row / group by the reciprocal (both at most 16)
          const int token = (nt * 8 + 2 * t4 + (i & 1)) * recip >> 16;
          const int hi_tok = a.causal ? rq.kv - rq.n + token : rq.kv - 1, lo_tok = a.window > 0 ? hi_tok - a.window + 1 : 0;
          return tok > hi_tok || tok < lo_tok || !(valid >> blk & 1);
        });
      };
#pragma unroll 1
      for (int blk = 0; blk < NB; blk += kPart) {
        const uint8_t* part = stage + blk * L::kBytes;
        if (masked) work(std::true_type{}, part, tok0 + blk * kKvBlock, valid >> blk);
        else work(std::false_type{}, part, tok0 + blk * kKvBlock, valid >> blk);
      }

      __syncwarp();   // every lane has read the stage
      const bool seg_done = tile + 1 == seg_end, done = tile + 1 == r1;
      const bool park = Sm::kPark && seg_done && !done && !from_start;
      if (park) {
        parked = slot;
      } else if (next < r1) {
        // descriptors run out S tiles ahead of the tile being read
        if (next - base >= 32) describe(tile + 1);
        __syncwarp();
        issue(next, slot);
        ++next;
      }
      cp_async_commit();

      // --------------------------------------- the end of a range or segment
      if (seg_done || done) {
        const bool whole = from_start && seg_done;
        // at the range's end clear of the parked stage: a partial that can be parked is one stage long
        const int at = (warp * S + (done ? parked == 0 : slot)) * (Sh::kStageBytes / 4);
        float* dst = Sm::kPark || done ? reinterpret_cast<float*>(smem_raw) + at
                                       : slots + (size_t)(cta * W + warp) * Slots<D, NT>::kFloats;
        if (lane == 0 && !whole) sm->piece[done ? 0 : 1][warp] = at;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float sum = st.l[nt][c];
            sum += __shfl_xor_sync(kFull, sum, 4);
            sum += __shfl_xor_sync(kFull, sum, 8);
            sum += __shfl_xor_sync(kFull, sum, 16);
            const int row = nt * 8 + 2 * t4 + c;
            if (whole) {
              if (row < rq.n * group) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / (sum * a.cache.v_gs);   // NaN stays NaN
                const size_t at = (size_t)(rq.row0 + row / group) * a.q_heads + h * group + row % group;
                uint32_t w[MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                  w[mt] = float2_to_bf16x2_bits(st.o[nt][mt][c] * inv, st.o[nt][mt][c + 2] * inv);
                uint4* out = reinterpret_cast<uint4*>(a.out + at * D + g8 * (D / 8));
#pragma unroll
                for (int i = 0; i < MT / 4; ++i) out[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                if (g8 == 0 && a.lse != nullptr)
                  a.lse[at] = sum == 0.0f ? -INFINITY : st.m[nt][c] * kLn2 + logf(sum);
              }
            } else {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                *reinterpret_cast<float2*>(dst + row * D + warp_chunk(row, g8 * (D / 32) + mt / 2) * 4 + mt % 2 * 2) =
                    make_float2(st.o[nt][mt][c], st.o[nt][mt][c + 2]);
              if (g8 == 0) *reinterpret_cast<float2*>(dst + kRows * D + 2 * row) = make_float2(st.m[nt][c], sum);
            }
          }
      }
      slot = advance(slot);
      if (slot == parked) slot = advance(slot);
    }
  }
  __syncthreads();

  // ------------------------------------ joins of what this CTA's warps cut
  // A segment that spans several warps' ranges, or leaves the CTA's, is
  // joined by those warps, each taking an equal share of its elements.
  auto warp_of = [&](int tile) { return (int)(((unsigned)(tile - C0 + 1) * wact - 1) / (unsigned)(C1 - C0)); };
  if (warp < wact) {
    for (int side = 0; side < 2; ++side) {   // the segment this range begins with, then the one it ends with
      const Ends sg = sm->ends[warp][side];
      if (side == 1 && sg.s0 <= r0) break;    // the same segment
      const int lo = max(sg.s0, C0), hi = min(sg.s1, C1);
      const int w0 = warp_of(lo), w1 = warp_of(hi - 1);
      const bool inside = sg.s0 >= C0 && sg.s1 <= C1;
      if (inside && w0 == w1) continue;       // written when it ended
      const Request rq = {sg.row0, sg.n, 0, false};
      // warp w's piece is in its tail slot when it reaches the end of w's range
      const bool short_last = sm->start[w1 + 1] > hi;
      auto src = [&](int i) -> const float* {
        const int w = w0 + i;
        if (!Sm::kPark && short_last && w == w1) return slots + (size_t)(cta * W + w) * Slots<D, NT>::kFloats;
        return reinterpret_cast<const float*>(smem_raw) + sm->piece[short_last && w == w1][w];
      };
      join_warps<D, NT>(a, rq, sg.h, w1 - w0 + 1, src, warp - w0, w1 - w0 + 1,
                         inside ? nullptr : cta_slot(cta, sg.s0 < C0 ? 0 : 1));
    }
  }

  // --------------------------- segments that several CTAs cut: the last joins
  const Ends first = sm->ends[0][0], end = sm->ends[wact - 1][1];
  const bool cut0 = first.s0 < C0, cut1 = end.s1 > C1 && end.s0 >= C0;
  if (!cut0 && !cut1) return;
  auto cta_of = [&](int tile) { return mul_div(tile + 1, G, total, -1); };   // the last c with total * c / G <= tile
  __syncthreads();
  if (tid < 2) {
    const bool cut = tid == 0 ? cut0 : cut1;
    int is_last = 0;
    if (cut) {
      const Ends& sg = tid == 0 ? first : end;
      const int c0 = cta_of(sg.s0), c1 = cta_of(sg.s1 - 1);
      __threadfence();   // cumulative: the CTA's partials, ordered before by the barrier
      if (atomicAdd(p.counters + c0, 1) == c1 - c0) {
        p.counters[c0] = 0;   // everyone has arrived: ready for the next launch
        is_last = 1;
      }
      __threadfence();
    }
    sm->last[tid] = is_last;
  }
  __syncthreads();
  for (int side = 0; side < 2; ++side) {
    if (!sm->last[side]) continue;
    const Ends& sg = side == 0 ? first : end;
    const int c0 = cta_of(sg.s0), n = cta_of(sg.s1 - 1) - c0 + 1;
    const Request rq = {sg.row0, sg.n, 0, false};
    // the CTA the segment begins in holds its tail, the others their head
    auto src = [&](int i) -> const float* { return cta_slot(c0 + i, i == 0 ? 1 : 0); };
    join_ctas<D, NT>(a, rq, sg.h, n, src, reinterpret_cast<float*>(smem_raw));
  }
}

template <int D, int NT>
size_t partial_floats() {
  return (size_t)kKvMaxCtas * (Shape<D, NT>::kWarps + 2) * Slots<D, NT>::kFloats;
}

template <int D, int NT>
cudaError_t launch(const DecodeArgs& p, int ctas, cudaStream_t s) {
  auto k = kv4_decode_kernel<D, NT>;
  const size_t smem = sizeof(Smem<D, NT>);
  static_assert(sizeof(Smem<D, NT>) <= 227 * 1024, "shared memory");
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = opt_in_smem(k, smem, done);
  if (e != cudaSuccess) return e;
  return launch_ex(true, k, dim3(ctas), dim3(Shape<D, NT>::kThreads), smem, s, p);
}

}  // namespace

size_t kv4_decode_ws_floats(int head_dim, int rows) {
  if (head_dim == 64) return rows <= 8 ? partial_floats<64, 1>() : partial_floats<64, 2>();
  return rows <= 8 ? partial_floats<128, 1>() : partial_floats<128, 2>();
}

moe_status launch_kv4_decode(const moe_kv4_attn_args& a, int max_rows, int* status, int* counters, float* partials,
                             cudaStream_t s) {
  DecodeArgs p;
  p.a = a;
  p.max_rows = max_rows;
  p.status = status;
  p.counters = counters;
  p.partials = partials;
  const int sms = sm_count(), ctas = sms < kKvMaxCtas ? sms : kKvMaxCtas;
  for (int b0 = 0; b0 < a.batch; b0 += kChunk) {
    p.b0 = b0;
    p.nb = a.batch - b0 < kChunk ? a.batch - b0 : kChunk;
    cudaError_t e;
    if (a.cache.head_dim == 64) e = max_rows <= 8 ? launch<64, 1>(p, ctas, s) : launch<64, 2>(p, ctas, s);
    else e = max_rows <= 8 ? launch<128, 1>(p, ctas, s) : launch<128, 2>(p, ctas, s);
    if (e != cudaSuccess) return cuda_ok(e);
    count_launches(1);
  }
  return MOE_OK;
}

}  // namespace moe
