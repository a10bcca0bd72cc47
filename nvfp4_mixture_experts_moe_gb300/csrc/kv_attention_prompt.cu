// Attention over the NVFP4 cache for many query rows (prompts, prompt chunks,
// long drafts): tcgen05 tiles of 2 x 128 query rows against 128 cached tokens.
//
// A row is one (token, query head) pair of a key/value head's group, so the
// heads of a group share every dequantised key and value. Mathematics as in
// kv_attention_decode.cu: rows as f16 times a power of two (exact), keys and
// values as e2m1 * e4m3 in f16 (exact), fp32 scores, p = 2^(s - m) rounded to
// f16, m at most 8 below the running maximum (log2), fp32 sums and output.
//
// Per CTA (one per SM):
// * four dequant warps, each two 16-token blocks of the tile: codes and scales
//   by plain loads a tile ahead (the packed cache is small and read by
//   several row tiles: it comes from L2), converted into 128-byte-swizzled
//   shared-memory tiles, keys K-major, values with d contiguous (MN-major);
// * one thread issues S_i = Q_i K^T and O_i += P_i V for the two row tiles i in
//   turn, so one tile's softmax runs under the other's MMAs; P_i (f16, read
//   from tensor memory) lies in S_i's columns;
// * eight softmax warps, one row per thread: one pass over S in 32-column
//   pieces with the running maximum of the tiles before; a piece that exceeds
//   it by more than 8 rescales O, the sum and the pieces of P already written
//   (rare after the first tiles), so S is read from tensor memory once.
//
// What bounds it: per 128 tokens and 256 rows at D = 128 the MMAs take 2048
// cycles and the exponentials 1024; the softmax and dequant warps' instructions
// are about as many as the schedulers issue in that time.
//
// Work is dealt out by KV tiles: all (request, head, row tile, KV tile) in
// order, one equal range per CTA; a row tile that two or more CTAs cut leaves
// fp32 partials that the last of them joins in order.
#include "kernels.cuh"
#include "kv4.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kTok = 128;              // cached tokens of a tile
constexpr int kRowTile = 256;          // query rows of an item: two M = 128 tiles
constexpr int kChunk = 1024;           // requests of one launch
constexpr int kSoftWarps = 8, kDeqWarps = 4;
constexpr int kWarpBlocks = kTok / kKvBlock / kDeqWarps;
static_assert(kWarpBlocks == 2, "blocks of a dequant warp");
constexpr int kMmaWarp = kSoftWarps + kDeqWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kTmemCols = 512;

struct PromptArgs {
  moe_kv4_attn_args a;
  int b0, nb;
  int min_rows;        // requests with at most this many rows belong to another kernel
  int* status;
  int* counters;       // [kKvMaxCtas] zero between launches
  float* partials;     // [kKvMaxCtas][2][kRowTile x D, then (m, l) per row]
  long long wait_limit;
};

template <int D>
constexpr int kSlotFloats = kRowTile * (D + 2);

template <int D>
struct Smem {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * 128 * 128;   // 128 rows x D f16
  alignas(1024) uint8_t q[2][kTile];
  alignas(1024) uint8_t k[2][kTile];
  alignas(1024) uint8_t v[2][kTile];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t drain;
  alignas(8) uint8_t hole[4][8];       // blocks of a tile whose page is bad
  int pre[kChunk + 1];                 // KV tiles (over all heads and row tiles) before each request
  uint32_t tmem_base;
  int abort;
  int last[2];
};

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

// First token and number of KV tiles of a request's row tile; at least one
// tile, so that rows that see nothing are written (as zeros) like any other.
__device__ __forceinline__ int row_tile_tiles(const moe_kv4_attn_args& a, const Request& r, int group, int q,
                                              int& first) {
  const int rows = r.n * group;
  const int i0 = q * kRowTile / group, i1 = (min(rows, (q + 1) * kRowTile) - 1) / group;
  const int hi = a.causal ? max(0, r.kv - r.n + i1 + 1) : r.kv;
  const int lo = a.window > 0 ? max(0, r.kv - r.n + i0 - a.window + 1) : 0;
  first = lo / kTok * kTok;
  return max(1, (hi + kTok - 1) / kTok - lo / kTok);
}

// The pieces of a CTA's range, one (request, head, row tile) after another.
// Every warp role walks them for itself; all lanes call it together.
struct Pieces {
  const moe_kv4_attn_args& a;
  const int* pre;
  int b0, nb, group, c1;
  // the current piece
  Request rq;
  int b, h, q;
  int x;            // linear index of the piece's first tile
  int first;        // first token of the row tile's first KV tile
  int tiles;        // KV tiles of the row tile
  int t0, t1;       // this piece's
  int per_head;     // KV tiles of the request per head

  __device__ __forceinline__ Pieces(const moe_kv4_attn_args& a_, const int* pre_, int b0_, int nb_, int group_, int C0,
                                    int C1)
      : a(a_), pre(pre_), b0(b0_), nb(nb_), group(group_), c1(C1), x(C0) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = nb - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= C0) lo = mid;
      else hi = mid - 1;
    }
    enter(lo);
    int rem = C0 - pre[b];
    h = rem / per_head;
    rem -= h * per_head;
    // 32 row tiles at a time until the one that holds the tile
    for (q = 0;; q += 32) {
      int f, v = (long long)(q + lane) * kRowTile < (long long)rq.n * group ? row_tile_tiles(a, rq, group, q + lane, f) : 0;
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
        q += at;
        break;
      }
      rem -= __shfl_sync(kFull, incl, 31);
    }
    tiles = row_tile_tiles(a, rq, group, q, first);
    t0 = rem;
    t1 = min(tiles, rem + c1 - x);
  }
  __device__ __forceinline__ void enter(int b_) {
    b = b_;
    rq = load_request(a, b0 + b);
    per_head = (pre[b + 1] - pre[b]) / a.cache.kv_heads;
  }
  __device__ __forceinline__ bool more() const { return x < c1; }
  __device__ __forceinline__ void next() {
    x += t1 - t0;
    if (x >= c1) return;
    if ((long long)(++q) * kRowTile >= (long long)rq.n * group) {
      q = 0;
      if (++h == a.cache.kv_heads) {
        h = 0;
        int nx = b + 1;
        while (pre[nx + 1] == pre[nx]) ++nx;
        enter(nx);
      }
    }
    tiles = row_tile_tiles(a, rq, group, q, first);
    t0 = 0;
    t1 = min(tiles, c1 - x);
  }
  __device__ __forceinline__ int rows() const { return min(kRowTile, rq.n * group - q * kRowTile); }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 pow2_pair(int k) {
  const int h = k >> 1;
  return make_float2(__int_as_float((127 + h) << 23), __int_as_float((127 + k - h) << 23));
}

// Byte offset of 16-byte chunk c (of D/8) of row r in a 128-row f16 tile:
// 64-column halves of 128-byte rows, chunks swizzled by the row.
__device__ __forceinline__ uint32_t tile_chunk(int r, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_prompt_kernel(PromptArgs p) {
  using L = Kv4Block<D>;
  using Sm = Smem<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Sm* sm = reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const moe_kv4_attn_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hk = a.cache.kv_heads, group = a.q_heads / Hk;

  // ------------------------------------------------ tiles before each request
  if (tid == 0) {
    sm->abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->q_full[i], 4);
      mbar_init(&sm->s_full[i], 1);
      mbar_init(&sm->p_full[i], 4);
      mbar_init(&sm->o_full[i], 1);
      mbar_init(&sm->k_full[i], kDeqWarps);
      mbar_init(&sm->k_empty[i], 1);
      mbar_init(&sm->v_full[i], kDeqWarps);
      mbar_init(&sm->v_empty[i], 1);
    }
    mbar_init(&sm->drain, 1);
    fence_barrier_init();
  }
  for (int b = warp; b < p.nb; b += kThreads / 32) {   // a warp per request
    const Request r = load_request(a, p.b0 + b);
    const long long rows = (long long)r.n * group;
    int sum = 0;
    if (rows > p.min_rows)
      for (int q = lane; (long long)q * kRowTile < rows; q += 32) {
        int f;
        sum += row_tile_tiles(a, r, group, q, f);
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
    int carry = 0;
    for (int base = 0; base < p.nb; base += 32) {
      const int i = base + lane;
      int v = i < p.nb ? sm->pre[i + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
      }
      if (i < p.nb) sm->pre[i + 1] = v + carry;
      carry += __shfl_sync(kFull, v, 31);
    }
    if (lane == 0) sm->pre[0] = 0;
  }
  __syncthreads();
  const int total = sm->pre[p.nb];
  const int G = min((int)gridDim.x, total), cta = blockIdx.x;
  if (cta >= G) return;
  const int C0 = (int)((long long)total * cta / G), C1 = (int)((long long)total * (cta + 1) / G);
  if (warp == kMmaWarp) tmem_alloc(&sm->tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  volatile int* abort = &sm->abort;
  auto slot = [&](int c, int which) { return p.partials + ((size_t)c * 2 + which) * kSlotFloats<D>; };
  auto wait = [&](uint64_t* bar, int phase) {   // all lanes: the warp's common answer
    return __all_sync(kFull, mbar_wait(bar, (uint32_t)(phase & 1), abort, p.wait_limit)) != 0;
  };
  Pieces pc(a, sm->pre, p.b0, p.nb, group, C0, C1);

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------- softmax
    const int i = warp >> 2;                       // row tile of this warpgroup
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + lanes + 128 * i, o_t = tmem + lanes + 256 + 128 * i;
    int js = 0, jo = 0;                            // S tiles and items this warpgroup has seen
    int jt = 0;                                    // tiles of the CTA before the current piece
    bool ok = true;
    for (; pc.more() && ok; pc.next()) {
      const int rows = pc.rows(), nt = pc.t1 - pc.t0;
      const int jt0 = jt;
      jt += nt;
      if (i * 128 >= rows) continue;
      const int r = i * 128 + (warp & 3) * 32 + lane;   // row within the item
      const bool real = r < rows, active = i * 128 + (warp & 3) * 32 < rows;
      const int rr = pc.q * kRowTile + (real ? r : 0), token = rr / group;
      const size_t at = (size_t)(pc.rq.row0 + token) * a.q_heads + pc.h * group + rr % group;
      // the row as f16, largest element in [2^14, 2^15)
      float c;
      {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (size_t)(pc.rq.row0 + token) * a.q_stride +
                                                          (pc.h * group + rr % group) * D);
        uint32_t mx = 0;
#pragma unroll
        for (int v = 0; v < D / 8; ++v) {
          const uint4 w = __ldg(src + v);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mx = max(mx, max(finite_mag(ww[j] & 0x7fffu), finite_mag((ww[j] >> 16) & 0x7fffu)));
        }
        const int ex = min(max((int)(mx >> 7), 1), 254);
        float2 up = pow2_pair(141 - ex);
        const float2 dn = pow2_pair(ex - 141);
        // never 0, so that a hidden score stays -inf
        c = fmaxf(fabsf(a.scale) * kLog2e / a.cache.k_gs * dn.x * dn.y, 1e-37f);
        if (a.scale < 0.0f) up.x = -up.x;          // so that larger scores stay larger products
        const uint32_t dst = smem_u32(&sm->q[i][0]);
#pragma unroll 4
        for (int v = 0; v < D / 8; ++v) {
          const uint4 w = __ldg(src + v);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = pack_f16x2(__uint_as_float(ww[j] << 16) * up.x * up.y,
                              __uint_as_float(ww[j] & 0xffff0000u) * up.x * up.y);
          sts16(dst + tile_chunk(r & 127, v), make_uint4(o[0], o[1], o[2], o[3]));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->q_full[i]);
      const int hi_tok = a.causal ? pc.rq.kv - pc.rq.n + token : pc.rq.kv - 1;
      const int lo_tok = a.window > 0 ? hi_tok - a.window + 1 : 0;
      float m = -INFINITY, l0 = 0.0f, l1 = 0.0f;
      for (int t = 0; t < nt; ++t, ++js) {
        if (!(ok = wait(&sm->s_full[i], js))) break;
        tc_fence_after();
        if (active) {
          const int tok0 = pc.first + (pc.t0 + t) * kTok;
          const uint64_t hole = *reinterpret_cast<const volatile uint64_t*>(sm->hole[(jt0 + t) & 3]);
          const bool masked = __any_sync(kFull, tok0 + kTok - 1 > hi_tok || tok0 < lo_tok) || hole != 0;
#pragma unroll 1
          for (int piece = 0; piece < 4; ++piece) {
            uint32_t sr[32];
            tmem_ld32(s_t + 32 * piece, sr);
            tmem_ld_wait();
            float s[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = __uint_as_float(sr[e]);
            if (masked) {
              const int base = tok0 + 32 * piece;
              const uint32_t bad = (uint32_t)(hole >> (16 * piece)) & 0xffffu;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (base + e > hi_tok || base + e < lo_tok || (bad >> (8 * (e / 16)) & 0xffu)) s[e] = -INFINITY;
            }
            float t0 = fmaxf(s[0], s[1]), t1 = fmaxf(s[2], s[3]);
#pragma unroll
            for (int e = 4; e < 32; e += 4) {
              t0 = fmaxf(t0, fmaxf(s[e], s[e + 1]));
              t1 = fmaxf(t1, fmaxf(s[e + 2], s[e + 3]));
            }
            const float top = fmaxf(t0, t1) * c;
            if (__any_sync(kFull, top > m + kSlack)) {
              const float mn = fmaxf(m, top), f = mn == -INFINITY ? 1.0f : ex2(m - mn);
              m = mn;
              l0 *= f;
              l1 *= f;
              if (t > 0) {
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
              const uint32_t f2 = pack_f16x2(f, f);   // pieces of P already stored: one more f16 rounding
#pragma unroll 1
              for (int pp = 0; pp < piece; ++pp) {
                uint32_t o[16];
                tmem_ld16(s_t + 16 * pp, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = hmul2_u32(o[e], f2);
                tmem_st16(s_t + 16 * pp, o);
              }
              tmem_st_wait();
            }
            const float mu = m == -INFINITY ? 0.0f : m;
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float p0 = ex2(fmaf(s[2 * e], c, -mu)), p1 = ex2(fmaf(s[2 * e + 1], c, -mu));
              l0 += p0;
              l1 += p1;
              pk[e] = pack_f16x2(p0, p1);
            }
            tmem_st16(s_t + 16 * piece, pk);
          }
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->p_full[i]);
      }
      if (!ok || !(ok = wait(&sm->o_full[i], jo))) break;
      ++jo;
      tc_fence_after();
      if (!active) continue;
      const float l = l0 + l1;
      if (pc.whole()) {
        const float inv = l > 0.0f ? 1.0f / (l * a.cache.v_gs) : 0.0f;
        uint4* out = reinterpret_cast<uint4*>(a.out + at * D);
#pragma unroll
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t o[32];
          tmem_ld32(o_t + cc, o);
          tmem_ld_wait();
          if (real) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = l > 0.0f ? float2_to_bf16x2_bits(__uint_as_float(o[e + 2 * j]) * inv,
                                                        __uint_as_float(o[e + 2 * j + 1]) * inv)
                                : 0u;
              out[(cc + e) / 8] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (real && a.lse != nullptr) a.lse[at] = l > 0.0f ? m * kLn2 + logf(l) : -INFINITY;
      } else {
        float* dst = slot(cta, pc.t0 > 0 ? 0 : 1);
#pragma unroll
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t o[32];
          tmem_ld32(o_t + cc, o);
          tmem_ld_wait();
          if (real) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(dst + r * D + cc + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        if (real) *reinterpret_cast<float2*>(dst + kRowTile * D + 2 * r) = make_float2(m, l);
      }
      tc_fence_before();
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------- dequant
    const int blk0 = (warp - kSoftWarps) * kWarpBlocks;   // this warp's 16-token blocks of every tile
    constexpr int kLoads = D / 64;                 // 16-byte code loads per lane for a block's keys
    constexpr int kChunks = D / 32;                // 16-byte code chunks of a row
    const int cl = lane % kChunks, tl = lane / kChunks;   // this lane's chunk, and its row within a load
    constexpr int kRowsPerLoad = 32 / kChunks;
    const int P = a.cache.page_tokens;
    struct Raw {
      uint4 codes[kWarpBlocks][kLoads];
      uint32_t sf[kWarpBlocks][kLoads];            // two scale bytes each
    } rk, rv;
    const uint8_t* src[kWarpBlocks];
    int left[kWarpBlocks];                         // tokens of the block that exist
    bool hole[kWarpBlocks];
    int lt = pc.t0;
    auto locate = [&]() {                          // the walk's next tile
#pragma unroll
      for (int x = 0; x < kWarpBlocks; ++x) {
        left[x] = 0;
        hole[x] = false;
      }
      if (!pc.more()) return;
#pragma unroll
      for (int x = 0; x < kWarpBlocks; ++x) {
        const int tok = pc.first + lt * kTok + (blk0 + x) * kKvBlock;
        if (tok < pc.rq.kv) {
          const int page = __ldg(a.block_table + (size_t)(pc.b0 + pc.b) * a.max_pages + tok / P);
          hole[x] = page < 0 || page >= a.cache.num_pages;
          if (!hole[x]) {
            left[x] = pc.rq.kv - tok;
            src[x] = static_cast<const uint8_t*>(a.cache.pool) +
                     kv4_block_offset(page, pc.h, Hk, P / kKvBlock, tok % P / kKvBlock, L::kBytes);
          } else if (lane == 0) {
            set_status(p.status, MOE_ERR_DEVICE);
          }
        }
      }
      if (++lt == pc.t1) {
        pc.next();
        lt = 0;
      }
    };
    auto load = [&](Raw& r, int codes, int scales) {
#pragma unroll
      for (int x = 0; x < kWarpBlocks; ++x)
#pragma unroll
        for (int y = 0; y < kLoads; ++y) {
          const int row = y * kRowsPerLoad + tl;
          r.codes[x][y] = make_uint4(0u, 0u, 0u, 0u);   // what was not appended enters as zeros
          r.sf[x][y] = 0u;
          if (row < left[x]) {
            r.codes[x][y] = __ldg(reinterpret_cast<const uint4*>(src[x] + codes + row * L::kCodeRow + 16 * cl));
            r.sf[x][y] = __ldg(reinterpret_cast<const uint16_t*>(src[x] + scales + row * L::kScaleRow + 2 * cl));
          }
        }
    };
    auto store = [&](uint32_t tile, const Raw& r) {
#pragma unroll
      for (int x = 0; x < kWarpBlocks; ++x)
#pragma unroll
        for (int y = 0; y < kLoads; ++y) {
          const int row = (blk0 + x) * kKvBlock + y * kRowsPerLoad + tl;
          const uint32_t two = cvt_e4m3x2_f16x2(r.sf[x][y]);
          const uint32_t s0 = __byte_perm(two, 0, 0x1010), s1 = __byte_perm(two, 0, 0x3232);
          const uint32_t w[4] = {r.codes[x][y].x, r.codes[x][y].y, r.codes[x][y].z, r.codes[x][y].w};
          uint4 f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t h[4];
            cvt_e2m1x8_f16(w[j], h);
            const uint32_t sc = j < 2 ? s0 : s1;
            f[j] = make_uint4(hmul2_u32(h[0], sc), hmul2_u32(h[1], sc), hmul2_u32(h[2], sc), hmul2_u32(h[3], sc));
          }
          // the two 64-column halves share banks: their lanes store in different orders
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool flip = D == 128 && cl >= 2;
            const uint4 v = flip ? f[j ^ 2] : f[j];
            sts16(tile + tile_chunk(row, 4 * cl + (flip ? j ^ 2 : j)), v);
          }
        }
    };
    locate();
    load(rk, 0, L::kKeyScales);
    load(rv, L::kValueCodes, L::kValueScales);
    const int n = C1 - C0;
    for (int j = 0; j < n; ++j) {
      const int s = j & 1, phase = (j >> 1) & 1;
      if (!wait(&sm->k_empty[s], phase ^ 1)) break;
      if (lane < kWarpBlocks) sm->hole[j & 3][blk0 + lane] = (lane == 0 ? hole[0] : hole[kWarpBlocks - 1]) ? 0xff : 0;
      store(smem_u32(&sm->k[s][0]), rk);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->k_full[s]);
      locate();
      load(rk, 0, L::kKeyScales);
      if (!wait(&sm->v_empty[s], phase ^ 1)) break;
      store(smem_u32(&sm->v[s][0]), rv);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->v_full[s]);
      load(rv, L::kValueCodes, L::kValueScales);
    }
  } else {
    // ------------------------------------------------------------------ MMA
    const uint32_t id_s = idesc_f16(128, 128, 0);
    const uint32_t id_o = idesc_f16(128, D, 0) | (1u << 16);   // values: N (d) contiguous
    constexpr int kHalf = 128 * 128;
    const uint64_t qd = smem_desc(smem_u32(&sm->q[0][0]), 16, 1024, kSwizzle128B);
    const uint64_t kd = smem_desc(smem_u32(&sm->k[0][0]), 16, 1024, kSwizzle128B);
    // MN-major: leading offset between 64-column halves, stride between 8-token groups
    const uint64_t vd = smem_desc(smem_u32(&sm->v[0][0]), kHalf, 1024, kSwizzle128B);
    auto issue_s = [&](int i, int s) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4);
        mma_f16(tmem + 128 * i, qd + (uint64_t)((i * Sm::kTile) >> 4) + off,
                kd + (uint64_t)((s * Sm::kTile) >> 4) + off, id_s, kk != 0);
      }
      tc_commit(&sm->s_full[i]);
    };
    auto issue_o = [&](int i, int s, bool first) {
#pragma unroll
      for (int kk = 0; kk < kTok / 16; ++kk)
        mma_f16_tmem_a(tmem + 256 + 128 * i, tmem + 128 * i + 8 * kk,
                       vd + (uint64_t)((s * Sm::kTile + kk * 2048) >> 4), id_o, !(first && kk == 0));
    };
    int j = 0, items0 = 0, items1 = 0, p0 = 0, p1 = 0;
    bool ok = true;
    for (; pc.more() && ok; pc.next()) {
      const int nt = pc.t1 - pc.t0, mine = pc.rows() > 128 ? 2 : 1;
      ok = wait(&sm->q_full[0], items0++);
      if (ok && mine == 2) ok = wait(&sm->q_full[1], items1++);
      if (!ok || !(ok = wait(&sm->k_full[j & 1], j >> 1))) break;
      tc_fence_after();
      if (lane == 0) {
        for (int i = 0; i < mine; ++i) issue_s(i, j & 1);
        tc_commit(&sm->k_empty[j & 1]);
      }
      __syncwarp();
      for (int t = 0; t < nt && ok; ++t, ++j) {
        const int s = j & 1;
        const bool next = t + 1 < nt;
        if (!(ok = wait(&sm->v_full[s], j >> 1))) break;
        for (int i = 0; i < mine; ++i) {
          if (!(ok = wait(&sm->p_full[i], i == 0 ? p0++ : p1++))) break;
          if (next && i == 0 && !(ok = wait(&sm->k_full[s ^ 1], (j + 1) >> 1))) break;
          tc_fence_after();
          if (lane == 0) {
            issue_o(i, s, t == 0);
            if (next) issue_s(i, s ^ 1);
            else tc_commit(&sm->o_full[i]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) {
          tc_commit(&sm->v_empty[s]);
          if (next) tc_commit(&sm->k_empty[s ^ 1]);
        }
        __syncwarp();
      }
    }
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

  // ----------------------------- row tiles that several CTAs cut: the last joins
  Pieces first(a, sm->pre, p.b0, p.nb, group, C0, C1), end(a, sm->pre, p.b0, p.nb, group, C1 - 1, C1);
  const int s0 = C0 - first.t0, s1 = s0 + first.tiles;            // tiles of the first row tile
  const int e0 = C1 - 1 - end.t0, e1 = e0 + end.tiles;            // and of the last
  const bool cut0 = s0 < C0, cut1 = e1 > C1 && e0 >= C0;
  if (!cut0 && !cut1) return;
  auto cta_of = [&](int tile) { return (int)(((long long)(tile + 1) * G - 1) / total); };
  __threadfence();
  __syncthreads();
  if (tid < 2) {
    const bool cut = tid == 0 ? cut0 : cut1;
    const int lo = cta_of(tid == 0 ? s0 : e0), hi = cta_of((tid == 0 ? s1 : e1) - 1);
    int is_last = 0;
    if (cut && atomicAdd(p.counters + lo, 1) == hi - lo) {
      p.counters[lo] = 0;   // everyone has arrived: ready for the next launch
      is_last = 1;
    }
    sm->last[tid] = is_last;
  }
  __syncthreads();
  for (int side = 0; side < 2; ++side) {
    if (!sm->last[side]) continue;
    __threadfence();
    const Pieces& pp = side == 0 ? first : end;
    const int lo = cta_of(side == 0 ? s0 : e0), n = cta_of((side == 0 ? s1 : e1) - 1) - lo + 1;
    for (int e = tid; e < pp.rows() * (D / 4); e += kThreads) {
      const int row = e / (D / 4), d = e % (D / 4) * 4;
      float m = -INFINITY;
      for (int x = 0; x < n; ++x) m = fmaxf(m, __ldcg(slot(lo + x, x == 0 ? 1 : 0) + kRowTile * D + 2 * row));
      const float mu = m == -INFINITY ? 0.0f : m;
      float l = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int x = 0; x < n; ++x) {
        const float* src = slot(lo + x, x == 0 ? 1 : 0);
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(src + kRowTile * D + 2 * row));
        const float4 v = __ldcg(reinterpret_cast<const float4*>(src + row * D + d));
        const float w = ex2(ml.x - mu);
        l += w * ml.y;
        o.x += w * v.x;
        o.y += w * v.y;
        o.z += w * v.z;
        o.w += w * v.w;
      }
      const float inv = l > 0.0f ? 1.0f / (l * a.cache.v_gs) : 0.0f;
      const int rr = pp.q * kRowTile + row;
      const size_t at = (size_t)(pp.rq.row0 + rr / group) * a.q_heads + pp.h * group + rr % group;
      *reinterpret_cast<uint2*>(a.out + at * D + d) =
          l > 0.0f ? make_uint2(float2_to_bf16x2_bits(o.x * inv, o.y * inv), float2_to_bf16x2_bits(o.z * inv, o.w * inv))
                   : make_uint2(0u, 0u);
      if (d == 0 && a.lse != nullptr) a.lse[at] = l > 0.0f ? mu * kLn2 + logf(l) : -INFINITY;
    }
  }
}

template <int D>
cudaError_t launch(const PromptArgs& p, int ctas, cudaStream_t s) {
  auto k = kv4_prompt_kernel<D>;
  constexpr size_t smem = sizeof(Smem<D>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = opt_in_smem(k, smem, done);
  if (e != cudaSuccess) return e;
  return launch_ex(false, k, dim3(ctas), dim3(kThreads), smem, s, p);
}

}  // namespace

size_t kv4_prompt_ws_floats(int head_dim) {
  return (size_t)kKvMaxCtas * 2 * (head_dim == 64 ? kSlotFloats<64> : kSlotFloats<128>);
}

moe_status launch_kv4_prompt(const moe_kv4_attn_args& a, int min_rows, int* status, int* counters, float* partials,
                             cudaStream_t s) {
  PromptArgs p;
  p.a = a;
  p.min_rows = min_rows;
  p.status = status;
  p.counters = counters;
  p.partials = partials;
  p.wait_limit = debug_wait_limit();
  const int sms = sm_count(), ctas = sms < kKvMaxCtas ? sms : kKvMaxCtas;
  for (int b0 = 0; b0 < a.batch; b0 += kChunk) {
    p.b0 = b0;
    p.nb = a.batch - b0 < kChunk ? a.batch - b0 : kChunk;
    cudaError_t e = a.cache.head_dim == 64 ? launch<64>(p, ctas, s) : launch<128>(p, ctas, s);
    if (e != cudaSuccess) return cuda_ok(e);
    count_launches(1);
  }
  return MOE_OK;
}

}  // namespace moe
