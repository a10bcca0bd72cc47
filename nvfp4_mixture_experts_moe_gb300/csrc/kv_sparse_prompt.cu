// Sparse attention for many query rows (prompts, prompt chunks): tcgen05 tiles
// of 128 query rows against the union of their tokens' lists, 64 cached tokens
// a step.
//
// Mathematics: kv_attention_decode.cu's (rows, keys and values exact in f16,
// fp32 scores and sums, p rounded to f16), over the tokens of the listed blocks
// up to the query's position.
//
// A unit is one key/value head of up to 32 neighbouring tokens (128 rows of
// their groups' heads). All its warps build the union of the lists: a bit a
// block, whose ranks give the blocks' order, and a bit a token for each block
// of the union. Then, in a CTA of which two share an SM:
// * four dequant warps convert a 16-token block each of every step, keys
//   K-major, values with d contiguous, from codes asked for a step ahead;
// * a thread issues S = Q K^T, another O += P V (an issue takes its thread 45
//   cycles and more: one thread for both took 2080 cycles a step without any
//   softmax);
// * four softmax warps have a row a thread. A warp none of whose tokens takes
//   the step's blocks leaves zeros as P without looking at S; a row whose token
//   does not has its P cleared; only where a block is not seen whole (the
//   diagonal, a bad page) is there a mask an element.
// While one CTA builds a union, enters or ends a unit, the other one's warps
// work.
//
// What bounds it (2048 rows over 32768 tokens, 16 blocks of 64 each, 32/8 heads x
// 128: 168 us; 17 by the products of each row with its own blocks): a unit
// multiplies all its rows by the union of what its tokens chose. These lists
// agree by runs of 32 tokens that are the units (58 blocks a union; other such
// lists 164); the same runs 16 tokens later (88) take 221, agreement that decays
// over 32 tokens (99) 247, nothing in common (287) 640, all tokens 916. A step of
// 64 tokens takes an SM 930 cycles (1860 in each of its CTAs), 770 of them by
// shared memory (operands of S 384, of O 128, stores of the tiles 256; Q in tensor
// memory would save a third of that, but S and O leave no columns); a unit's entry
// and end take 17,000 of its 135,000; 512 units are four for 56 of the SMs and
// three for the others.
// S whole in registers spilled (229 us), as did two threads a row (334); one
// thread issuing all products 189.
#include "kernels.cuh"
#include "kv4.cuh"
#include "kv_lookup.cuh"
#include "kv_tiles.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;
using namespace tiles;

constexpr int kStep = 64;               // cached tokens of a step
constexpr int kTokens = 32;             // query tokens of a unit: a bit each of a word
constexpr int kUnion = kTokens * kSparseTop;
constexpr int kWindow = 8192;           // blocks whose union is built at once: longer contexts take several
constexpr int kSoftWarps = 4, kDeqWarps = 4, kMmaWarp = kSoftWarps + kDeqWarps;
constexpr int kThreads = (kMmaWarp + 2) * 32;
constexpr int kTmemCols = 256;          // S of two steps, O
static_assert(kStep / kKvBlock == kDeqWarps, "a 16-token block a dequant warp");

struct Args {
  moe_kv4_sparse_args a;
  int tokens;        // query rows of a unit
  int units;
  int block_log;     // log2 of block_tokens
  int min_tokens;    // requests of at most this many belong to another kernel
  long long wait_limit;
};

template <int D>
struct Smem {
  static constexpr int kTile = kStep * D * 2;
  alignas(1024) uint8_t q[128 * D * 2];
  alignas(1024) uint8_t k[2][kTile];
  alignas(1024) uint8_t v[2][kTile];
  uint32_t mask[kUnion];                // tokens that take a block of the union
  uint32_t bits[kWindow / 32];          // blocks of the window that are in it
  uint16_t before[kWindow / 32];        // how many come before a word's
  uint16_t id[kUnion];                  // its blocks, within the window
  uint64_t q_full, s_full[2], p_full[2], pv_done[2], o_full;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], drain;
  alignas(4) uint8_t hole[4][4];        // 16-token blocks of a step whose page is bad
  int warp_sum[kThreads / 32 + 1];
  uint32_t tmem;
  int abort;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2) kv4_sparse_prompt_kernel(const __grid_constant__ Args p) {
  using L = Kv4Block<D>;
  using Sm = Smem<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Sm* sm = reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const moe_kv4_sparse_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hk = a.cache.kv_heads, group = a.q_heads / Hk, P = a.cache.page_tokens, p_log = __ffs(P) - 1;
  const int sub_log = p.block_log - 4;    // log2 of a block's 16-token blocks
  if (tid == 0) {
    sm->abort = 0;
    mbar_init(&sm->q_full, kSoftWarps);
    mbar_init(&sm->o_full, 1);
    mbar_init(&sm->drain, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->s_full[i], 1);
      mbar_init(&sm->pv_done[i], 1);
      mbar_init(&sm->p_full[i], kSoftWarps);
      mbar_init(&sm->k_full[i], kDeqWarps);
      mbar_init(&sm->v_full[i], kDeqWarps);
      mbar_init(&sm->k_empty[i], 1);
      mbar_init(&sm->v_empty[i], 1);
    }
    fence_barrier_init();
  }
  pdl_wait();
  if (warp == kMmaWarp) tmem_alloc(&sm->tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem, o_tmem = tmem + 2 * kStep;
  volatile int* const abort = &sm->abort;
  auto wait = [&](uint64_t* bar, int phase) {   // all lanes: the warp's common answer
    return __all_sync(kFull, mbar_wait(bar, (uint32_t)(phase & 1), abort, p.wait_limit)) != 0;
  };
  int js = 0;          // steps of the CTA so far, the same for every warp
  int jq = 0;          // runs of rows

  for (int unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
    const int h = unit % Hk, t_end = min((unit / Hk + 1) * p.tokens, a.total_q);
    // The rows of the unit that belong to one request, then those of the next.
    for (int t = unit / Hk * p.tokens, ntok; t < t_end; t += ntok) {
      const RowOwner own = row_owner(a.cu_q, a.kv_len, a.batch, a.total_q, a.max_q, a.max_pages * P, t);
      if (own.bad && tid == 0 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
      ntok = own.n > 0 ? min(t_end, own.c0 + own.n) - t : t_end - t;
      if (own.b < 0 || own.n <= p.min_tokens) continue;
      const int pos0 = own.kv - own.n + t - own.c0;            // the first row's position
      const int last = pos0 + ntok - 1, entries = ntok * a.top;
      const int32_t* const blocks = a.blocks + ((size_t)t * Hk + h) * a.top;
      const size_t stride = (size_t)Hk * a.top;                // of blocks
      const int32_t* const table = a.block_table + (size_t)own.b * a.max_pages;
      const int rows = ntok * group;

      // what a softmax thread has of its row
      const int token = min(tid / group, ntok - 1), pos = pos0 + token;
      const bool real = warp < kSoftWarps && tid < rows;
      const size_t at = (size_t)(t + token) * a.q_heads + h * group + tid % group;
      float m = -INFINITY, c = 0.0f;
      uint64_t l2 = pack2(0.0f, 0.0f);
      int steps_so_far = 0;
      bool entered = false;

      for (int base = 0; base <= last >> p.block_log || base == 0; base += kWindow) {
        // --------------------------------------------- the union of the lists
        __syncthreads();   // the last one is no longer in use
        for (int i = tid; i < kWindow / 32; i += kThreads) sm->bits[i] = 0;
        __syncthreads();
        for (int e = tid; e < entries; e += kThreads) {
          const int i = e / a.top, x = __ldg(blocks + i * stride + e - i * a.top);
          if (x >= base && x - base < kWindow && pos0 + i >= 0 && x <= (pos0 + i) >> p.block_log)
            atomicOr(&sm->bits[(x - base) >> 5], 1u << (x & 31));
        }
        __syncthreads();
        const uint32_t word = tid < kWindow / 32 ? sm->bits[tid] : 0u;
        int incl = __popc(word);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(kFull, incl, o);
          if (lane >= o) incl += v;
        }
        if (lane == 31) sm->warp_sum[warp] = incl;
        __syncthreads();
        int count = 0, k = incl - __popc(word);
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
          const int v = sm->warp_sum[w];
          if (w < warp) k += v;
          count += v;
        }
        if (tid < kWindow / 32) {
          sm->before[tid] = (uint16_t)k;
          for (uint32_t left = word; left; left &= left - 1, ++k) {
            sm->id[k] = (uint16_t)(tid * 32 + __ffs(left) - 1);
            sm->mask[k] = 0;
          }
        }
        __syncthreads();
        for (int e = tid; e < entries; e += kThreads) {
          const int i = e / a.top, x = __ldg(blocks + i * stride + e - i * a.top);
          if (x >= base && x - base < kWindow && pos0 + i >= 0 && x <= (pos0 + i) >> p.block_log) {
            const int w = (x - base) >> 5;
            atomicOr(&sm->mask[sm->before[w] + __popc(sm->bits[w] & ((1u << (x & 31)) - 1))], 1u << i);
          }
        }
        __syncthreads();
        const int steps = ((count << sub_log) + kDeqWarps - 1) / kDeqWarps;
        if (steps == 0) continue;
        const bool first = steps_so_far == 0;
        steps_so_far += steps;
        // entry of the union that 16-token block x of step s belongs to
        auto entry = [&](int s, int x) { return (s * kDeqWarps + x) >> sub_log; };

        if (warp < kSoftWarps) {
          // ----------------------------------------------------------- softmax
          const uint32_t lanes = (uint32_t)(warp * 32) << 16;
          bool ok = true;
          if (!entered) {
            // The rows as f16 times a power of two that puts the largest element in [2^14, 2^15) (smaller only below
            // 2^-112); a row's 16-byte pieces come by neighbouring lanes.
            const uint4* src =
                reinterpret_cast<const uint4*>(a.q + (size_t)(t + token) * a.q_stride + (h * group + tid % group) * D);
            constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks;
            const uint32_t dst = smem_u32(sm->q);
#pragma unroll
            for (int v = 0; v < kChunks; ++v) {
              const uint4 x = __ldg(reinterpret_cast<const uint4*>(__shfl_sync(
                                        kFull, reinterpret_cast<unsigned long long>(src), v * kAtOnce + lane / kChunks)) +
                                    lane % kChunks);
              sts16(dst + tile_chunk<>(warp * 32 + v * kAtOnce + lane / kChunks, lane % kChunks), x);
            }
            __syncwarp();
            uint32_t mx = 0;
#pragma unroll
            for (int v = 0; v < kChunks; ++v) {
              const uint4 x = *reinterpret_cast<const uint4*>(sm->q + tile_chunk<>(tid, v));
              mx = max_u16x2(max_u16x2(mx, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
              mx = max_u16x2(max_u16x2(mx, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
            }
            const uint32_t big = max(mx & 0xffffu, mx >> 16);
            const int ex = min(max((int)(big >> 7), 15), 254);
            // never 0, so that a hidden score stays -inf
            c = fmaxf(fabsf(a.scale) * kLog2e / a.cache.k_gs * pow2(ex - 141), 1e-37f);
            // a larger score is a larger product; a row with a NaN or an infinity has no softmax whatever it sees: all NaN
            const float up = big >= 0x7f80u ? __int_as_float(0x7fffffff) : a.scale < 0.0f ? -pow2(141 - ex) : pow2(141 - ex);
#pragma unroll 4
            for (int v = 0; v < kChunks; ++v) {
              uint4* chunk = reinterpret_cast<uint4*>(sm->q + tile_chunk<>(tid, v));
              uint4 x = *chunk;
              uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                xw[j] = pack_f16x2(__uint_as_float(xw[j] << 16) * up, __uint_as_float(xw[j] & 0xffff0000u) * up);
              *chunk = x;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->q_full);
          }
          for (int s = 0; s < steps; ++s) {
            const int j = js + s, buf = j & 1;
            const uint32_t s_t = tmem + lanes + kStep * buf;
            // which of the step's two halves this row's token takes
            const int e0 = entry(s, 0), e1 = entry(s, 2);
            const uint32_t who0 = sm->mask[e0], who1 = e1 < count ? sm->mask[e1] : 0u;
            const bool take0 = who0 >> token & 1, take1 = who1 >> token & 1;
            if (!(ok = wait(&sm->s_full[buf], j >> 1))) break;
            tc_fence_after();
            if (!__any_sync(kFull, real && (take0 || take1))) {
              uint32_t zero[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) zero[i] = 0u;
              tmem_st16(s_t, zero);
              tmem_st16(s_t + 16, zero);
            } else {
              const uint32_t hole = *reinterpret_cast<const volatile uint32_t*>(&sm->hole[j & 3][0]);
              const int tok0 = ((base + sm->id[e0]) << p.block_log) + ((s * kDeqWarps) & ((1 << sub_log) - 1)) * kKvBlock;
              const int tok1 = sub_log > 1 ? tok0 + kStep / 2
                                           : e1 < count ? (base + sm->id[e1]) << p.block_log : tok0;
              const bool partial = __any_sync(kFull, real && ((take0 && tok0 + kStep / 2 - 1 > pos) ||
                                                              (take1 && tok1 + kStep / 2 - 1 > pos))) || hole != 0;
              const bool some = !__all_sync(kFull, !real || (take0 && take1));   // rows that do not take it all
              // A half of S at a time: 96 registers a thread are what two CTAs an SM leave, so the second half is read
              // once more for its exponentials.
              uint32_t sr[32];
              auto read = [&](int piece) {
                tmem_ld32(s_t + 32 * piece, sr);
                ld_wait(sr);
                if (partial) {   // bit e: column e is seen
                  const int hi = pos - (piece ? tok1 : tok0);
                  uint32_t see = hi >= 31 ? ~0u : hi < 0 ? 0u : (2u << hi) - 1u;
                  const uint32_t bad = hole >> (16 * piece);
                  if (bad & 0xffu) see &= 0xffff0000u;
                  if (bad & 0xff00u) see &= 0x0000ffffu;
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (!(see >> e & 1u)) sr[e] = 0xff800000u;
                }
              };
              auto peak = [&]() {
                float u0 = __uint_as_float(sr[0]), u1 = __uint_as_float(sr[1]);
#pragma unroll
                for (int e = 2; e < 30; e += 4) {
                  u0 = max3(u0, __uint_as_float(sr[e]), __uint_as_float(sr[e + 1]));
                  u1 = max3(u1, __uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3]));
                }
                return max3(u0, u1, fmaxf(__uint_as_float(sr[30]), __uint_as_float(sr[31])));
              };
              read(1);
              const float p1 = peak();
              read(0);
              const float top = fmaxf(take0 ? peak() : -INFINITY, take1 ? p1 : -INFINITY) * c;
              if (__any_sync(kFull, top > m + kSlack)) {
                const float mn = fmaxf(m, top - kLead), f = mn == -INFINITY ? 1.0f : ex2(m - mn);
                m = mn;
                const float2 l = unpack2(l2);
                l2 = pack2(l.x * f, l.y * f);
                if (!first || s > 0) {   // O holds the steps before, once the last of them has gone in
                  if (!(ok = wait(&sm->pv_done[(j - 1) & 1], (j - 1) >> 1))) break;
                  tc_fence_after();
#pragma unroll 1
                  for (int cc = 0; cc < D; cc += 16) {
                    uint32_t o[16];
                    tmem_ld16(o_tmem + lanes + cc, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                    tmem_st16(o_tmem + lanes + cc, o);
                  }
                }
              }
              const float mu = m == -INFINITY ? 0.0f : m;
              const uint64_t m2 = pack2(-mu, -mu), c2 = pack2(c, c);
              auto exps = [&](uint32_t (&pk)[16], bool take) {
                uint64_t sum = pack2(0.0f, 0.0f);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 y = unpack2(fma2(pack2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), c2, m2));
                  const float x0 = ex2(y.x), x1 = ex2(y.y);
                  sum = add2(sum, pack2(x0, x1));
                  pk[e] = pack_f16x2(x0, x1);
                }
                if (some) {   // whatever the scores of a row that does not take the block are
                  const uint32_t keep = take ? ~0u : 0u;
#pragma unroll
                  for (int e = 0; e < 16; ++e) pk[e] &= keep;
                  if (!take) sum = pack2(0.0f, 0.0f);
                }
                l2 = add2(l2, sum);
              };
              uint32_t pk0[16], pk1[16];
              exps(pk0, take0);
              read(1);
              exps(pk1, take1);
              tmem_st16(s_t, pk0);   // P takes the columns of S, read by then
              tmem_st16(s_t + 16, pk1);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->p_full[buf]);
          }
        } else if (warp < kMmaWarp) {
          // ----------------------------------------------------------- dequant
          const int x = warp - kSoftWarps;             // this warp's 16-token block of every step
          constexpr int kLoads = D / 64;               // 16-byte code loads a lane for a block's keys
          // This lane's 16-byte piece of a row's codes (32 elements) and its row within a load. Eight neighbouring lanes
          // take two neighbouring pieces of four rows: their stores to the swizzled tile hit different banks.
          const int cl = (lane & 1) + (D == 128 ? lane >> 4 << 1 : 0), tl = D == 128 ? lane >> 1 & 7 : lane >> 1;
          constexpr int kRowsPerLoad = D == 128 ? 8 : 16;
          struct Raw {
            uint4 codes[kLoads];
            uint32_t sf[kLoads];                       // two scale bytes each
          };
          // A step's block goes through three stages, a step apart: its page id is asked for, its codes are, it is
          // converted (the keys behind one more step's).
          struct Block {
            int page, tok;                             // tok < 0: there is none
            int to;                                    // its tokens that are there; -1: the page is bad
            Raw k, v;
          } blk;
          auto look_up = [&](Block& b, int s) {
            const int e = s < steps ? entry(s, x) : count;
            b.tok = -1;
            if (e >= count) return;
            const int tok = ((base + sm->id[e]) << p.block_log) + ((s * kDeqWarps + x) & ((1 << sub_log) - 1)) * kKvBlock;
            if (tok >= own.kv) return;
            b.tok = tok;
            b.page = __ldg(table + (tok >> p_log));
          };
          auto load = [&](Raw& r, const uint8_t* src, auto there) {
            const uint8_t *codes = src + tl * L::kCodeRow + 16 * cl, *scales = src + L::kKeyScales + tl * L::kScaleRow + 2 * cl;
#pragma unroll
            for (int y = 0; y < kLoads; ++y) {
              r.codes[y] = make_uint4(0u, 0u, 0u, 0u);   // what may not have been appended enters as zeros
              r.sf[y] = 0u;
              if (there(y * kRowsPerLoad + tl)) {
                r.codes[y] = __ldg(reinterpret_cast<const uint4*>(codes + y * kRowsPerLoad * L::kCodeRow));
                r.sf[y] = __ldg(reinterpret_cast<const uint16_t*>(scales + y * kRowsPerLoad * L::kScaleRow));
              }
            }
          };
          auto fetch = [&](Block& b) {
            const uint8_t* src = nullptr;
            b.to = 0;
            if (b.tok >= 0) {
              if (b.page >= 0 && b.page < a.cache.num_pages) {
                src = static_cast<const uint8_t*>(a.cache.pool) +
                      kv4_block_offset(b.page, h, Hk, P / kKvBlock, (b.tok & (P - 1)) / kKvBlock, L::kBytes);
                b.to = own.kv - b.tok;
              } else {
                b.to = -1;
                if (lane == 0 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
              }
            }
            auto both = [&](auto there) {
              load(b.k, src, there);
              load(b.v, src + L::kValueCodes, there);
            };
            if (b.to >= kKvBlock) both([](int) { return true; });   // one branch for all: 182 us with one for each load
            else both([&](int row) { return row < b.to; });
          };
          uint32_t off[4];                             // of this lane's four 16-byte stores, in a tile
#pragma unroll
          for (int i = 0; i < 4; ++i) off[i] = tile_chunk<kStep>(x * kKvBlock + tl, 4 * cl + i);
          auto store = [&](uint32_t tile, const Raw& r) {
#pragma unroll
            for (int y = 0; y < kLoads; ++y) {
              const uint32_t two = cvt_e4m3x2_f16x2(r.sf[y]);
              const uint32_t sc0 = __byte_perm(two, 0, 0x1010), sc1 = __byte_perm(two, 0, 0x3232);
              const uint32_t wd[4] = {r.codes[y].x, r.codes[y].y, r.codes[y].z, r.codes[y].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t f[4];
                cvt_e2m1x8_f16(wd[i], f);
                const uint32_t sc = i < 2 ? sc0 : sc1;
                sts16(tile + off[i] + y * kRowsPerLoad * 128,
                      make_uint4(hmul2_u32(f[0], sc), hmul2_u32(f[1], sc), hmul2_u32(f[2], sc), hmul2_u32(f[3], sc)));
              }
            }
          };
          look_up(blk, 0);
          fetch(blk);
          look_up(blk, 1);
          for (int s = 0; s < steps; ++s) {
            const int j = js + s, st = j & 1;
            if (!wait(&sm->k_empty[st], (j >> 1) ^ 1)) break;
            if (lane == 0) sm->hole[j & 3][x] = blk.to < 0 ? 0xff : 0;
            store(smem_u32(sm->k[st]), blk.k);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->k_full[st]);
            if (!wait(&sm->v_empty[st], (j >> 1) ^ 1)) break;
            store(smem_u32(sm->v[st]), blk.v);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->v_full[st]);
            fetch(blk);
            look_up(blk, s + 2);
          }
        } else {
          // --------------------------------------------------------------- MMA
          bool ok = true;
          const bool one = elect_one();   // (by lane 0 on its own 179 us)
          if (warp == kMmaWarp) {
            constexpr uint32_t id_s = idesc_f16(128, kStep, 0);
            const uint64_t qd = smem_desc(smem_u32(sm->q), 16, 1024, kSwizzle128B);
            const uint64_t kd = smem_desc(smem_u32(sm->k[0]), 16, 1024, kSwizzle128B);
            if (!entered) ok = wait(&sm->q_full, jq);
            for (int s = 0; s < steps && ok; ++s) {
              const int j = js + s, st = j & 1;
              // the columns' last P has gone into O
              if (!(ok = wait(&sm->k_full[st], j >> 1) && wait(&sm->pv_done[st], (j >> 1) ^ 1))) break;
              tc_fence_after();
              if (one) {
                const uint64_t kb = kd + (uint64_t)((st * Sm::kTile) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                  mma_f16(tmem + kStep * st, qd + (uint64_t)(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4),
                          kb + (uint64_t)(((kk >> 2) * (kStep * 128) + (kk & 3) * 32) >> 4), id_s, kk != 0);
                tc_commit(&sm->s_full[st]);
                tc_commit(&sm->k_empty[st]);
              }
              __syncwarp();
            }
          } else {
            constexpr uint32_t id_o = idesc_f16(128, D, 0) | (1u << 16);   // values: N (d) contiguous
            // MN-major: leading offset between 64-column halves, stride between 8-token groups
            const uint64_t vd = smem_desc(smem_u32(sm->v[0]), kStep * 128, 1024, kSwizzle128B);
            for (int s = 0; s < steps && ok; ++s) {
              const int j = js + s, st = j & 1;
              if (!(ok = wait(&sm->v_full[st], j >> 1) && wait(&sm->p_full[st], j >> 1))) break;
              tc_fence_after();
              if (one) {
                const uint64_t vb = vd + (uint64_t)((st * Sm::kTile) >> 4);
#pragma unroll
                for (int kk = 0; kk < kStep / 16; ++kk)
                  mma_f16_tmem_a(o_tmem, tmem + kStep * st + 8 * kk, vb + kk * (2048 >> 4), id_o, !first || s > 0 || kk > 0);
                tc_commit(&sm->pv_done[st]);
                tc_commit(&sm->v_empty[st]);
              }
              __syncwarp();
            }
          }
        }
        entered = true;
        js += steps;
      }

      // --------------------------------------------------------- the results
      if (steps_so_far > 0) {
        // by the lane that issued (the elected one, each time the same): a commit is for its own thread's operations
        if (warp == kMmaWarp + 1 && elect_one()) tc_commit(&sm->o_full);
        if (warp < kSoftWarps && wait(&sm->o_full, jq)) {
          tc_fence_after();
          const float2 two = unpack2(l2);
          const float l = two.x + two.y, inv = l == 0.0f ? 0.0f : 1.0f / (l * a.cache.v_gs);   // NaN stays NaN
          const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t o[32];
            tmem_ld32(o_tmem + ((uint32_t)(warp * 32) << 16) + cc, o);
            ld_wait(o);
            if (!real) continue;
            uint16_t* out = a.out + at * D + cc;
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t b[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                b[i] = l == 0.0f ? 0u : float2_to_bf16x2_bits(__uint_as_float(o[e + 2 * i]) * inv,
                                                              __uint_as_float(o[e + 2 * i + 1]) * inv);
              if (wide) {   // a whole sector a thread
                stg_v8(out + e, b);
              } else {
                reinterpret_cast<uint4*>(out + e)[0] = make_uint4(b[0], b[1], b[2], b[3]);
                reinterpret_cast<uint4*>(out + e)[1] = make_uint4(b[4], b[5], b[6], b[7]);
              }
            }
          }
          if (real && a.lse != nullptr) a.lse[at] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
          tc_fence_before();
        }
        ++jq;
      } else if (real) {   // nothing listed
        uint4* const out = reinterpret_cast<uint4*>(a.out + at * D);
        for (int i = 0; i < D / 8; ++i) out[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse != nullptr) a.lse[at] = -INFINITY;
      }
    }
  }
  if (warp >= kMmaWarp && elect_one()) {   // what was issued is complete before tensor memory is given back
    tc_commit(&sm->drain);
    const long long t0 = clock64();
    while (!mbar_try_wait(&sm->drain, 0) && clock64() - t0 < 4000000000ll) {
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
  if (tid == 0 && sm->abort && a.device_status != nullptr) set_status(a.device_status, MOE_ERR_TIMEOUT);
}

template <int D>
cudaError_t launch(Args& p, cudaStream_t s) {
  auto k = kv4_sparse_prompt_kernel<D>;
  constexpr size_t smem = sizeof(Smem<D>) + 1024;
  static_assert(2 * (smem + 1024) <= 228 * 1024, "two CTAs an SM");
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(k, smem, done);
  if (e != cudaSuccess) return e;
  const int ctas = p.units < 2 * sm_count() ? p.units : 2 * sm_count();
  return launch_ex(true, k, dim3(ctas), dim3(kThreads), smem, s, p);
}

}  // namespace

moe_status launch_kv4_sparse_prompt(const moe_kv4_sparse_args& a, int min_tokens, cudaStream_t s) {
  Args p;
  p.a = a;
  p.block_log = __builtin_ctz(a.block_tokens);
  p.min_tokens = min_tokens;
  p.wait_limit = debug_wait_limit();
  const int group = a.q_heads / a.cache.kv_heads, most = 128 / group;
  p.tokens = most < kTokens ? most : kTokens;
  p.units = (int)(((long long)a.total_q + p.tokens - 1) / p.tokens * a.cache.kv_heads);
  const cudaError_t e = a.cache.head_dim == 64 ? launch<64>(p, s) : launch<128>(p, s);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

}  // namespace moe
