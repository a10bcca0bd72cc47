// Attention of each query over the cached blocks of its own list.
//
// Mathematics: kv_attention_decode.cu's, over the tokens of the listed blocks
// up to the query's position.
//
// A unit of work is one key/value head of up to `tile` neighbouring query rows
// (as many as fit the 8 or 16 rows of a matrix product with the group's heads)
// and the union of their lists: each block of it is converted once, and a bit
// a row says who attends to it. The union is a set, so lists may come in any
// order. A unit belongs to one warp where there are many of them, to several
// warps, a CTA or a cluster of CTAs where there are few, each with an equal
// share of the unit's tiles and a private ring of stages; their partial results
// meet in shared memory (of the cluster), in the order of the shares.
//
// What bounds it: for batches (64 single tokens, 32 blocks of 64 each, 64/8
// heads x 128: 39 us, 22.5 by the bytes) what a unit does before its first tile
// (lengths, list, page ids, rows), which nothing covers where every group of
// four warps has one unit of 16 tiles a warp, and 24 of the 152 SMs, which have
// none: 840 tiles a us, where attention over all tokens does the same work on
// 1220 (a scheduler's four warps issue in 0.6 of the cycles in both). The chain
// lengths, lists, page ids, rows, joins for few (one token 9.4 us; 16 requests of
// 4 drafted ones, 24 blocks of 32, 32/8 x 64, 13.9).
#include <cooperative_groups.h>

#include "kernels.cuh"
#include "kv4.cuh"
#include "kv_lookup.cuh"
#include "kv_rows.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace rows;
using namespace tc;

constexpr int kListMax = 256;   // entries of a unit's lists: tile * top
constexpr int kRawMax = kListMax + 3 * 8;   // with places of whole 16 bytes each, of up to 8 tokens

struct SparseArgs {
  moe_kv4_sparse_args a;
  int tile;       // query rows of a unit
  int split;      // warps of a CTA that share a unit
  int cluster;    // CTAs that share one (split is then a whole CTA)
  int units;
  int block_log;  // log2 of block_tokens
  int per;        // units of a request and head, of up to kSparseFewTokens rows (longer ones are another kernel's); 0: units
                  // are runs of all rows
};

// A tile is 4608 bytes of one head: 2 blocks of 16 tokens at D = 128, 4 at 64.
template <int D, int NT>
struct Shape {
  static constexpr int kWarps = NT == 1 ? 16 : 12;
  static constexpr int kBlocks = 256 / D;
  static constexpr int kStageBytes = kBlocks * Kv4Block<D>::kBytes;
  static constexpr int kStages = NT == 1 ? 3 : 4;
  static constexpr int kThreads = kWarps * 32;
};

template <int D, int NT>
struct Smem {
  using Sh = Shape<D, NT>;
  alignas(128) uint8_t ring[Sh::kWarps][Sh::kStages][Sh::kStageBytes];
  uint16_t list[Sh::kWarps][kListMax];   // the union: place in the lists, and rows (high byte)
  static_assert(Sh::kStageBytes >= kRawMax * 4, "the lists fit a stage");
  static_assert(Sh::kStages * Sh::kStageBytes >= 2 * Slots<D, NT>::kFloats * 4, "a ring holds two partials");
};

__device__ __forceinline__ void group_sync(int group, int split) {
  if (split == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(split * 32) : "memory");
}

// Joins n partials in their order: element e (four neighbouring columns of a
// row) of threads `mine`, `mine` + stride, ...
template <int D, int NT, class Src, class Put>
__device__ __forceinline__ void join(int n, int rows_used, int mine, int stride, bool swizzled, Src src, Put put) {
  constexpr int kRows = 8 * NT, kBatch = 4;
  for (int e = mine; e < rows_used * (D / 4); e += stride) {
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
          v[j] = *reinterpret_cast<const float4*>(s + row * D + (swizzled ? warp_chunk(row, d / 4) : d / 4) * 4);
        }
      }
      x.add(ml, v);
    }
    put(row, d, x);
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, 1) kv4_sparse_kernel(const __grid_constant__ SparseArgs p) {
  using Sh = Shape<D, NT>;
  using L = Kv4Block<D>;
  constexpr int S = Sh::kStages, kRows = 8 * NT, MT = D / 16;
  constexpr int NB = Sh::kBlocks, kPart = NT == 1 ? NB : 2;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<D, NT>* sm = reinterpret_cast<Smem<D, NT>*>(smem_raw);
  const moe_kv4_sparse_args& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, t4 = lane & 3;
  const int P = a.cache.page_tokens, p_log = __ffs(P) - 1, Hk = a.cache.kv_heads, heads = a.q_heads / Hk;
  const int group = warp / p.split, groups = Sh::kWarps / p.split;
  const int rank = p.cluster > 1 ? (int)(blockIdx.x % p.cluster) : 0;
  const int members = p.split * p.cluster, me = rank * p.split + warp % p.split;
  const int sub_log = p.block_log - 4;                         // log2 of the 16-token blocks of a listed block
  uint8_t* const ring = &sm->ring[warp][0][0];
  uint16_t* const list = sm->list[warp];
  pdl_wait();

  for (int unit = (int)(blockIdx.x / p.cluster) * groups + group; unit < p.units;
       unit += (int)(gridDim.x / p.cluster) * groups) {
    const int h = unit % Hk;
    int t0 = unit / Hk * p.tile, t_end = min(t0 + p.tile, a.total_q);
    RowOwner own;
    if (p.per > 0) {
      own = request_of(a.cu_q, a.kv_len, a.total_q, a.max_q, a.max_pages * P, unit / Hk / p.per);
      t0 = own.c0 + unit / Hk % p.per * p.tile;
      t_end = own.b >= 0 && own.n <= kSparseFewTokens ? min(t0 + p.tile, own.c0 + own.n) : t0;
    }
    // The rows of the unit that belong to one request, then those of the next.
    for (int t = t0, nrow; t < t_end; t += nrow) {
      if (p.per == 0) own = row_owner(a.cu_q, a.kv_len, a.batch, a.total_q, a.max_q, a.max_pages * P, t);
      if (own.bad && lane == 0 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
      nrow = own.n > 0 ? min(t_end, own.c0 + own.n) - t : t_end - t;
      if (own.b < 0) continue;
      const int pos0 = own.kv - own.n + t - own.c0;              // the first row's position
      const int32_t* const blocks = a.blocks + ((size_t)t * Hk + h) * a.top;
      const int32_t* const table = a.block_table + (size_t)own.b * a.max_pages;
      const size_t row_stride = (size_t)Hk * a.top;              // of blocks

      // ------------------------------------------- the union of the lists
      // The rows are asked for now: they would wait behind all the tiles in flight.
      for (int i = 0; i < nrow; ++i)
        if (lane * 128 < heads * D * 2)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(
              reinterpret_cast<const char*>(a.q + (size_t)(t + i) * a.q_stride + (size_t)h * heads * D) + lane * 128));
      // A list has places of whole 16 bytes; -1: nothing. An entry is in the union where its list has it first.
      int* const raw = reinterpret_cast<int*>(ring);
      const int places = (a.top + 3) & ~3, entries = nrow * places;
      for (int e = lane; e < entries; e += 32) {
        const int i = e / places, k = e - i * places, x = k < a.top ? __ldg(blocks + i * row_stride + k) : -1, pos = pos0 + i;
        raw[e] = x >= 0 && pos >= 0 && x <= pos >> p.block_log ? x : -1;
      }
      __syncwarp();
      int count = 0;
#pragma unroll 1
      for (int e0 = 0; e0 < entries; e0 += 32) {
        const int e = e0 + lane, x = e < entries ? raw[e] : -1;
        unsigned mask = 0;
        bool before = false;   // it is listed before this place
#pragma unroll 1
        for (int i = 0, j = 0; i < nrow; ++i)
#pragma unroll 4
          for (int k = 0; k < places; k += 4, j += 4) {   // without branches: one took 200 cycles a round
            const int4 y = *reinterpret_cast<const int4*>(raw + j);
            const bool same = y.x == x || y.y == x || y.z == x || y.w == x;
            mask |= (unsigned)same << i;
            before |= same && j + 4 <= e;
          }
        const int4 y = *reinterpret_cast<const int4*>(raw + min(e & ~3, entries - 4));
        before |= ((e & 3) > 0 && y.x == x) || ((e & 3) > 1 && y.y == x) || ((e & 3) > 2 && y.z == x);
        const bool keep = x >= 0 && !before;
        const unsigned kept = __ballot_sync(kFull, keep);
        // its token, its place in the list, the tokens that take it
        if (keep) list[count + __popc(kept & ((1u << lane) - 1))] = (uint16_t)(e / places * a.top + e % places | mask << 8);
        count += __popc(kept);
      }
      __syncwarp();

      // ----------------------------------------------- this warp's tiles
      const int tiles = ((count << sub_log) + NB - 1) / NB, active = min(members, tiles);
      const int r0 = me < active ? (int)((long long)tiles * me / active) : 0;
      const int r1 = me < active ? (int)((long long)tiles * (me + 1) / active) : 0;
      const unsigned full = (1u << nrow) - 1;
      const int used = nrow * heads;
      auto out_row = [&](int row) { return (size_t)(t + row / heads) * a.q_heads + h * heads + row % heads; };

      RowState<D, NT> st;
      if (r0 < r1) {
        // Lane i holds where tile base + i comes from: its two halves' first
        // tokens and rows, and a place for each 16-token block.
        int d_tok[2] = {0, 0}, d_rows = 0, d_valid = 0, base = r0;
        const uint8_t* d_src[NB];
        // (fresh: the lists are still where the union was built)
        auto describe = [&](int from, bool fresh) {
          base = from;
          d_valid = d_rows = 0;
          d_tok[0] = d_tok[1] = 0;
#pragma unroll
          for (int i = 0; i < NB; ++i) d_src[i] = nullptr;
          const int tile = from + lane;
          if (tile >= r1) return;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int sub = tile * NB + half * (NB / 2), at = sub >> sub_log;
            if (at >= count) break;
            const int code = list[at], e = code & 0xff, i = e / a.top;
            const int blk = fresh ? raw[i * places + e - i * a.top] : __ldg(blocks + i * row_stride + e - i * a.top);
            d_tok[half] = (blk << p.block_log) + (sub - (at << sub_log)) * kKvBlock;
            d_rows |= code >> 8 << (8 * half);
#pragma unroll
            for (int j = 0; j < NB / 2; ++j) {
              const int tok = d_tok[half] + j * kKvBlock;
              if (tok >= own.kv) break;
              const int page = __ldg(table + (tok >> p_log));
              if (page >= 0 && page < a.cache.num_pages) {
                d_valid |= 1 << (half * (NB / 2) + j);
                d_src[half * (NB / 2) + j] =
                    static_cast<const uint8_t*>(a.cache.pool) +
                    kv4_block_offset(page, h, Hk, P / kKvBlock, (tok & (P - 1)) / kKvBlock, L::kBytes);
              } else if (a.device_status != nullptr) {
                *a.device_status = MOE_ERR_DEVICE;
              }
            }
          }
        };
        auto issue = [&](int tile, int slot) {
          const int valid = __shfl_sync(kFull, d_valid, tile - base);
          const uint32_t dst = smem_u32(ring) + slot * Sh::kStageBytes + lane * 16;
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const uint8_t* f = reinterpret_cast<const uint8_t*>(
                                   __shfl_sync(kFull, reinterpret_cast<unsigned long long>(d_src[i]), tile - base)) + lane * 16;
            if (!(valid >> i & 1)) continue;
#pragma unroll
            for (int c = 0; c < L::kBytes; c += 512)
              if (c + 512 <= L::kBytes || lane * 16 < L::kBytes - c) cp_async_16(dst + i * L::kBytes + c, f + c, 16);
          }
        };

        describe(r0, true);
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < S; ++i) {
          if (r0 + i < r1) issue(r0 + i, i);
          cp_async_commit();
        }
        start_rows<D, NT>(st, g8, t4, a.scale, a.cache.k_gs, [&](int row) {
          return row < used ? a.q + (size_t)(t + row / heads) * a.q_stride + (h * heads + row % heads) * D : nullptr;
        });
        int next = r0 + min(S, r1 - r0), slot = 0;
        for (int tile = r0; tile < r1; ++tile) {
          const int src = tile - base;
          const int tok0 = __shfl_sync(kFull, d_tok[0], src), tok1 = __shfl_sync(kFull, d_tok[1], src);
          const int who = __shfl_sync(kFull, d_rows, src), valid = __shfl_sync(kFull, d_valid, src);
          cp_async_wait<S - 1>();
          __syncwarp();
          const uint8_t* stage = ring + slot * Sh::kStageBytes;
          const bool masked = who != (int)(full | full << 8) || valid != (1 << NB) - 1 ||
                              max(tok0, tok1) + NB / 2 * kKvBlock - 1 > pos0;
          auto work = [&](auto with_mask, int blk0) {
            constexpr bool kMask = decltype(with_mask)::value;
            const int recip = kMask ? (65535 + heads) / heads : 0;
            attend_blocks<D, NT, kPart, kMask>(st, g8, t4, stage + blk0 * L::kBytes, [&](int b, int nt, int i) {
              const int blk = blk0 + b, half = blk / (NB / 2);
              const int tok = (half ? tok1 : tok0) + blk % (NB / 2) * kKvBlock + token_of(g8) + 8 * (i >> 1);
              const int row = (nt * 8 + 2 * t4 + (i & 1)) * recip >> 16;   // row / heads (both at most 16)
              return tok > pos0 + row || !(who >> (8 * half) >> row & 1) || !(valid >> blk & 1);
            });
          };
#pragma unroll 1
          for (int blk = 0; blk < NB; blk += kPart) {
            if (masked) work(std::true_type{}, blk);
            else work(std::false_type{}, blk);
          }
          __syncwarp();   // every lane has read the stage
          if (next < r1) {
            if (next - base >= 32) describe(tile + 1, false);
            __syncwarp();
            issue(next, slot);
            ++next;
          }
          cp_async_commit();
          slot = slot + 1 == S ? 0 : slot + 1;
        }
      }

      // ------------------------------------------------------ the results
      if (active <= 1) {
        if (me == 0) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float sum = tiles ? st.l[nt][c] : 0.0f;
              sum += __shfl_xor_sync(kFull, sum, 4);
              sum += __shfl_xor_sync(kFull, sum, 8);
              sum += __shfl_xor_sync(kFull, sum, 16);
              const int row = nt * 8 + 2 * t4 + c;
              if (row >= used) continue;
              const float inv = sum == 0.0f ? 0.0f : 1.0f / (sum * a.cache.v_gs);   // NaN stays NaN
              uint32_t w[MT];
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                w[mt] = tiles ? float2_to_bf16x2_bits(st.o[nt][mt][c] * inv, st.o[nt][mt][c + 2] * inv) : 0u;
              uint4* out = reinterpret_cast<uint4*>(a.out + out_row(row) * D + g8 * (D / 8));
#pragma unroll
              for (int i = 0; i < MT / 4; ++i) out[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
              if (g8 == 0 && a.lse != nullptr)
                a.lse[out_row(row)] = sum == 0.0f ? -INFINITY : st.m[nt][c] * kLn2 + logf(sum);
            }
        }
        __syncwarp();
        continue;
      }
      // a warp's partial in its first stages
      if (me < active) {
        float* const dst = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float sum = st.l[nt][c];
            sum += __shfl_xor_sync(kFull, sum, 4);
            sum += __shfl_xor_sync(kFull, sum, 8);
            sum += __shfl_xor_sync(kFull, sum, 16);
            const int row = nt * 8 + 2 * t4 + c;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              *reinterpret_cast<float2*>(dst + row * D + warp_chunk(row, g8 * (D / 32) + mt / 2) * 4 + mt % 2 * 2) =
                  make_float2(st.o[nt][mt][c], st.o[nt][mt][c + 2]);
            if (g8 == 0) *reinterpret_cast<float2*>(dst + kRows * D + 2 * row) = make_float2(st.m[nt][c], sum);
          }
      }
      auto put_out = [&](int row, int d, const Joined& x) {
        const float inv = x.l == 0.0f ? 0.0f : 1.0f / (x.l * a.cache.v_gs);
        const size_t at = out_row(row);
        *reinterpret_cast<uint2*>(a.out + at * D + d) =
            make_uint2(float2_to_bf16x2_bits(x.o.x * inv, x.o.y * inv), float2_to_bf16x2_bits(x.o.z * inv, x.o.w * inv));
        if (d == 0 && a.lse != nullptr) a.lse[at] = x.l == 0.0f ? -INFINITY : x.m * kLn2 + logf(x.l);
      };
      const int here = min(p.split, max(0, active - rank * p.split));   // partials of this CTA
      auto mine_of = [&](int i) { return reinterpret_cast<const float*>(&sm->ring[group * p.split + i][0][0]); };
      group_sync(group, p.split);
      if (p.cluster == 1) {
        join<D, NT>(here, used, me * 32 + lane, p.split * 32, true, mine_of, put_out);
        group_sync(group, p.split);   // read before the ring is filled again
        continue;
      }
      namespace cg = cooperative_groups;
      cg::cluster_group cluster = cg::this_cluster();
      float* const joined = reinterpret_cast<float*>(&sm->ring[0][0][0]) + Slots<D, NT>::kFloats;
      join<D, NT>(here, used, warp * 32 + lane, Sh::kThreads, true, mine_of, [&](int row, int d, const Joined& x) {
        *reinterpret_cast<float4*>(joined + row * D + d) = x.o;
        if (d == 0) *reinterpret_cast<float2*>(joined + kRows * D + 2 * row) = make_float2(x.m, x.l);
      });
      cluster.sync();
      join<D, NT>((active + p.split - 1) / p.split, used, me * 32 + lane, members * 32, false,
                  [&](int i) { return cluster.map_shared_rank(joined, i); }, put_out);
      cluster.sync();
    }
  }
}

template <int D, int NT>
cudaError_t launch(SparseArgs& p, bool by_request, cudaStream_t s) {
  using Sh = Shape<D, NT>;
  auto k = kv4_sparse_kernel<D, NT>;
  constexpr size_t smem = sizeof(Smem<D, NT>);
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = opt_in_smem(k, smem, done);
  if (e != cudaSuccess) return e;
  const int heads = p.a.q_heads / p.a.cache.kv_heads, sms = sm_count();
  // Rows of one unit: neighbours only where a request can have any.
  p.tile = p.a.max_q == 1 ? 1 : 8 * NT / heads;
  if (p.tile > 8) p.tile = 8;                                   // a row has a bit of a byte
  if (p.tile > kListMax / p.a.top) p.tile = kListMax / p.a.top;
  p.per = by_request ? (kSparseFewTokens + p.tile - 1) / p.tile : 0;
  const long long units =
      (by_request ? (long long)p.a.batch * p.per : ((long long)p.a.total_q + p.tile - 1) / p.tile) * p.a.cache.kv_heads;
  p.units = (int)units;
  // Enough warps a unit to fill the GPU once, as long as each has a tile.
  const int tiles = (p.tile * p.a.top * (p.a.block_tokens / kKvBlock) + Sh::kBlocks - 1) / Sh::kBlocks;
  auto wanted = [&](int n) { return units * n <= (long long)sms * Sh::kWarps && n <= tiles; };
  p.split = 1;
  while (p.split < Sh::kWarps && wanted(p.split * 2)) p.split *= 2;
  if (Sh::kWarps % p.split || (p.split * 2 > Sh::kWarps && wanted(Sh::kWarps))) p.split = Sh::kWarps;
  p.cluster = 1;
  if (p.split == Sh::kWarps)
    while (p.cluster < 8 && wanted(p.cluster * 2 * Sh::kWarps)) p.cluster *= 2;
  const int groups = Sh::kWarps / p.split;
  const long long ctas = (units + groups - 1) / groups, most = sms / p.cluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((ctas < most ? ctas : most) * p.cluster));
  cfg.blockDim = dim3(Sh::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)p.cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}

}  // namespace

moe_status launch_kv4_sparse(const moe_kv4_sparse_args& a, cudaStream_t s) {
  SparseArgs p;
  p.a = a;
  p.block_log = __builtin_ctz(a.block_tokens);
  const bool wide = a.q_heads / a.cache.kv_heads > 8;
  // Which kernel. Requests of up to kSparseFewTokens rows are this one's (16
  // requests of 24 new tokens over 16 blocks of 64, 32/8 heads x 128: 98 us here,
  // 114 there; of 32: 99 and 81), and all are where the other one would not
  // have a unit for most of the SMs (one of 64: 20 and 59 us; 16 of 64 190 and
  // 94) or a group has one head (its 32 tokens fill a quarter of the tile's rows:
  // 16 of 32 57 and 76). Lengths are on the device: a call that allows longer
  // requests launches both kernels, each skipping the other's.
  const int group = a.q_heads / a.cache.kv_heads;
  const bool many = a.max_q > kSparseFewTokens && group > 1 &&
                    (long long)a.total_q * a.cache.kv_heads >= kSparseManyUnits * (long long)(group < 4 ? 32 : 128 / group);
  cudaError_t e;
  if (a.cache.head_dim == 64) e = wide ? launch<64, 2>(p, many, s) : launch<64, 1>(p, many, s);
  else e = wide ? launch<128, 2>(p, many, s) : launch<128, 1>(p, many, s);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return many ? launch_kv4_sparse_prompt(a, kSparseFewTokens, s) : MOE_OK;
}

}  // namespace moe
