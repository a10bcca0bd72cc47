// Mean keys of complete blocks of cached tokens, on a grid of whole numbers.
//
// Mathematics. code * scale of a key element is a whole number of 2^-10 below
// 2^22 (e2m1 is one of 1/2, E4M3 one of 2^-9), so the sum over up to 128 tokens
// is one of 32 bits and exact in any order. The mean n 2^s has n of 8 bits: the
// sum is rounded, nearest even, to 2^(E - 6) with E the exponent of the row's
// largest.
//
// What bounds it: a decode step completes few blocks, so latency (64 requests:
// 3.3 us); prompts read the key half of their cache, 0.5625 bytes an element (4
// of up to 8191 tokens in pages of 16, 8 heads x 128: 7.8 us, 1.6 by the bytes):
// a CTA's lengths, page ids and rows are three trips to memory one after the
// other, then comes the conversion of the rows; at 138 registers three CTAs fit
// an SM, so that case's 544 with work are two waves, among 384 more that the
// bound on lengths launches and that leave at once.
//
// A warp has one block of one head: a lane holds the sums of 32 elements over
// every 8th (head_dim 64: 16th) token.
#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4, kAtOnce = 4;   // 16-token blocks asked for together
constexpr unsigned kFull = 0xffffffffu;

struct IndexArgs {
  moe_kv4_index x;
  int max_q, max_pages;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* table;
  int* status;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv4_index_kernel(const __grid_constant__ IndexArgs p) {
  using L = Kv4Block<D>;
  constexpr int kLanes = D / 32;             // lanes of a token's row, 32 elements each
  constexpr int kRows = 32 / kLanes;         // tokens of a round
  constexpr int kRounds = kKvBlock / kRows;  // rounds of a 16-token block
  const moe_kv4_cache& c = p.x.cache;
  pdl_wait();
  const int lane = threadIdx.x & 31, h = blockIdx.z * kWarps + (threadIdx.x >> 5), b = blockIdx.y;
  const int c0 = __ldg(p.cu_q + b), n = __ldg(p.cu_q + b + 1) - c0, kv = __ldg(p.kv_len + b);
  const int B = p.x.block_tokens, P = c.page_tokens;
  if (c0 < 0 || n < 0 || n > p.max_q || kv < n || kv > p.max_pages * P) {
    if (threadIdx.x == 0 && p.status != nullptr) *p.status = MOE_ERR_DEVICE;
    return;
  }
  const int blk = (kv - n) / B + blockIdx.x;
  if (blk >= kv / B || h >= c.kv_heads) return;
  const int32_t* const table = p.table + (size_t)b * p.max_pages;
  const int tok0 = blk * B, row0 = lane / kLanes, part = lane % kLanes;

  // Page ids first, all at once, then the rows of kAtOnce 16-token blocks.
  const int subs = B / kKvBlock;
  const int my_page = lane < subs ? __ldg(table + (tok0 + lane * kKvBlock) / P) : 0;
  if (__any_sync(kFull, my_page < 0 || my_page >= c.num_pages)) {
    if (lane == 0 && p.status != nullptr) *p.status = MOE_ERR_DEVICE;
    return;
  }
  // Whose rows: the first page's, or, where another block has those, the last one's. All heads get the same answer.
  int row_page = __shfl_sync(kFull, my_page, 0);
  if (B > P) {
    const int end = __shfl_sync(kFull, my_page, subs - 1);
    int owner = -1;
    if (lane == 0) owner = atomicCAS(p.x.owners + row_page, -1, end);
    owner = __shfl_sync(kFull, owner, 0);
    if (owner >= 0 && owner != end) row_page = end;
  }
  int sum[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) sum[i] = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < subs; s0 += kAtOnce) {
    uint4 codes[kAtOnce][kRounds];
    uint32_t two[kAtOnce][kRounds];
#pragma unroll
    for (int s = 0; s < kAtOnce; ++s) {
      const int tok = tok0 + (s0 + s) * kKvBlock, page = __shfl_sync(kFull, my_page, s0 + s);
      const uint8_t* const src = static_cast<const uint8_t*>(c.pool) +
                                 kv4_block_offset(page, h, c.kv_heads, P / kKvBlock, tok % P / kKvBlock, L::kBytes);
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int row = r * kRows + row0;
        codes[s][r] = make_uint4(0u, 0u, 0u, 0u);
        two[s][r] = 0u;
        if (s0 + s < subs) {
          codes[s][r] = __ldg(reinterpret_cast<const uint4*>(src + row * L::kCodeRow) + part);
          two[s][r] = __ldg(reinterpret_cast<const uint16_t*>(src + L::kKeyScales + row * L::kScaleRow) + part);
        }
      }
    }
#pragma unroll
    for (int pair = 0; pair < kAtOnce; pair += 2) {
      float part_sum[32];   // of at most four tokens, below 2^14: exact
#pragma unroll
      for (int i = 0; i < 32; ++i) part_sum[i] = 0.0f;
#pragma unroll
      for (int s = pair; s < pair + 2; ++s)
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
          const uint32_t sc = cvt_e4m3x2_f16x2(two[s][r]);
          const uint32_t w[4] = {codes[s][r].x, codes[s][r].y, codes[s][r].z, codes[s][r].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t v[4];
            cvt_e2m1x8_f16(w[i], v);
            const uint32_t s2 = __byte_perm(sc, 0, i < 2 ? 0x1010 : 0x3232);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t prod = hmul2_u32(v[j], s2);   // exact
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&prod));
              part_sum[8 * i + 2 * j] += f.x;
              part_sum[8 * i + 2 * j + 1] += f.y;
            }
          }
        }
#pragma unroll
      for (int i = 0; i < 32; ++i) sum[i] += __float2int_rn(part_sum[i] * 1024.0f);
    }
  }
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1) sum[i] += __shfl_xor_sync(kFull, sum[i], o);
    top = max(top, (unsigned)abs(sum[i]));
  }
  top = __reduce_max_sync(kFull, top);
  const int shift = max(0, 31 - __clz((int)max(top, 1u)) - 6);   // step 2^shift; what has 7 bits or fewer stays as it is
  // nearest even multiple of 2^shift, as f16: at most 8 significant bits, from 2^-17 up
  const float unit = __int_as_float((127 + shift - 10 - (31 - __clz(B))) << 23);
  if (row0 == 0) {
    uint32_t out[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int x = sum[2 * i + j];
        const int r = shift == 0 ? x : (x + (1 << (shift - 1)) - 1 + (x >> shift & 1)) >> shift;
        v[j] = (float)r * unit;
      }
      const __half2 o = __floats2half2_rn(v[0], v[1]);
      out[i] = *reinterpret_cast<const uint32_t*>(&o);
    }
    const int per = P > B ? P / B : 1;
    const size_t entry = (size_t)row_page * per + tok0 % P / B;
    uint4* const dst = reinterpret_cast<uint4*>(p.x.means + (entry * c.kv_heads + h) * D + part * 32);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
  }
}

}  // namespace

moe_status launch_kv4_index_update(const moe_kv4_index& x, int batch, int max_q, int max_pages, const int32_t* cu_q,
                                   const int32_t* kv_len, const int32_t* table, int32_t* status, cudaStream_t s) {
  IndexArgs p = {x, max_q, max_pages, cu_q, kv_len, table, status};
  // n tokens make at most ceil(n / B) blocks complete
  const long long most = (long long)max_pages * x.cache.page_tokens, q = max_q < most ? max_q : most;
  const unsigned blocks = (unsigned)((q + x.block_tokens - 1) / x.block_tokens);
  if (blocks == 0) return MOE_OK;
  const dim3 grid(blocks, batch, (x.cache.kv_heads + kWarps - 1) / kWarps);
  const cudaError_t e = launch_ex(true, x.cache.head_dim == 64 ? kv4_index_kernel<64> : kv4_index_kernel<128>, grid,
                                  dim3(kWarps * 32), 0, s, p);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

}  // namespace moe
