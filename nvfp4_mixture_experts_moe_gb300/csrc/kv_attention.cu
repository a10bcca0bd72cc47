// Attention over the NVFP4 cache: one warp per (query row, query head).
#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv4_attention_simple_kernel(moe_kv4_attn_args a, int min_rows, int* status) {
  using L = Kv4Block<D>;
  __shared__ float qs[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long item = (long long)blockIdx.x * kWarps + warp;
  if (item >= (long long)a.total_q * a.q_heads) return;
  const int row = (int)(item / a.q_heads), h = (int)(item % a.q_heads);
  const int group = a.q_heads / a.cache.kv_heads, kh = h / group;
  int lo = 0, hi = a.batch;  // the request of this row
  if (row < a.cu_q[0] || row >= a.cu_q[a.batch]) return;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu_q[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  const int b = lo, n = a.cu_q[b + 1] - a.cu_q[b], i = row - a.cu_q[b];
  if (n * group <= min_rows) return;
  if (n > a.max_q || a.cu_q[b + 1] > a.total_q) {
    if (lane == 0) set_status(status, MOE_ERR_DEVICE);
    return;
  }
  const int P = a.cache.page_tokens;
  int kv = a.kv_len[b];
  if (kv > a.max_pages * P || kv < 0) {
    if (lane == 0) set_status(status, MOE_ERR_DEVICE);
    kv = max(0, min(kv, a.max_pages * P));
  }
  const int pos = a.causal ? kv - n + i : kv - 1;
  const int end = pos + 1, begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  for (int d = lane; d < D; d += 32) qs[warp][d] = bf16_bits_to_float(a.q[row * a.q_stride + h * D + d]);
  __syncwarp();
  const float sc = a.scale / a.cache.k_gs;
  float m = -INFINITY, l = 0.0f, acc[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) acc[d] = 0.0f;
  for (int t0 = begin; t0 < end; t0 += 32) {
    const int t = t0 + lane;
    float s = -INFINITY;
    const uint8_t* blk = nullptr;
    if (t < end) {
      const int page = a.block_table[(size_t)b * a.max_pages + t / P], pos_in = t % P;
      if (page >= 0 && page < a.cache.num_pages) {
        blk = static_cast<const uint8_t*>(a.cache.pool) +
              kv4_block_offset(page, kh, a.cache.kv_heads, P / kKvBlock, pos_in / kKvBlock, L::kBytes);
        const uint8_t* codes = blk + (t % kKvBlock) * L::kCodeRow;
        const uint8_t* sf = blk + L::kKeyScales + (t % kKvBlock) * L::kScaleRow;
        s = 0.0f;
        for (int g = 0; g < D / 16; ++g) {
          const float f = e4m3_decode(sf[g]);
          for (int j = 0; j < 8; ++j) {
            const uint32_t v = cvt_e2m1x2_f16x2(codes[g * 8 + j]);
            const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&v));
            s += f * (e.x * qs[warp][g * 16 + 2 * j] + e.y * qs[warp][g * 16 + 2 * j + 1]);
          }
        }
        s *= sc;
      } else {
        set_status(status, MOE_ERR_DEVICE);
      }
    }
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY) continue;
    const float corr = __expf(m - mn), p = __expf(s - mn);
    l = l * corr + p;
    m = mn;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) acc[d] *= corr;
    for (int j = 0; j < 32; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j);
      const uint8_t* bj = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(blk), j));
      if (bj == nullptr || t0 + j >= end) continue;
      const int tj = (t0 + j) % kKvBlock;
#pragma unroll
      for (int d = 0; d < D / 64; ++d) {
        const int c = d * 64 + 2 * lane;
        const uint32_t v = cvt_e2m1x2_f16x2(bj[L::kValueCodes + tj * L::kCodeRow + c / 2]);
        const float f = e4m3_decode(bj[L::kValueScales + tj * L::kScaleRow + c / 16]) * pj;
        const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&v));
        acc[2 * d] += f * e.x;
        acc[2 * d + 1] += f * e.y;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.0f ? 1.0f / (l * a.cache.v_gs) : 0.0f;
  uint16_t* out = a.out + ((size_t)row * a.q_heads + h) * D;
#pragma unroll
  for (int d = 0; d < D / 64; ++d)
    *reinterpret_cast<uint32_t*>(out + d * 64 + 2 * lane) = float2_to_bf16x2_bits(acc[2 * d] * inv, acc[2 * d + 1] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[(size_t)row * a.q_heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

// A request's query rows per key/value head (its tokens times the group's
// query heads) decide its kernel; max_q bounds them, so calls of single or
// few drafted tokens launch only the decode kernel.
size_t kv4_attention_ws_bytes(const moe_kv4_attn_args& a) {
  const long long rows = (long long)a.max_q * (a.q_heads / a.cache.kv_heads);
  const int decode_rows = rows < kKvDecodeRows ? (int)rows : kKvDecodeRows;
  return align_up(MOE_KV4_WS_ZERO + kv4_decode_ws_floats(a.cache.head_dim, decode_rows) * sizeof(float));
}

moe_status launch_kv4_attention(const moe_kv4_attn_args& a, void* ws, cudaStream_t s) {
  int* status = &static_cast<WsHeader*>(ws)->status;
  int* counters = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + sizeof(WsHeader));
  static_assert(sizeof(WsHeader) + kKvMaxCtas * sizeof(int) <= MOE_KV4_WS_ZERO, "zero region");
  float* partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + MOE_KV4_WS_ZERO);
  const long long rows = (long long)a.max_q * (a.q_heads / a.cache.kv_heads);
  moe_status st = launch_kv4_decode(a, rows < kKvDecodeRows ? (int)rows : kKvDecodeRows, status, counters, partials, s);
  if (st != MOE_OK || rows <= kKvDecodeRows) return st;
  const long long ctas = ((long long)a.total_q * a.q_heads + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
  auto k = a.cache.head_dim == 64 ? kv4_attention_simple_kernel<64> : kv4_attention_simple_kernel<128>;
  cudaError_t e = launch_ex(false, k, dim3((unsigned)ctas), dim3(kWarps * 32), 0, s, a, kKvDecodeRows, status);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

}  // namespace moe
