// C ABI entry points of the block operators (include/moe_block.h): argument
// validation on the host, then the launchers.
#include <climits>
#include <cmath>

#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Sizes of a cache; what is legal but not built is UNSUPPORTED.
moe_status check_cache_sizes(int num_pages, int page_tokens, int kv_heads, int head_dim) {
  if (num_pages < 1 || page_tokens < 1 || kv_heads < 1 || head_dim < 1) return MOE_ERR_INVALID_ARG;
  if (page_tokens != 16 && page_tokens != 32 && page_tokens != 64 && page_tokens != 128) return MOE_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return MOE_ERR_UNSUPPORTED;
  if (kv_heads > 1024 || (long long)num_pages * page_tokens > INT_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_cache(const moe_kv4_cache& c) {
  const moe_status st = check_cache_sizes(c.num_pages, c.page_tokens, c.kv_heads, c.head_dim);
  if (st != MOE_OK) return st;
  if (c.pool == nullptr || !aligned(c.pool, 16)) return MOE_ERR_INVALID_ARG;
  if (!(c.k_gs > 0.0f) || !std::isfinite(c.k_gs) || !(c.v_gs > 0.0f) || !std::isfinite(c.v_gs))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Everything about an attention call that needs no device and no workspace.
moe_status check_attention(const moe_kv4_attn_args* a) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  const moe_status st =
      check_cache_sizes(a->cache.num_pages, a->cache.page_tokens, a->cache.kv_heads, a->cache.head_dim);
  if (st != MOE_OK) return st;
  if (a->batch < 0 || a->q_heads < 1 || a->total_q < 0 || a->max_q < 0 || a->max_pages < 0 || a->window < 0)
    return MOE_ERR_INVALID_ARG;
  if (a->window > 0 && !a->causal) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale)) return MOE_ERR_INVALID_ARG;
  if (a->q_heads % a->cache.kv_heads || a->batch > 4096 || a->q_heads > 65536) return MOE_ERR_UNSUPPORTED;
  const long long row_tokens = (long long)a->max_pages * a->cache.page_tokens;
  if (row_tokens > INT_MAX - 128) return MOE_ERR_UNSUPPORTED;   // lengths are rounded up to tiles in 32 bits
  const long long tiles = (row_tokens + 31) / 32;
  if (a->batch > 0 && tiles > INT_MAX / ((long long)a->batch * a->cache.kv_heads)) return MOE_ERR_UNSUPPORTED;
  if ((long long)a->total_q * (a->q_heads / a->cache.kv_heads) > INT_MAX) return MOE_ERR_UNSUPPORTED;
  if (kv4_prompt_units(*a) > INT_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Whether one of a step's outputs shares memory with an input or another
// output: CTA 0 writes some of them while other CTAs still read lengths, and
// the stack and the table are read and written without an order.
bool step_arrays_overlap(const moe_kv_step_args& a) {
  struct Array {
    const int32_t* at;
    long long n;
  };
  const Array arrays[] = {
      {a.kv_len, a.batch}, {a.cu_q, a.batch + 1ll}, {a.slots, a.tokens}, {a.positions, a.tokens},
      {a.free_count_out, 1}, {a.block_table, (long long)a.batch * a.max_pages}, {a.device_status, a.device_status ? 1 : 0},
      // inputs
      {a.ctx_len, a.batch}, {a.new_len, a.batch}, {a.free_pages, a.free_capacity}, {a.free_count, 1}};
  constexpr int kOutputs = 7, kArrays = sizeof(arrays) / sizeof(arrays[0]);
  for (int i = 0; i < kOutputs; ++i)
    for (int j = i + 1; j < kArrays; ++j) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(arrays[i].at), y = reinterpret_cast<uintptr_t>(arrays[j].at);
      if (arrays[i].n > 0 && arrays[j].n > 0 && x < y + 4 * arrays[j].n && y < x + 4 * arrays[i].n) return true;
    }
  return false;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_kv4_pool_size(int num_pages, int page_tokens, int kv_heads, int head_dim) {
  if (check_cache_sizes(num_pages, page_tokens, kv_heads, head_dim) != MOE_OK) return 0;
  return (size_t)num_pages * page_tokens * kv_heads * (size_t)(18 * head_dim / kKvBlock);
}

moe_status moe_kv4_append(const moe_kv4_cache* cache, const uint16_t* k, const uint16_t* v, long long k_stride,
                          long long v_stride, const int32_t* slots, int tokens, int32_t* device_status,
                          moe_stream_t stream) {
  if (cache == nullptr || tokens < 0) return MOE_ERR_INVALID_ARG;
  moe_status st = check_cache(*cache);
  if (st != MOE_OK) return st;
  if (tokens == 0) return MOE_OK;
  const long long row = (long long)cache->kv_heads * cache->head_dim;
  if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16)) return MOE_ERR_INVALID_ARG;
  if (k_stride % 8 || v_stride % 8 || k_stride < row || v_stride < row) return MOE_ERR_INVALID_ARG;
  st = check_device();
  if (st != MOE_OK) return st;
  return launch_kv4_append(*cache, k, v, k_stride, v_stride, slots, tokens, device_status, (cudaStream_t)stream);
}

moe_status moe_kv4_read(const moe_kv4_cache* cache, const int32_t* slots, int n, uint16_t* k_out, uint16_t* v_out,
                        int32_t* device_status, moe_stream_t stream) {
  if (cache == nullptr || n < 0) return MOE_ERR_INVALID_ARG;
  moe_status st = check_cache(*cache);
  if (st != MOE_OK) return st;
  if (n == 0) return MOE_OK;
  if (!slots || (!k_out && !v_out) || !aligned(k_out, 16) || !aligned(v_out, 16)) return MOE_ERR_INVALID_ARG;
  st = check_device();
  if (st != MOE_OK) return st;
  return launch_kv4_read(*cache, slots, n, k_out, v_out, device_status, (cudaStream_t)stream);
}

size_t moe_kv4_attention_workspace_size(const moe_kv4_attn_args* args) {
  return check_attention(args) == MOE_OK ? kv4_attention_ws_bytes(*args) : 0;
}

moe_status moe_kv4_attention(const moe_kv4_attn_args* args, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status st = check_attention(args);
  if (st != MOE_OK) return st;
  st = check_cache(args->cache);
  if (st != MOE_OK) return st;
  if (args->batch == 0 || args->total_q == 0) return MOE_OK;
  const long long row = (long long)args->q_heads * args->cache.head_dim;
  if (args->max_q < 1) return MOE_ERR_INVALID_ARG;
  if (!args->q || !args->cu_q || !args->kv_len || !args->out) return MOE_ERR_INVALID_ARG;
  if (!args->block_table && args->max_pages > 0) return MOE_ERR_INVALID_ARG;
  if (!aligned(args->q, 16) || !aligned(args->out, 16) || args->q_stride % 8 || args->q_stride < row)
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign) || ws_bytes < kv4_attention_ws_bytes(*args)) return MOE_ERR_WORKSPACE;
  st = check_device();
  if (st != MOE_OK) return st;
  return launch_kv4_attention(*args, ws, (cudaStream_t)stream);
}

moe_status moe_kv_step(const moe_kv_step_args* a, moe_stream_t stream) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  if (a->batch < 0 || a->tokens < 0 || a->free_capacity < 0 || a->page_tokens < 1 || a->max_pages < 1)
    return MOE_ERR_INVALID_ARG;
  if (a->batch > 4096) return MOE_ERR_UNSUPPORTED;
  if ((long long)a->page_tokens * a->max_pages > INT_MAX) return MOE_ERR_INVALID_ARG;
  if (!a->free_count || !a->free_count_out || !a->cu_q) return MOE_ERR_INVALID_ARG;
  if (a->batch > 0 && (!a->ctx_len || !a->new_len || !a->block_table || !a->kv_len)) return MOE_ERR_INVALID_ARG;
  if (a->free_capacity > 0 && !a->free_pages) return MOE_ERR_INVALID_ARG;
  if (a->tokens > 0 && (!a->slots || !a->positions)) return MOE_ERR_INVALID_ARG;
  if (step_arrays_overlap(*a)) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_device();
  if (st != MOE_OK) return st;
  return launch_kv_step(*a, (cudaStream_t)stream);
}

moe_status moe_block_norm(const moe_block_norm_args* a, moe_stream_t stream) {
  if (a == nullptr || a->T < 0 || a->H < 1) return MOE_ERR_INVALID_ARG;
  if (a->H > 16384) return MOE_ERR_UNSUPPORTED;
  if (!std::isfinite(a->residual_scale) || !std::isfinite(a->branch_scale) || !std::isfinite(a->w_offset) ||
      !std::isfinite(a->eps) || a->eps < 0.0f)
    return MOE_ERR_INVALID_ARG;
  if (a->T == 0) return MOE_OK;
  if (!a->residual || (!a->residual_out && !a->w_pre) || (a->w_pre && !a->out)) return MOE_ERR_INVALID_ARG;
  if (a->residual_stride < a->H || (a->x && a->x_stride < a->H)) return MOE_ERR_INVALID_ARG;
  if (a->gate && a->gate_stride != 0 && a->gate_stride < a->H) return MOE_ERR_INVALID_ARG;
  const size_t re = a->residual_f32 ? 4 : 2;
  if (!aligned(a->x, 2) || !aligned(a->gate, 2) || !aligned(a->w_post, 2) || !aligned(a->w_pre, 2) ||
      !aligned(a->out, 2) || !aligned(a->residual, re) || !aligned(a->residual_out, re))
    return MOE_ERR_INVALID_ARG;
  if (a->residual_out == a->residual && a->residual_stride != a->H) return MOE_ERR_INVALID_ARG;
  const moe_status st = check_device();
  if (st != MOE_OK) return st;
  return launch_block_norm(*a, (cudaStream_t)stream);
}

}  // extern "C"
