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

// Elements of rows [0, n) x [0, width) at `at`, `stride` apart.
struct Rows {
  const uint16_t* at;
  long long stride, width;
};

// Whether two sets of n rows share an element. Rows of one stride may lie next
// to one another (columns of one buffer).
bool rows_overlap(const Rows& x, const Rows& y, long long n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.at), b = reinterpret_cast<uintptr_t>(y.at);
  const uintptr_t a1 = a + 2 * ((n - 1) * x.stride + x.width), b1 = b + 2 * ((n - 1) * y.stride + y.width);
  if (a >= b1 || b >= a1) return false;
  if (x.stride != y.stride) return true;
  const uintptr_t step = 2 * x.stride;
  if (a <= b) {   // y's rows start `off` bytes into x's
    const uintptr_t off = (b - a) % step;
    return off < 2 * (uintptr_t)x.width || off + 2 * y.width > step;
  }
  const uintptr_t off = (a - b) % step;
  return off < 2 * (uintptr_t)y.width || off + 2 * x.width > step;
}

moe_status check_plan(const moe_rope_plan& r, int head_dim) {
  if (r.rotary_dim < 2 || r.rotary_dim % 2 || r.rotary_dim > head_dim || r.axes < 1 || r.axes > MOE_ROPE_MAX_AXES ||
      !std::isfinite(r.scale) || !r.turns || !aligned(r.turns, 8))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_index_sizes(const moe_kv4_cache& c, int block_tokens) {
  const moe_status st = check_cache_sizes(c.num_pages, c.page_tokens, c.kv_heads, c.head_dim);
  if (st != MOE_OK) return st;
  return block_tokens == 32 || block_tokens == 64 || block_tokens == 128 ? MOE_OK
         : block_tokens < 1                                              ? MOE_ERR_INVALID_ARG
                                                                         : MOE_ERR_UNSUPPORTED;
}

moe_status check_index(const moe_kv4_index& x) {
  moe_status st = check_index_sizes(x.cache, x.block_tokens);
  if (st == MOE_OK) st = check_cache(x.cache);
  if (st != MOE_OK) return st;
  if (!x.means || !aligned(x.means, 16)) return MOE_ERR_INVALID_ARG;
  // which blocks have the rows of their first pages: needed where blocks have several
  return x.block_tokens <= x.cache.page_tokens || (x.owners && aligned(x.owners, 4)) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// The sizes of a selection and of an attention over what it selected.
moe_status check_sparse_sizes(const moe_kv4_cache& c, int batch, int q_heads, int total_q, int max_q, int max_pages, int top) {
  if (batch < 0 || q_heads < 1 || total_q < 0 || max_q < 0 || max_pages < 0 || top < 1) return MOE_ERR_INVALID_ARG;
  if (q_heads % c.kv_heads || q_heads / c.kv_heads > kSparseGroup || top > kSparseTop || batch > 4096)
    return MOE_ERR_UNSUPPORTED;
  if ((long long)max_pages * c.page_tokens > 1 << 28) return MOE_ERR_UNSUPPORTED;
  if ((long long)total_q * c.kv_heads > 1 << 30) return MOE_ERR_UNSUPPORTED;   // units are counted in 32 bits
  return MOE_OK;
}

moe_status check_sparse_pointers(const moe_kv4_cache& c, int q_heads, int max_q, int max_pages, const void* q, long long q_stride,
                                 const void* cu_q, const void* kv_len, const void* block_table, const void* blocks) {
  if (max_q < 1 || !q || !cu_q || !kv_len || !blocks || (!block_table && max_pages > 0)) return MOE_ERR_INVALID_ARG;
  if (!aligned(q, 16) || q_stride % 8 || q_stride < (long long)q_heads * c.head_dim) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
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

moe_status moe_rope_turns(const double* inv_freq, const int32_t* axis, int n, uint64_t* turns) {
  if (n < 0 || (n > 0 && (!inv_freq || !turns))) return MOE_ERR_INVALID_ARG;
  // 1 / (2 pi) as a fraction of 192 bits, most significant first
  static const uint64_t kInverse[3] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull};
  for (int i = 0; i < n; ++i) {
    const double f = inv_freq[i];
    if (!std::isfinite(f) || std::fabs(f) > 1024.0 || (axis && (axis[i] < 0 || axis[i] >= MOE_ROPE_MAX_AXES)))
      return MOE_ERR_INVALID_ARG;
    // |f| = m 2^e with m a whole number of 53 bits; m / (2 pi) as 53 + 192 bits
    int e = 0;
    uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(f), &e), 53);
    e -= 53;
    uint64_t w[4] = {0, 0, 0, 0};   // w[3] whole numbers, then 192 bits of fraction downwards
    unsigned __int128 carry = 0;
    for (int k = 2; k >= 0; --k) {
      carry += (unsigned __int128)m * kInverse[k];
      w[2 - k] = (uint64_t)carry;
      carry >>= 64;
    }
    w[3] = (uint64_t)carry;
    // times 2^e, modulo 1, to 64 bits (e <= -42)
    const int shift = -e;
    uint64_t t = shift < 128 ? (uint64_t)(((unsigned __int128)w[3] << 64 | w[2]) >> shift) : 0;
    if (f < 0) t = 0 - t;
    // the lowest two bits are the axis: the nearest multiple of four
    turns[i] = ((t + 2) & ~3ull) | (axis ? (uint64_t)axis[i] : 0);
  }
  return MOE_OK;
}

moe_status moe_rope(const moe_rope_args* a, moe_stream_t stream) {
  if (a == nullptr || a->tokens < 0 || a->head_dim < 1 || a->q_heads < 1 || a->k_heads < 0) return MOE_ERR_INVALID_ARG;
  if (a->head_dim > 512 || (long long)a->q_heads + a->k_heads > 65536) return MOE_ERR_UNSUPPORTED;
  moe_status st = check_plan(a->plan, a->head_dim);
  if (st != MOE_OK) return st;
  if (a->tokens == 0) return MOE_OK;
  if ((long long)a->tokens * (a->q_heads + a->k_heads) > (1ll << 32) / a->head_dim) return MOE_ERR_UNSUPPORTED;
  const bool k = a->k_heads > 0;
  if (!a->q || !a->q_out || !a->positions || (k && (!a->k || !a->k_out))) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->q, 2) || !aligned(a->q_out, 2) || (k && (!aligned(a->k, 2) || !aligned(a->k_out, 2))))
    return MOE_ERR_INVALID_ARG;
  const long long qw = (long long)a->q_heads * a->head_dim, kw = (long long)a->k_heads * a->head_dim;
  if (a->q_stride < qw || a->q_out_stride < qw || (k && (a->k_stride < kw || a->k_out_stride < kw)))
    return MOE_ERR_INVALID_ARG;
  const Rows q = {a->q, a->q_stride, qw}, qo = {a->q_out, a->q_out_stride, qw};
  const Rows ki = {a->k, a->k_stride, kw}, ko = {a->k_out, a->k_out_stride, kw};
  auto same = [](const Rows& x, const Rows& y) { return x.at == y.at && x.stride == y.stride; };
  const long long n = a->tokens;
  if (!same(q, qo) && rows_overlap(q, qo, n)) return MOE_ERR_INVALID_ARG;
  if (k && ((!same(ki, ko) && rows_overlap(ki, ko, n)) || rows_overlap(qo, ki, n) || rows_overlap(ko, q, n) ||
            rows_overlap(qo, ko, n)))
    return MOE_ERR_INVALID_ARG;
  st = check_device();
  if (st != MOE_OK) return st;
  return launch_rope(*a, (cudaStream_t)stream);
}

moe_status moe_kv4_append_rope(const moe_kv4_append_rope_args* a, moe_stream_t stream) {
  if (a == nullptr || a->tokens < 0 || a->q_heads < 0) return MOE_ERR_INVALID_ARG;
  moe_status st = check_cache(a->cache);
  if (st != MOE_OK) return st;
  st = check_plan(a->plan, a->cache.head_dim);
  if (st != MOE_OK) return st;
  if (a->plan.rotary_dim % (a->plan.adjacent ? 16 : 32) || a->q_heads > 65536 || a->tokens > 1 << 30)
    return MOE_ERR_UNSUPPORTED;
  if (a->tokens == 0) return MOE_OK;
  const long long row = (long long)a->cache.kv_heads * a->cache.head_dim, qw = (long long)a->q_heads * a->cache.head_dim;
  if (!a->k || !a->v || !a->slots || !a->positions || !aligned(a->k, 16) || !aligned(a->v, 16)) return MOE_ERR_INVALID_ARG;
  if (a->k_stride % 8 || a->v_stride % 8 || a->k_stride < row || a->v_stride < row) return MOE_ERR_INVALID_ARG;
  if (a->q_heads > 0) {
    if (!a->q || !a->q_out || !aligned(a->q, 16) || !aligned(a->q_out, 16) || a->q_stride % 8 || a->q_out_stride % 8 ||
        a->q_stride < qw || a->q_out_stride < qw)
      return MOE_ERR_INVALID_ARG;
    const Rows q = {a->q, a->q_stride, qw}, qo = {a->q_out, a->q_out_stride, qw};
    if ((q.at != qo.at || q.stride != qo.stride) && rows_overlap(q, qo, a->tokens)) return MOE_ERR_INVALID_ARG;
    if (rows_overlap(qo, {a->k, a->k_stride, row}, a->tokens) || rows_overlap(qo, {a->v, a->v_stride, row}, a->tokens))
      return MOE_ERR_INVALID_ARG;
  }
  st = check_device();
  if (st != MOE_OK) return st;
  return launch_kv4_append_rope(*a, (cudaStream_t)stream);
}

size_t moe_kv4_index_size(int num_pages, int page_tokens, int kv_heads, int head_dim, int block_tokens) {
  const moe_kv4_cache c = {num_pages, page_tokens, kv_heads, head_dim, 1.0f, 1.0f, nullptr};
  if (check_index_sizes(c, block_tokens) != MOE_OK) return 0;
  const int per = page_tokens > block_tokens ? page_tokens / block_tokens : 1;
  return (size_t)num_pages * per * kv_heads * head_dim * 2;
}

moe_status moe_kv4_index_update(const moe_kv4_index* x, int batch, int max_q, int max_pages, const int32_t* cu_q,
                                const int32_t* kv_len, const int32_t* block_table, int32_t* device_status,
                                moe_stream_t stream) {
  if (x == nullptr || batch < 0 || max_q < 0 || max_pages < 0) return MOE_ERR_INVALID_ARG;
  moe_status st = check_index(*x);
  if (st != MOE_OK) return st;
  if (batch > 4096 || (long long)max_pages * x->cache.page_tokens > INT_MAX - 128) return MOE_ERR_UNSUPPORTED;
  if (batch == 0) return MOE_OK;
  if (max_q < 1 || !cu_q || !kv_len || (!block_table && max_pages > 0)) return MOE_ERR_INVALID_ARG;
  st = check_device();
  if (st != MOE_OK) return st;
  return launch_kv4_index_update(*x, batch, max_q, max_pages, cu_q, kv_len, block_table, device_status,
                                 (cudaStream_t)stream);
}

moe_status moe_kv4_select(const moe_kv4_select_args* a, moe_stream_t stream) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  moe_status st = check_index(a->index);
  if (st == MOE_OK)
    st = check_sparse_sizes(a->index.cache, a->batch, a->q_heads, a->total_q, a->max_q, a->max_pages, a->top);
  if (st != MOE_OK) return st;
  if (a->sink < 0 || a->local < 1 || a->sink > a->top || a->local > a->top - a->sink) return MOE_ERR_INVALID_ARG;
  if (a->batch == 0 || a->total_q == 0) return MOE_OK;
  st = check_sparse_pointers(a->index.cache, a->q_heads, a->max_q, a->max_pages, a->q, a->q_stride, a->cu_q, a->kv_len,
                             a->block_table, a->blocks);
  if (st != MOE_OK) return st;
  st = check_device();
  if (st != MOE_OK) return st;
  return launch_kv4_select(*a, (cudaStream_t)stream);
}

moe_status moe_kv4_sparse_attention(const moe_kv4_sparse_args* a, moe_stream_t stream) {
  if (a == nullptr) return MOE_ERR_INVALID_ARG;
  moe_status st = check_cache(a->cache);
  if (st == MOE_OK) st = check_index_sizes(a->cache, a->block_tokens);
  if (st == MOE_OK) st = check_sparse_sizes(a->cache, a->batch, a->q_heads, a->total_q, a->max_q, a->max_pages, a->top);
  if (st != MOE_OK) return st;
  if (!std::isfinite(a->scale)) return MOE_ERR_INVALID_ARG;
  if (a->batch == 0 || a->total_q == 0) return MOE_OK;
  st = check_sparse_pointers(a->cache, a->q_heads, a->max_q, a->max_pages, a->q, a->q_stride, a->cu_q, a->kv_len,
                             a->block_table, a->blocks);
  if (st != MOE_OK) return st;
  if (!a->out || !aligned(a->out, 16)) return MOE_ERR_INVALID_ARG;
  st = check_device();
  if (st != MOE_OK) return st;
  return launch_kv4_sparse(*a, (cudaStream_t)stream);
}

}  // extern "C"
