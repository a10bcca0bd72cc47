// Attention over the NVFP4 cache: which kernel takes which request.
#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {

// A request's query rows per key/value head (its new tokens times the group's
// query heads) decide its kernel: up to kKvDecodeRows the mma.sync kernel,
// which streams the cache at its rate with rows padded to 8 or 16, above that
// the tcgen05 kernel, whose tiles hold 128 rows. Lengths live on the device,
// so a call whose max_q allows both kinds launches both and each skips the
// other's requests; a call of one request needs only the kernel for max_q, and
// a group of more query heads than the first takes rows only the second.
static int decode_rows(const moe_kv4_attn_args& a) {
  const int group = a.q_heads / a.cache.kv_heads;
  const long long rows = (long long)a.max_q * group;
  if (rows <= kKvDecodeRows) return (int)rows;
  return a.batch == 1 || group > kKvDecodeRows ? 0 : kKvDecodeRows;
}

static bool any_prompt(const moe_kv4_attn_args& a) {
  return (long long)a.max_q * (a.q_heads / a.cache.kv_heads) > kKvDecodeRows;
}

// The two kernels of a call overlap: each has its own part of the workspace.
// A workspace serves calls of any smaller size, fewer query heads among them,
// so a group too wide for the first kernel leaves its part in.
static size_t decode_ws_bytes(const moe_kv4_attn_args& a) {
  const int few = any_prompt(a) ? (a.batch == 1 ? 0 : kKvDecodeRows) : decode_rows(a);
  return few > 0 ? align_up(kv4_decode_ws_floats(a.cache.head_dim, few) * sizeof(float)) : 0;
}

size_t kv4_attention_ws_bytes(const moe_kv4_attn_args& a) {
  const size_t many = any_prompt(a) ? kv4_prompt_ws_floats(a.cache.head_dim) * sizeof(float) : 0;
  return align_up(MOE_KV4_WS_ZERO + decode_ws_bytes(a) + many);
}

moe_status launch_kv4_attention(const moe_kv4_attn_args& args, void* ws, cudaStream_t s) {
  moe_kv4_attn_args a = args;
  // A window of all the tokens a table holds hides none. Below that the
  // kernels' position - window stays within 32 bits, also for queries that
  // stand before token 0.
  if (a.window >= a.max_pages * a.cache.page_tokens) a.window = 0;
  int* status = &static_cast<WsHeader*>(ws)->status;
  int* counters = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + sizeof(WsHeader));
  static_assert(sizeof(WsHeader) + kKvMaxCtas * sizeof(int) <= MOE_KV4_WS_ZERO, "zero region");
  uint8_t* const partials = static_cast<uint8_t*>(ws) + MOE_KV4_WS_ZERO;
  const int few = decode_rows(a);
  moe_status st = MOE_OK;
  if (few > 0) st = launch_kv4_decode(a, few, status, counters, reinterpret_cast<float*>(partials), s);
  if (st == MOE_OK && any_prompt(a))
    st = launch_kv4_prompt(a, few, status, reinterpret_cast<float*>(partials + decode_ws_bytes(a)), few > 0, s);
  return st;
}

}  // namespace moe
