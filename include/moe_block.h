/*
 * moe_block.h -- C ABI of the operators a decoder block runs around the
 * fused NVFP4 MoE layer (moe_nvfp4.h) when it serves tokens:
 *
 *   moe_kv_step        block tables and slot maps of one step, from request lengths
 *   moe_kv4_append     keys and values into a paged NVFP4 cache
 *   moe_kv4_read       cached rows back to bf16
 *   moe_kv4_attention  attention over that cache (single tokens, drafted tokens, prompts)
 *   moe_block_norm     norm after a block, gate, residual, norm before the next block
 *
 * The conventions of moe_nvfp4.h hold: device pointers unless a comment says
 * "host", caller-owned buffers, asynchronous on `stream`, argument errors
 * found on the host before anything is enqueued, bf16 as uint16_t bit
 * patterns, sm_103 only. `device_status` arguments (nullable, device int32)
 * are set to MOE_ERR_DEVICE when the device meets bad data and left alone
 * otherwise.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * The NVFP4 key/value cache: one pool of pages of `page_tokens` tokens.
 *
 * Layout: uint8 [num_pages][kv_heads][page_tokens / 16][18 * head_dim]. Each
 * block of 16 tokens holds, one after the other,
 *   key codes    [16][head_dim / 2]   e2m1, element 2j in the low nibble of byte j
 *   key scales   [16][head_dim / 16]  E4M3, one per 16 elements
 *   value codes  [16][head_dim / 2]
 *   value scales [16][head_dim / 16]
 * so that any run of blocks of one (page, head) is one contiguous copy. A
 * value decodes as e2m1 * e4m3 / gs with the keys' or the values' global
 * scale (quant convention, calibrated once per layer; the kernels multiply by
 * the fp32 reciprocal). 0.5625 bytes per
 * element ("Qwen3.8-Flash-Next-NVFP4 . 2x DGX Spark . SGLang TP2": packed FP4
 * and FP8 scales for the KV cache).
 *
 * slot = page * page_tokens + position within the page.
 * Limits: page_tokens 16, 32, 64 or 128; head_dim 64 or 128; kv_heads 1..1024;
 * num_pages * page_tokens <= 2^31 - 1; k_gs, v_gs positive and finite; pool
 * 16-byte aligned. The pool needs no initialisation: what was not appended is
 * never used in a result.
 */
typedef struct {
  int num_pages, page_tokens, kv_heads, head_dim;
  float k_gs, v_gs;
  void* pool;
} moe_kv4_cache;

/* Bytes of a pool; 0 for sizes outside the limits. */
size_t moe_kv4_pool_size(int num_pages, int page_tokens, int kv_heads, int head_dim);

/* Quantises `tokens` rows of keys and values into the cache, with the steps
 * of moe_nvfp4_quantize_static (amax / 6 * gs to E4M3, codes of x * (gs /
 * scale), nearest even, saturating). A NaN element is stored as 0, an
 * infinite one saturates.
 *
 * k, v   bf16 [tokens, kv_heads, head_dim]; row t starts k_stride (v_stride)
 *        elements after row t - 1, a row's heads are contiguous
 * slots  int32 [tokens]; a negative slot's token is skipped; a slot past the
 *        pool is skipped and reported in device_status; slots of one call are
 *        distinct (otherwise either row may end up stored)
 * Errors: NULL or not 16-byte aligned k, v, pool; a stride that is not a
 * multiple of 8 or smaller than kv_heads * head_dim; sizes outside the limits
 * -> MOE_ERR_INVALID_ARG (head_dim or page_tokens of another value ->
 * MOE_ERR_UNSUPPORTED). tokens = 0 -> MOE_OK.
 */
moe_status moe_kv4_append(const moe_kv4_cache* cache, const uint16_t* k, const uint16_t* v,
                          long long k_stride, long long v_stride, const int32_t* slots, int tokens,
                          int32_t* device_status, moe_stream_t stream);

/* Cached rows back to bf16: k_out, v_out bf16 [n, kv_heads, head_dim] (either
 * may be NULL), e2m1 * e4m3 / gs rounded once to bf16. A negative slot gives
 * zeros; a slot past the pool gives zeros and is reported in device_status.
 */
moe_status moe_kv4_read(const moe_kv4_cache* cache, const int32_t* slots, int n, uint16_t* k_out,
                        uint16_t* v_out, int32_t* device_status, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention over the cache. Request b has the query rows cu_q[b] ..
 * cu_q[b+1] - 1 and kv_len[b] cached tokens, its new ones (already appended)
 * included; its query i stands at position kv_len[b] - n_b + i. Query head h
 * reads key/value head h / (q_heads / kv_heads).
 *
 *   s_j = scale * q . k_j;  p = softmax(s over the visible j);  out = sum p_j v_j
 *
 * causal = 1: j <= position; window > 0 (causal only): also j > position -
 * window. A query that sees nothing gets a zero row and lse = -inf; one with a
 * NaN gets NaN in both (an infinity does where its scores have no softmax),
 * and no other row changes. lse is the natural logarithm of sum exp(s_j).
 * Products of q with the codes are exact, sums and softmax statistics are
 * fp32; the probabilities enter the second product as f16. Results do not
 * depend on timing: the same call gives the same bits.
 *
 * q           bf16 [total_q, q_heads, head_dim], row stride q_stride elements
 * cu_q        int32 [batch + 1], ascending from 0; cu_q[batch] <= total_q
 * kv_len      int32 [batch]
 * block_table int32 [batch, max_pages]
 * max_q       host bound on every request's query rows (chooses the kernels)
 * out         bf16 [total_q, q_heads, head_dim]; rows no request owns are left alone
 * lse         fp32 [total_q, q_heads] or NULL
 * ws          moe_kv4_attention_workspace_size(args) bytes, 256-byte aligned;
 *             its first MOE_KV4_WS_ZERO bytes must be zero before its first
 *             use (the library leaves them so); one call at a time.
 * Bad device data is reported as MOE_ERR_DEVICE in the workspace status word
 * (moe_get_device_status): a page id outside the pool (its tokens count as
 * hidden), kv_len above max_pages * page_tokens (cut there), more query rows
 * than max_q or total_q (those requests' rows are not written). What lies
 * before every query's window is not used: those tokens need not have been
 * appended, and entries of pages that hold no others may be anything.
 * Errors: NULL pointers (lse may be), misaligned pool / q / out (16 bytes), a
 * q_stride that is not a multiple of 8 or smaller than a row, negative sizes,
 * max_q < 1, a non-finite scale, a window without causal ->
 * MOE_ERR_INVALID_ARG; q_heads % kv_heads != 0, head_dim or page_tokens
 * outside the cache's limits, batch > 4096, max_pages * page_tokens > 2^31 -
 * 129, or more than 2^31 - 1 (request, head, 32 cached tokens) or (256 rows,
 * head, 128 cached tokens) tiles, the table taken as full ->
 * MOE_ERR_UNSUPPORTED; a missing, misaligned or short workspace ->
 * MOE_ERR_WORKSPACE. batch = 0 or total_q = 0 -> MOE_OK with nothing enqueued.
 */
typedef struct {
  moe_kv4_cache cache;
  int batch, q_heads, total_q, max_q, max_pages;
  const uint16_t* q;
  long long q_stride;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* block_table;
  float scale;
  int causal;
  int window;
  uint16_t* out;
  float* lse;
} moe_kv4_attn_args;

#define MOE_KV4_WS_ZERO 4096
size_t moe_kv4_attention_workspace_size(const moe_kv4_attn_args* args);
moe_status moe_kv4_attention(const moe_kv4_attn_args* args, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * One step's tables. Request b holds ctx_len[b] cached tokens in the pages
 * block_table[b][0 .. ceil(ctx_len[b] / page_tokens)) and brings new_len[b]
 * more. Pages it then lacks are taken from the free stack in request order:
 * the i-th page taken is free_pages[free_count - 1 - i].
 *
 * A request is refused when the stack cannot cover it and everything before
 * it, or when its tokens would not fit max_pages pages (such a request takes
 * nothing from the ones after it). A request that needs no new page is never
 * refused for lack of pages. A refused request keeps its pages and length;
 * its new tokens get slot -1 and device_status becomes MOE_ERR_DEVICE. A
 * token whose page id (from the table or the stack) is negative, or gives a
 * slot past 2^31 - 1, gets slot -1 and is reported too.
 *
 * ctx_len, new_len int32 [batch] (a negative value counts as 0 and is reported)
 * block_table      int32 [batch, max_pages], in place: only the new entries are written
 * free_pages       int32 [free_capacity]
 * free_count       int32 [1]; free_count_out int32 [1] out
 * kv_len           int32 [batch] out: ctx_len + new_len, or ctx_len when refused
 * cu_q             int32 [batch + 1] out: prefix sums of new_len
 * slots, positions int32 [tokens] out: slot and position of each new token, in
 *                  request order; entries past the step's tokens get -1 and 0
 * tokens           host bound on the step's tokens (new tokens past it are
 *                  reported and not written; cu_q stays at the true sums)
 * Errors: batch outside 0..4096 -> MOE_ERR_UNSUPPORTED; page_tokens < 1,
 * max_pages < 1, negative sizes, max_pages * page_tokens > 2^31 - 1, NULL
 * pointers, an output that overlaps an input or another output ->
 * MOE_ERR_INVALID_ARG.
 */
typedef struct {
  int batch, page_tokens, max_pages, tokens, free_capacity;
  const int32_t* ctx_len;
  const int32_t* new_len;
  int32_t* block_table;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* kv_len;
  int32_t* cu_q;
  int32_t* slots;
  int32_t* positions;
  int32_t* device_status;
} moe_kv_step_args;

moe_status moe_kv_step(const moe_kv_step_args* args, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Norm after a block, its gate, the residual and the norm before the next
 * block, in one pass over each row:
 *
 *   n = x * rsqrt(mean(x^2) + eps) * (w_post + w_offset)     (w_post NULL: n = x)
 *   r = residual_scale * residual + branch_scale * gate * n  (gate NULL: 1; x NULL: no second term)
 *   residual_out = r;  out = r * rsqrt(mean(r^2) + eps) * (w_pre + w_offset)
 *
 * All in fp32 from the inputs on, each output rounded once (the second norm
 * takes r before its rounding).
 *
 * x            bf16 [T, H] (row stride x_stride) or NULL
 * gate         bf16: [T, H] with row stride gate_stride, or [H] for every row (gate_stride = 0), or NULL
 * residual     bf16 or (residual_f32) fp32 [T, H], row stride residual_stride
 * w_post, w_pre bf16 [H] or NULL; with w_pre NULL `out` is not written (may be NULL)
 * residual_out like residual, [T, H] contiguous; may be `residual` itself when
 *              that is contiguous; NULL: not written
 * out          bf16 [T, H] contiguous
 * Limits: 1 <= H <= 16384, any alignment of the element type; strides >= H.
 * Errors: sizes, strides, NULL residual, both outputs missing, non-finite
 * scales, eps < 0 -> MOE_ERR_INVALID_ARG; H > 16384 -> MOE_ERR_UNSUPPORTED.
 */
typedef struct {
  int T, H;
  const uint16_t* x;
  long long x_stride;
  const uint16_t* gate;
  long long gate_stride;
  const void* residual;
  long long residual_stride;
  int residual_f32;
  const uint16_t* w_post;
  const uint16_t* w_pre;
  float residual_scale, branch_scale, eps, w_offset;
  void* residual_out;
  uint16_t* out;
} moe_block_norm_args;

moe_status moe_block_norm(const moe_block_norm_args* args, moe_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_BLOCK_H */
