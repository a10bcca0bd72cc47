// One serving step's tables: pages for the new tokens, the slot and position
// of each, from request lengths alone, in one launch.
//
// With P = page_tokens: need_b = ceil((ctx_b + new_b) / P) - ceil(ctx_b / P),
// an inclusive scan S_b over the requests decides who gets pages (S_b <=
// free_count), the i-th page taken is free[free_count - 1 - i], and a token
// at position p of request b goes to table[b][p / P] * P + p % P.
//
// What bounds it: latency. Lengths, then a table entry, then the store are
// three trips to memory of some 0.7 us; the scan between them is shuffles
// and one exchange between warps. 64 decoding requests take 2.9 us, 500
// requests with 31,000 new tokens 4.4 (replayed).
#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

constexpr int kMaxBatch = 4096;
constexpr int kMaxThreads = 1024;

struct Req {
  int ctx, cnt;      // cleaned lengths
  int need;          // pages it lacks; 0 when its tokens do not fit the table
  bool fits, bad;
};

__device__ __forceinline__ unsigned ceil_div(unsigned a, unsigned b) { return (a + b - 1) / b; }

// A row of the table holds at most INT_MAX tokens, so two cleaned lengths that
// fit it, and their sum rounded up, are below 2^32.
__device__ __forceinline__ Req load_req(const moe_kv_step_args& a, int b) {
  Req r;
  const int ctx = a.ctx_len[b], cnt = a.new_len[b];
  r.bad = ctx < 0 || cnt < 0;
  r.ctx = max(ctx, 0);
  r.cnt = max(cnt, 0);
  const unsigned P = a.page_tokens, all = (unsigned)r.ctx + (unsigned)r.cnt;
  r.fits = all <= P * (unsigned)a.max_pages;
  r.need = r.fits ? (int)(ceil_div(all, P) - ceil_div(r.ctx, P)) : 0;
  return r;
}

// Sums are capped at 2^31: past every token and page there can be.
constexpr unsigned kCap = 1u << 31;
__device__ __forceinline__ unsigned add_capped(unsigned a, unsigned b) { return a + min(b, kCap - a); }
__device__ __forceinline__ int saturated(unsigned x) { return (int)min(x, 0x7fffffffu); }

__device__ __forceinline__ void warp_scan(unsigned& c, unsigned& n, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, c, o), y = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) {
      c = add_capped(c, x);
      n = add_capped(n, y);
    }
  }
}

// Last index i in [0, n] with arr[i] <= x, for an ascending arr with arr[0] <= x.
__device__ __forceinline__ int last_at_most(const int* arr, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (arr[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Every CTA scans all the lengths (at most 4096) for itself, so nothing waits
// on another CTA; the pages and the tokens are then dealt out over the grid.
// New pages are read from the free stack, never from table entries that
// another CTA may be writing.
// kPer requests per thread.
template <int kPer>
__global__ void __launch_bounds__(kMaxThreads) kv_step_kernel(moe_kv_step_args a) {
  __shared__ unsigned warp_cnt[32], warp_need[32];
  __shared__ int cu[kMaxThreads * kPer + 1];      // tokens before each request   (both
  __shared__ int first[kMaxThreads * kPer + 1];   // pages wanted before each request   saturated)
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.batch, P = a.page_tokens;
  pdl_wait();
  const int count = *a.free_count;

  unsigned cnt[kPer], need[kPer], sc = 0, sn = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    cnt[i] = need[i] = 0;
    if (b < B) {
      const Req r = load_req(a, b);
      cnt[i] = r.cnt;
      need[i] = r.need;
      bad |= r.bad || !r.fits;
    }
    sc = add_capped(sc, cnt[i]);
    sn = add_capped(sn, need[i]);
  }
  unsigned ic = sc, in = sn;
  warp_scan(ic, in, lane);
  if (lane == 31) {
    warp_cnt[warp] = ic;
    warp_need[warp] = in;
  }
  __syncthreads();
  unsigned tc = lane < (threads >> 5) ? warp_cnt[lane] : 0, tn = lane < (threads >> 5) ? warp_need[lane] : 0;
  warp_scan(tc, tn, lane);
  const unsigned all_cnt = __shfl_sync(0xffffffffu, tc, 31), all_need = __shfl_sync(0xffffffffu, tn, 31);
  tc = __shfl_sync(0xffffffffu, tc, max(warp - 1, 0));
  tn = __shfl_sync(0xffffffffu, tn, max(warp - 1, 0));
  // tokens and pages before this thread's requests: the warps before and the lanes before
  unsigned bc = __shfl_up_sync(0xffffffffu, ic, 1), bn = __shfl_up_sync(0xffffffffu, in, 1);
  bc = add_capped(warp ? tc : 0, lane ? bc : 0);
  bn = add_capped(warp ? tn : 0, lane ? bn : 0);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    if (b < B) {
      cu[b] = saturated(bc);
      first[b] = saturated(bn);
    }
    bc = add_capped(bc, cnt[i]);
    bn = add_capped(bn, need[i]);
  }
  if (tid == 0) {
    cu[B] = saturated(all_cnt);
    first[B] = saturated(all_need);
  }
  const int avail = min(max(count, 0), a.free_capacity);
  bad |= count != avail || all_cnt > (unsigned)a.tokens;
  __syncthreads();

  // requests whose inclusive sum fits the stack get their pages: a prefix
  const int granted = last_at_most(first, B, avail);   // requests [0, granted) fit
  const int taken = first[granted];
  const int gthread = blockIdx.x * threads + tid, gsize = gridDim.x * threads;

  if (blockIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * kPer + i;
      if (b < B) {
        const Req r = load_req(a, b);
        const bool ok = r.fits && (r.need == 0 || b < granted);
        bad |= !ok;
        a.kv_len[b] = ok ? r.ctx + r.cnt : r.ctx;
      }
      if (b < B) a.cu_q[b] = cu[b];
    }
    if (tid == 0) {
      a.cu_q[B] = cu[B];
      *a.free_count_out = avail - taken;
    }
    if (bad && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
  }

  // (unsigned: a step past the last of 2^31 - 1 stays an integer past it)
  for (unsigned next = gthread; next < (unsigned)taken; next += gsize) {
    const int i = (int)next;
    const int b = last_at_most(first, B, i);  // the last request that starts at or before page i takes it
    const int old = (int)ceil_div(max(a.ctx_len[b], 0), P);
    a.block_table[(size_t)b * a.max_pages + old + (i - first[b])] = a.free_pages[avail - 1 - i];
  }

  for (unsigned next = gthread; next < (unsigned)a.tokens; next += gsize) {
    const int t = (int)next;
    int slot = -1, pos = 0;
    if (t < cu[B]) {
      const int b = last_at_most(cu, B, t);
      const Req r = load_req(a, b);
      pos = saturated((unsigned)r.ctx + (unsigned)(t - cu[b]));
      if (r.fits && (r.need == 0 || b < granted)) {
        const int page = pos / P, old = (int)ceil_div(r.ctx, P);
        const int id = page < old ? a.block_table[(size_t)b * a.max_pages + page]
                                  : a.free_pages[avail - 1 - (first[b] + page - old)];
        const long long s = (long long)id * P + (pos - page * P);
        slot = id < 0 || s > 0x7fffffff ? -1 : (int)s;
        if (slot < 0 && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
}

}  // namespace

moe_status launch_kv_step(const moe_kv_step_args& a, cudaStream_t s) {
  // A thread per request and per token of an SM's share, as far as 1024 go;
  // small CTAs start and synchronise sooner.
  const long long sms = sm_count(), share = (a.tokens + sms - 1) / sms;
  const long long want = share > a.batch ? share : a.batch;
  const int threads = want > kMaxThreads ? kMaxThreads : want < 128 ? 128 : (int)(want + 31) / 32 * 32;
  const long long need = ((long long)a.tokens + threads - 1) / threads;
  const int ctas = (int)(need < 1 ? 1 : need < sms ? need : sms);
  auto k = a.batch <= threads ? kv_step_kernel<1> : kv_step_kernel<kMaxBatch / kMaxThreads>;
  cudaError_t e = launch_ex(true, k, dim3(ctas), dim3(threads), 0, s, a);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

}  // namespace moe
