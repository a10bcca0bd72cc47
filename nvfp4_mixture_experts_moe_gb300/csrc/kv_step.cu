// One serving step's tables: pages for the new tokens, the slot and position
// of each, from request lengths alone, in one launch.
//
// With P = page_tokens: need_b = ceil((ctx_b + new_b) / P) - ceil(ctx_b / P),
// an inclusive scan S_b over the requests decides who gets pages (S_b <=
// free_count), the i-th page taken is free[free_count - 1 - i], and a token
// at position p of request b goes to table[b][p / P] * P + p % P.
#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

constexpr int kMaxBatch = 4096;
constexpr int kThreads = 1024;
constexpr int kPerThread = kMaxBatch / kThreads;

struct Req {
  int ctx, cnt;      // cleaned lengths
  int need;          // pages it lacks; 0 when its tokens do not fit the table
  bool fits, bad;
};

__device__ __forceinline__ Req load_req(const moe_kv_step_args& a, int b) {
  Req r;
  const int ctx = a.ctx_len[b], cnt = a.new_len[b];
  r.bad = ctx < 0 || cnt < 0;
  r.ctx = max(ctx, 0);
  r.cnt = max(cnt, 0);
  const long long P = a.page_tokens, all = (long long)r.ctx + r.cnt;
  r.fits = all <= P * a.max_pages;
  r.need = r.fits ? (int)((all + P - 1) / P - (r.ctx + P - 1) / P) : 0;
  return r;
}

__device__ __forceinline__ int saturated(long long x) { return (int)min(x, (long long)0x7fffffff); }

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
__global__ void __launch_bounds__(kThreads) kv_step_kernel(moe_kv_step_args a) {
  __shared__ long long warp_cnt[32], warp_need[32];
  __shared__ int cu[kMaxBatch + 1];          // tokens before each request   (both
  __shared__ int first[kMaxBatch + 1];       // pages wanted before each request   saturated)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.batch, P = a.page_tokens;
  const int avail = min(max(*a.free_count, 0), a.free_capacity);
  bool bad = *a.free_count != avail;

  long long cnt[kPerThread], need[kPerThread], sc = 0, sn = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    cnt[i] = need[i] = 0;
    if (b < B) {
      const Req r = load_req(a, b);
      cnt[i] = r.cnt;
      need[i] = r.need;
      bad |= r.bad || !r.fits;
    }
    sc += cnt[i];
    sn += need[i];
  }
  long long ic = sc, in = sn;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, ic, o), y = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) {
      ic += x;
      in += y;
    }
  }
  if (lane == 31) {
    warp_cnt[warp] = ic;
    warp_need[warp] = in;
  }
  __syncthreads();
  long long bc = ic - sc, bn = in - sn;
  for (int w = 0; w < warp; ++w) {
    bc += warp_cnt[w];
    bn += warp_need[w];
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    if (b <= B) {
      cu[b] = saturated(bc);
      first[b] = saturated(bn);
    }
    bc += cnt[i];
    bn += need[i];
  }
  if (tid == kThreads - 1 && B == kMaxBatch) {
    cu[B] = saturated(bc);
    first[B] = saturated(bn);
  }
  bad |= bc > a.tokens;
  __syncthreads();

  // requests whose inclusive sum fits the stack get their pages: a prefix
  const int granted = last_at_most(first, B, avail);   // requests [0, granted) fit
  const int taken = first[granted];
  const int gthread = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;

  if (blockIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int b = tid * kPerThread + i;
      if (b < B) {
        const Req r = load_req(a, b);
        const bool ok = r.fits && (r.need == 0 || b < granted);
        bad |= !ok;
        a.kv_len[b] = ok ? r.ctx + r.cnt : r.ctx;
      }
      if (b <= B) a.cu_q[b] = cu[b];
    }
    if (tid == kThreads - 1 && B == kMaxBatch) a.cu_q[B] = cu[B];
    if (tid == 0) *a.free_count_out = avail - taken;
    if (bad && a.device_status != nullptr) *a.device_status = MOE_ERR_DEVICE;
  }

  for (int i = gthread; i < taken; i += gsize) {
    const int b = last_at_most(first, B, i);  // the last request that starts at or before page i takes it
    const int old = (int)(((long long)max(a.ctx_len[b], 0) + P - 1) / P);
    a.block_table[(size_t)b * a.max_pages + old + (i - first[b])] = a.free_pages[avail - 1 - i];
  }

  for (int t = gthread; t < a.tokens; t += gsize) {
    int slot = -1, pos = 0;
    if (t < cu[B]) {
      const int b = last_at_most(cu, B, t);
      const Req r = load_req(a, b);
      const long long at = (long long)r.ctx + (t - cu[b]);
      pos = saturated(at);
      if (r.fits && (r.need == 0 || b < granted)) {
        const int page = pos / P, old = (int)(((long long)r.ctx + P - 1) / P);
        const int id = page < old ? a.block_table[(size_t)b * a.max_pages + page]
                                  : a.free_pages[avail - 1 - (first[b] + page - old)];
        const long long s = (long long)id * P + (pos - page * P);
        slot = id < 0 || s > 0x7fffffff ? -1 : (int)s;
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
}

}  // namespace

moe_status launch_kv_step(const moe_kv_step_args& a, cudaStream_t s) {
  const int sms = sm_count();
  const int want = (int)(((long long)a.tokens + kThreads - 1) / kThreads);
  const int ctas = want < 1 ? 1 : (want < sms ? want : sms);
  cudaError_t e = launch_ex(false, kv_step_kernel, dim3(ctas), dim3(kThreads), 0, s, a);
  if (e != cudaSuccess) return cuda_ok(e);
  count_launches(1);
  return MOE_OK;
}

}  // namespace moe
