// Which request a query row belongs to, found on the device.
#pragma once

#include "kernels.cuh"
#include "kv4.cuh"

namespace moe {

struct RowOwner {
  int b;         // request, -1: none (or one whose lengths cannot be)
  int c0, n;     // its first row, its rows
  int kv;        // its cached tokens, at most its table's
  bool bad;
};

// Request b, its lengths cut to what the tables hold; n is set, b is -1 and bad
// true for one whose rows cannot be.
__device__ __forceinline__ RowOwner request_of(const int32_t* cu_q, const int32_t* kv_len, int total_q, int max_q, int cap,
                                               int b) {
  const int c0 = __ldg(cu_q + b), c1 = __ldg(cu_q + b + 1), kv = __ldg(kv_len + b);
  RowOwner r = {b, c0, c1 - c0, max(0, min(kv, cap)), false};
  r.bad = kv != r.kv;
  if (c0 < 0 || r.n < 0 || c1 > total_q || r.n > max_q) {
    r.b = -1;
    r.bad = true;
  }
  return r;
}

// The request of row t, by a whole warp: cu_q ascends from 0. One load decides
// where every request before t has one row (a decode step); otherwise 32
// places at a time.
__device__ __forceinline__ RowOwner row_owner(const int32_t* cu_q, const int32_t* kv_len, int batch, int total_q, int max_q,
                                              int cap, int t) {
  const int lane = threadIdx.x & 31;
  RowOwner r = {-1, 0, 0, 0, false};
  const int guess = min(t, batch - 1);
  int lo = guess;
  if (__ldg(cu_q + lo) > t || __ldg(cu_q + lo + 1) <= t) {
    lo = 0;   // the last b with cu_q[b] <= t lies in [lo, lo + width)
    for (int width = batch; width > 1;) {
      const int step = (width + 31) / 32, at = lo + lane * step;
      const unsigned below = __ballot_sync(0xffffffffu, at < lo + width && __ldg(cu_q + at) <= t);
      const int k = max(31 - __clz((int)below), 0);
      const int end = lo + width;
      lo += k * step;
      width = min(step, end - lo);
    }
  }
  if (__ldg(cu_q + lo) > t || __ldg(cu_q + lo + 1) <= t) return r;   // past the last request
  return request_of(cu_q, kv_len, total_q, max_q, cap, lo);
}

}  // namespace moe
