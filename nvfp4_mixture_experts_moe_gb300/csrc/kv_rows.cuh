// Attention of up to 16 query rows over NVFP4 rows in shared memory, a warp at
// a time: what the few-row kernels share (mathematics and figures in
// kv_attention_decode.cu).
#pragma once

#include "kernels.cuh"
#include "kv4.cuh"
#include "kv_math.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace rows {

using namespace kv;

// One partial result: rows x D fp32 output, then (m, l) of each row.
template <int D, int NT>
struct Slots {
  static constexpr int kRows = 8 * NT;
  static constexpr int kFloats = kRows * (D + 2);
};

// Row of the MMA's token side <-> token of a 16-token block (the same map
// within each half): with it the 16-byte key loads are free of bank conflicts
// and the value loads have two-way ones (128 cycles of shared memory a tile
// with the identity, 80 with this).
__device__ __forceinline__ int token_of(int r) { return r ^ ((r >> 1) & 1); }

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// What a warp holds of 8 NT rows: the rows as B fragments, out^T (rows d,
// columns query rows), and of columns 2 t4 and 2 t4 + 1 the factor of a score,
// m and this lane's share of l.
template <int D, int NT>
struct RowState {
  uint32_t qf[NT][D / 16][2];
  float o[NT][D / 16][4];
  float mult[NT][2], m[NT][2], l[NT][2];
};

// Rows as f16 times a power of two, and empty sums. row_of(r): where row r
// starts, nullptr for one that is not there. g8, t4: lane / 4 and lane % 4 (an
// argument: worked out here they cost the tile loop 2.5 %).
template <int D, int NT, class RowOf>
__device__ __forceinline__ void start_rows(RowState<D, NT>& st, int g8, int t4, float scale, float k_gs, RowOf row_of) {
  constexpr int MT = D / 16;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = nt * 8 + g8;
    const uint16_t* q = row_of(row);   // nullptr: none
    uint4 raw[D / 32];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      raw[i] = q != nullptr ? __ldg(reinterpret_cast<const uint4*>(q + t4 * (D / 4)) + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      mx = max_u16x2(max_u16x2(mx, raw[i].x & 0x7fff7fffu), raw[i].y & 0x7fff7fffu);
      mx = max_u16x2(max_u16x2(mx, raw[i].z & 0x7fff7fffu), raw[i].w & 0x7fff7fffu);
    }
    mx = max_u16x2(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = max_u16x2(mx, __shfl_xor_sync(kFull, mx, 2));
    // largest element to [2^14, 2^15) (smaller only below 2^-112)
    const uint32_t big = max(mx & 0xffffu, mx >> 16);
    const int ex = min(max((int)(big >> 7), 15), 254);
    // a larger score is a larger product; a row with a NaN or an infinity has no softmax whatever it sees: all NaN
    // (chosen in one expression with the sign, 4 x 131072 tokens take 108.6 us of 107.5)
    float up = scale < 0.0f ? -pow2(141 - ex) : pow2(141 - ex);
    up += big >= 0x7f80u ? __int_as_float(0x7fffffff) : 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        st.qf[nt][2 * i + j / 2][j & 1] = pack_f16x2(__uint_as_float(w[j] << 16) * up,
                                                  __uint_as_float(w[j] & 0xffff0000u) * up);
    }
    // row g8's factor, fetched as columns 2t, 2t + 1; never 0, so that a hidden score stays -inf
    const float mine = fmaxf(fabsf(scale) * kLog2e / k_gs * pow2(ex - 141), 1e-37f);
    st.mult[nt][0] = __shfl_sync(kFull, mine, 8 * t4);
    st.mult[nt][1] = __shfl_sync(kFull, mine, 8 * t4 + 4);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      st.m[nt][c] = -INFINITY;
      st.l[nt][c] = 0.0f;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.o[nt][mt][i] = 0.0f;
  }
}

// The products and the softmax of kPart blocks of 16 tokens. kMask: hidden(blk,
// nt, i) says whether element i of the accumulator of a block is not seen.
template <int D, int NT, int kPart, bool kMask, class Hidden>
__device__ __forceinline__ void attend_blocks(RowState<D, NT>& st, int g8, int t4, const uint8_t* part, Hidden hidden) {
  using L = Kv4Block<D>;
  constexpr int MT = D / 16, kKeyWords = D / 32;   // 32-bit code words of one key row per lane
  // ---------------------------------------------------------- scores
  float s[NT][kPart][4];
#pragma unroll
  for (int blk = 0; blk < kPart; ++blk) {
    const uint8_t* kb = part + blk * L::kBytes;
    uint32_t kw[2][kKeyWords];   // key codes of MMA rows g8 and g8 + 8
    uint32_t ks[2][2];           // their scales, each doubled to f16x2
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = token_of(g8) + 8 * r;
      const uint8_t* sf = kb + L::kKeyScales + row * L::kScaleRow;
      if constexpr (D == 128) {
        const uint4 v = *reinterpret_cast<const uint4*>(kb + row * L::kCodeRow + 16 * t4);
        kw[r][0] = v.x, kw[r][1] = v.y, kw[r][2] = v.z, kw[r][3] = v.w;
        const uint32_t two = cvt_e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(sf + 2 * t4));
        ks[r][0] = __byte_perm(two, 0, 0x1010);
        ks[r][1] = __byte_perm(two, 0, 0x3232);
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(kb + row * L::kCodeRow + 8 * t4);
        kw[r][0] = v.x, kw[r][1] = v.y;
        ks[r][0] = ks[r][1] = cvt_e4m3x2_f16x2((uint32_t)sf[t4] * 0x101u);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][blk][i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kKeyWords; ++w) {
      uint32_t lo[4], hi[4];
      cvt_e2m1x8_f16(kw[0][w], lo);
      cvt_e2m1x8_f16(kw[1][w], hi);
      const uint32_t s0 = ks[0][w * 2 / kKeyWords], s1 = ks[1][w * 2 / kKeyWords];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t af[4] = {hmul2_u32(lo[2 * i], s0), hmul2_u32(hi[2 * i], s1),
                                hmul2_u32(lo[2 * i + 1], s0), hmul2_u32(hi[2 * i + 1], s1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(s[nt][blk], af, st.qf[nt][2 * w + i][0], st.qf[nt][2 * w + i][1]);
      }
    }
    if constexpr (kMask) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (hidden(blk, nt, i)) s[nt][blk][i] = -INFINITY;
    }
  }

  // ------------------------------------------- running maximum and p
  bool grow = false;
  float top[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float x = fmaxf(s[nt][0][c], s[nt][0][c + 2]);
#pragma unroll
      for (int blk = 1; blk < kPart; ++blk) x = fmaxf(x, fmaxf(s[nt][blk][c], s[nt][blk][c + 2]));
      top[nt][c] = x * st.mult[nt][c];
      grow |= top[nt][c] > st.m[nt][c] + kSlack;
    }
  if (__any_sync(kFull, grow)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = top[nt][c];
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
        x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
        const float mn = fmaxf(st.m[nt][c], x - kLead);
        const float f = mn == -INFINITY ? 1.0f : ex2(st.m[nt][c] - mn);   // 0 from -inf
        st.m[nt][c] = mn;
        st.l[nt][c] *= f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          st.o[nt][mt][c] *= f;
          st.o[nt][mt][c + 2] *= f;
        }
      }
  }
  uint32_t pf[NT][kPart][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float m0 = st.m[nt][0], m1 = st.m[nt][1];
    if constexpr (kMask) {   // a row that has seen nothing yet
      if (m0 == -INFINITY) m0 = 0.0f;
      if (m1 == -INFINITY) m1 = 0.0f;
    }
#pragma unroll
    for (int blk = 0; blk < kPart; ++blk) {
      const float p0 = ex2(fmaf(s[nt][blk][0], st.mult[nt][0], -m0)), p1 = ex2(fmaf(s[nt][blk][1], st.mult[nt][1], -m1));
      const float p2 = ex2(fmaf(s[nt][blk][2], st.mult[nt][0], -m0)), p3 = ex2(fmaf(s[nt][blk][3], st.mult[nt][1], -m1));
      st.l[nt][0] += p0 + p2;
      st.l[nt][1] += p1 + p3;
      pf[nt][blk][0] = movmatrix_trans(pack_f16x2(p0, p1));
      pf[nt][blk][1] = movmatrix_trans(pack_f16x2(p2, p3));
    }
  }

  // ----------------------------------------------------------- values
#pragma unroll
  for (int blk = 0; blk < kPart; ++blk) {
    const uint8_t* vb = part + blk * L::kBytes;
    uint32_t vw[4][MT / 4];    // value codes of MMA columns 2t, 2t + 1, 2t + 8, 2t + 9
    uint32_t sc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int tok = token_of(2 * t4 + (k & 1)) + 8 * (k >> 1);
      sc[k] = vb[L::kValueScales + tok * L::kScaleRow + (D == 128 ? g8 : g8 / 2)];
      if constexpr (D == 128) {
        const uint2 v = *reinterpret_cast<const uint2*>(vb + L::kValueCodes + tok * L::kCodeRow + 8 * g8);
        vw[k][0] = v.x, vw[k][1] = v.y;
      } else {
        vw[k][0] = *reinterpret_cast<const uint32_t*>(vb + L::kValueCodes + tok * L::kCodeRow + 4 * g8);
      }
      // What was never appended, lies before every row's window or has a
      // bad page is hidden (p = 0), but its scale may decode as NaN, which
      // no appended row's does: 0 instead.
      if constexpr (kMask) {
        if ((sc[k] & 0x7fu) == 0x7fu) sc[k] = 0;
      }
    }
    const uint32_t s01 = cvt_e4m3x2_f16x2(sc[0] | sc[1] << 8), s23 = cvt_e4m3x2_f16x2(sc[2] | sc[3] << 8);
#pragma unroll
    for (int w = 0; w < MT / 4; ++w) {
      // bytes (even d of token 2t, of 2t + 1) and (odd d ...): one conversion gives an MMA register
      uint32_t e01[4], o01[4], e23[4], o23[4];
      cvt_e2m1x8_f16((vw[0][w] & 0x0f0f0f0fu) | (vw[1][w] << 4 & 0xf0f0f0f0u), e01);
      cvt_e2m1x8_f16((vw[0][w] >> 4 & 0x0f0f0f0fu) | (vw[1][w] & 0xf0f0f0f0u), o01);
      cvt_e2m1x8_f16((vw[2][w] & 0x0f0f0f0fu) | (vw[3][w] << 4 & 0xf0f0f0f0u), e23);
      cvt_e2m1x8_f16((vw[2][w] >> 4 & 0x0f0f0f0fu) | (vw[3][w] & 0xf0f0f0f0u), o23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t af[4] = {hmul2_u32(e01[i], s01), hmul2_u32(o01[i], s01), hmul2_u32(e23[i], s23),
                                hmul2_u32(o23[i], s23)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(st.o[nt][4 * w + i], af, pf[nt][blk][0], pf[nt][blk][1]);
      }
    }
  }
}

// The running join of partials of one row's four neighbouring columns.
struct Joined {
  float m = -INFINITY, l = 0.0f;
  float4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  template <int N>
  __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&v)[N]) {
    float mn = m;
#pragma unroll
    for (int j = 0; j < N; ++j) mn = fmaxf(mn, ml[j].x);
    const float mu = mn == -INFINITY ? 0.0f : mn, w0 = ex2(m - mu);   // 0 from -inf
    m = mn;
    l *= w0;
    o.x *= w0;
    o.y *= w0;
    o.z *= w0;
    o.w *= w0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float w = ex2(ml[j].x - mu);
      l += w * ml[j].y;
      o.x += w * v[j].x;
      o.y += w * v[j].y;
      o.z += w * v[j].z;
      o.w += w * v[j].w;
    }
  }
};

// Where a warp's partial holds four neighbouring columns of a row: the lanes
// of a store have four pairs of rows and every fourth or second chunk, and
// would otherwise meet in two banks' worth of addresses.
__device__ __forceinline__ int warp_chunk(int row, int chunk) { return chunk ^ (row >> 1 & 3); }


}  // namespace rows
}  // namespace moe
