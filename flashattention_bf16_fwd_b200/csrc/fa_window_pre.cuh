// fa_window_pre.cuh - the windowed backward's first kernel: D_i and a zeroed FP32
// dQ accumulator, as fa_bwd_pre_kernel, with a D of its own for rows that see few
// keys.
#pragma once

#include "sm100.cuh"

namespace fa {

// D_i = sum_k dO_ik O_ik, from the O that the forward rounded, is off by up to
// half a step of every O_ik.  That is the larger part of the error of dS = P
// (dP - D) where a row sees few keys, for O does not average over many and dP - D
// is small; a row that sees one key has dS = 0.  So rows of up to kFewKeys keys
// take D_i = sum_j P_ij dP_ij from their own scores:
//   D_i = sum_j e_j (dO_i.V_j) / sum_j e_j,  e_j = exp(scale Q_i.K_j - LSE_i).
// These are the first tokens of every sequence, and all where window + sinks is
// that small.  (Relative error of dq and dk, 365 bf16 sequences of 1 to 300 tokens:
// 35 above 5e-3 and up to 3.6e-2 by the first formula, 4.1e-3 at most by this one;
// that of B=1 H=12 N=1024 d=64, window 256, falls from 2.77e-3 to 2.67e-3 only, for
// there O's rounding counts for less than that of dS.)
constexpr int kFewKeys = 8;

struct BwdPreParams {
  const float* lse;
  float* dsum;           // [BH, N]
  float* dq_acc;         // [BH, N, D], or nullptr where nothing is added to it
  long long rows;        // BH * N
  int N, H, group, window, sinks;
  int few;               // a row i sees min(i + 1, window + sinks) keys: the first `few` of each head see few
  unsigned few_blocks;   // the first blocks take those, a warp per row
  float scale_log2;
};

// The dot product of two rows' slices of 8 W elements.
template <typename E, int W>
__device__ __forceinline__ float slice_dot(const uint4 (&x)[W], const uint4 (&y)[W]) {
  float acc = 0.f;
#pragma unroll
  for (int c = 0; c < W; ++c) {
    const uint32_t* a = reinterpret_cast<const uint32_t*>(&x[c]);
    const uint32_t* b = reinterpret_cast<const uint32_t*>(&y[c]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 fa = E::unpack(a[i]), fb = E::unpack(b[i]);
      acc = fmaf(fa.x, fb.x, acc);
      acc = fmaf(fa.y, fb.y, acc);
    }
  }
  return acc;
}

// HBM-bound over the rows, eight threads each.  A row of few keys has a warp, four
// lanes per key, so that all its loads are in flight at once and the kernel's tail
// is no longer than the other blocks' (eight threads per row for these too, four
// keys at a time: 3 us more for the smallest calls, 6 us for 8 x 12 heads of 1024
// tokens; so 0.5 and 2 us).
template <int D, typename E>
__global__ void __launch_bounds__(256) fa_bwd_window_pre_kernel(const typename E::T* __restrict__ o,
                                                                const typename E::T* __restrict__ dout,
                                                                const typename E::T* __restrict__ q,
                                                                const typename E::T* __restrict__ k,
                                                                const typename E::T* __restrict__ v,
                                                                const BwdPreParams p) {
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x < p.few_blocks) {
    constexpr int kPart = D / 4, kWords = kPart / 8;
    static_assert(kFewKeys * 4 == 32, "a warp is not a row");
    const int lane = int(lane_id()), t = lane >> 2, at = (lane & 3) * kPart;
    const long long r = (long long)blockIdx.x * 8 + warp_id();
    const int bh = int(r / p.few), i = int(r % p.few);
    if (bh >= int(p.rows / p.N)) return;
    const int hidden = max(0, i + 1 - p.window), sk = min(p.sinks, hidden);   // keys before the window; sinks there
    const bool seen = t < sk + i + 1 - hidden;
    const int j = !seen ? i : t < sk ? t : hidden + t - sk;
    const int kv_bh = (bh / p.H) * (p.H / p.group) + (bh % p.H) / p.group;
    const size_t row = size_t(bh) * p.N + i, key = size_t(kv_bh) * p.N + j;
    uint4 qd[kWords], kd[kWords], vd[kWords], dd[kWords];
#pragma unroll
    for (int c = 0; c < kWords; ++c) {
      qd[c] = reinterpret_cast<const uint4*>(q + row * D + at)[c];
      kd[c] = reinterpret_cast<const uint4*>(k + key * D + at)[c];
      vd[c] = reinterpret_cast<const uint4*>(v + key * D + at)[c];
      dd[c] = reinterpret_cast<const uint4*>(dout + row * D + at)[c];
    }
    const float shift = p.lse[row] * 1.4426950408889634f;
    float s = slice_dot<E>(qd, kd), dp = slice_dot<E>(dd, vd);
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, x);
      dp += __shfl_xor_sync(0xffffffffu, dp, x);
    }
    float e = seen ? ex2(fmaf(s, p.scale_log2, -shift)) : 0.f;
    float top = seen ? e * dp : 0.f;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      e += __shfl_xor_sync(0xffffffffu, e, x);
      top += __shfl_xor_sync(0xffffffffu, top, x);
    }
    if (lane == 0) p.dsum[row] = top / e;
    return;
  }
  constexpr int kPer = D / 8, kWords = kPer / 8;
  const long long tid = (long long)(blockIdx.x - p.few_blocks) * blockDim.x + threadIdx.x;
  const long long row = tid >> 3;
  float sum = 0.f;
  if (row < p.rows) {
    const size_t base = size_t(row) * D + size_t(tid & 7) * kPer;
    uint4 od[kWords], dd[kWords];
    float4* z = reinterpret_cast<float4*>(p.dq_acc + base);
#pragma unroll
    for (int c = 0; c < kWords; ++c) {
      od[c] = reinterpret_cast<const uint4*>(o + base)[c];
      dd[c] = reinterpret_cast<const uint4*>(dout + base)[c];
      if (p.dq_acc) z[2 * c] = z[2 * c + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    sum = slice_dot<E>(od, dd);
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  sum += __shfl_xor_sync(0xffffffffu, sum, 4);
  if (row < p.rows && (tid & 7) == 0 && int(unsigned(row) % unsigned(p.N)) >= p.few) p.dsum[row] = sum;
}

}  // namespace fa
