// Rows of a few hundred fp32 values held by a group of lanes: loads, sums and the softmax's
// exponential, shared by the kernels that work on the router's logits (internal header).
#pragma once

#include "common.h"

namespace moe {
namespace {

typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// columns 4 (sub + LPR i) .. + 3 of the row, columns at or past E as fill
template <int LPR, int NV>
__device__ __forceinline__ void load_row(const float* row, int sub, int E, float fill, float (&v)[NV][4]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 4 * (sub + LPR * i);
    if (e + 4 <= E) {
      const f32x4 u = *reinterpret_cast<const f32x4_a4*>(row + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = u[j];
    } else {   // the row's end: three loads at clamped columns, issued before one is looked at
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = fill;
      if (e < E) {
        float u[3];
#pragma unroll
        for (int j = 0; j < 3; ++j) u[j] = row[min(e + j, E - 1)];
#pragma unroll
        for (int j = 0; j < 3; ++j) v[i][j] = e + j < E ? u[j] : fill;
      }
    }
  }
}

// exp(d), d <= 0 or NaN: 2^(d log2 e) with the product's rounding error put back (log2 e as
// a pair; 2^r = 1 + r ln 2 to first order, |r| < 2^-16 before 2^h leaves fp32's range)
__device__ __forceinline__ float exp_neg(float d) {
  constexpr float L2E = 1.44269502f, L2E_LO = 1.92596302e-8f, LN2 = 0.693147182f;
  const float h = d * L2E;
  const float r = fmaf(d, L2E_LO, fmaf(d, L2E, -h));
  const float p = __builtin_amdgcn_exp2f(h);
  return d < -104.f ? 0.f : fmaf(p, r * LN2, p);   // below 2^-150; -inf has no r
}

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

}  // namespace
}  // namespace moe
