// Pieces shared by the kernels of the matrix product with an epilogue (internal header).
#pragma once

#include "common.h"

namespace moe {
namespace {

// 1 - sigmoid and sigmoid by the hardware reciprocal (1 ulp)
__device__ __forceinline__ float act_value(float z, int act) {
  if (act == MOE_ACT_RELU) return z < 0.f ? 0.f : z;   // NaN stays
  if (act == MOE_ACT_SILU) return silu_f(z);
  if (act == MOE_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.707106781f));
  return z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == MOE_ACT_RELU) return z > 0.f ? 1.f : z == z ? 0.f : z;
  if (act == MOE_ACT_SILU) {
    const float s = sigmoid_f(z);
    return s * (1.f + z * (1.f - s));
  }
  if (act == MOE_ACT_GELU)
    return 0.5f * (1.f + erff(z * 0.707106781f)) + z * 0.398942280f * __expf(-0.5f * z * z);
  return 1.f;
}

// What becomes of an element of a product: bias, z kept, activation, a matrix added
template <typename T>
struct Epilogue {
  T* out;
  T* z;            // or null
  const T* bias;   // or null
  const T* add;    // or null; may be out
  int act;
  __device__ __forceinline__ void store(int64_t m, int64_t n, int64_t N, float v) const {
    if (bias) v += elem<T>::load(bias + n);
    if (z) elem<T>::store(z + m * N + n, v);
    v = act_value(v, act);
    if (add) v += elem<T>::load(add + m * N + n);
    elem<T>::store(out + m * N + n, v);
  }
};

}  // namespace
}  // namespace moe
