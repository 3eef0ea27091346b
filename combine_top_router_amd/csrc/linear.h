// Pieces shared by the kernels of the matrix product with an epilogue (internal header).
#pragma once

#include "common.h"

namespace moe {
namespace {

// The normal law's distribution function at -|z| as t P(t) e^(-z^2 / 2), t = 1 / (1 + c |z|), P of
// degree 6: fitted so that the error stays within 1.1e-5 of the value itself, far out, too (1 - erf
// would lose its last digits there), and within 0.5 of 2^-24 (rounded: 2.4).  e: the exponential.
__device__ __forceinline__ float normal_tail(float z, float& e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.3375f, 1.f));
  e = __expf(-0.5f * z * z);
  float p = fmaf(0.0427256961f, t, -0.195736752f);
  p = fmaf(fmaf(fmaf(p, t, 0.263344286f), t, -0.0292280576f), t, 0.154773731f);
  return fmaf(fmaf(p, t, 0.129138247f), t, 0.134982824f) * t * e;
}

// act: one of moe_act_kind; uniform
template <int N>
__device__ __forceinline__ void act_values(float (&v)[N], int act) {
  if (act == MOE_ACT_NONE) return;
  if (act == MOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];   // NaN stays
  } else if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = silu_f(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float e;
      const float t = normal_tail(v[i], e);
      v[i] *= v[i] < 0.f ? t : 1.f - t;
    }
  }
}
__device__ __forceinline__ void act8(float (&v)[8], int act) { act_values<8>(v, act); }

// d act'(z)
__device__ __forceinline__ void slope8(float (&d)[8], const float (&z)[8], int act) {
  if (act == MOE_ACT_NONE) return;
  if (act == MOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= z[i] > 0.f ? 1.f : z[i] == z[i] ? 0.f : z[i];
  } else if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid_f(z[i]);
      d[i] *= s * (1.f + z[i] * (1.f - s));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float e;
      const float t = normal_tail(z[i], e);
      d[i] *= (z[i] < 0.f ? t : 1.f - t) + z[i] * 0.398942280f * e;
    }
  }
}

// 16 bytes at a multiple of an element's size (the hardware takes them from anywhere)
typedef i32x4 i32x4_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_e4 __attribute__((aligned(4)));

// 8 consecutive elements as loaded, and as fp32
template <typename T> struct raw8;
template <> struct raw8<bf16_t> {
  i32x4 u;
  __device__ __forceinline__ void load(const bf16_t* p) { u = *reinterpret_cast<const i32x4_a2*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float((uint32_t)u[j] << 16);
      v[2 * j + 1] = __uint_as_float((uint32_t)u[j] & 0xffff0000u);
    }
  }
};
template <> struct raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4_e4*>(p);
    b = *reinterpret_cast<const f32x4_e4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  }
};
__device__ __forceinline__ void load8(const bf16_t* p, bf16_t (&v)[8]) {
  const i32x4 u = *reinterpret_cast<const i32x4_a2*>(p);
  __builtin_memcpy(v, &u, 16);
}
__device__ __forceinline__ void load8(const bf16_t* p, float (&v)[8]) {
  raw8<bf16_t> r;
  r.load(p);
  r.get(v);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  raw8<float> r;
  r.load(p);
  r.get(v);
}
// the first `left` of them, 0 behind
template <typename T>
__device__ __forceinline__ void load_some(const T* p, int left, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < left ? elem<T>::load(p + j) : 0.f;
}
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
  i32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = (int)pk_bf16(v[2 * j], v[2 * j + 1]);
  *reinterpret_cast<i32x4_a2*>(p) = o;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<f32x4_e4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<f32x4_e4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, int left, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) elem<T>::store(p + j, v[j]);
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
    float w[1] = {v};
    act_values<1>(w, act);
    v = w[0];
    if (add) v += elem<T>::load(add + m * N + n);
    elem<T>::store(out + m * N + n, v);
  }
};

// Which tiles, and into how many shares a product is split along K: by the estimated time.  A
// step of K takes a workgroup alone on its CU `alone` us (barrier, LDS and load latency) and r of
// them r `share` us together, and a round of workgroups `over` us (first loads, epilogue), as
// measured on one MI355X; the shares' sums cost a launch and the shares' bytes.
struct Plan {
  int shape, splits;
  int64_t ks;       // of K a share, whole steps
};
struct PlanCost {
  int tm, tn, occ;  // outputs of a tile, workgroups on a CU
  double alone, share, over;
  double join;      // of the second launch
  double bytes;     // of an output's share, at 4 TB/s
};
inline double plan_us(const PlanCost& c, int step, int cus, int64_t M, int64_t N, int64_t ks, int splits) {
  const int64_t wgs = ceil_div(M, c.tm) * ceil_div(N, c.tn) * splits, slots = (int64_t)cus * c.occ;
  auto of = [&](double r) { return r * c.share > c.alone ? r * c.share : c.alone; };
  const int64_t full = wgs / slots, rest = wgs - full * slots;
  const double r = 0.5 * ((double)rest / cus + (double)ceil_div(rest, (int64_t)cus));   // some CUs have one more
  const double steps = (double)ceil_div(ks, step);
  double us = full * (steps * of(c.occ) + c.over) + (rest > 0 ? steps * of(r) + c.over : 0.0);
  if (splits > 1) us += c.join + (double)splits * M * N * c.bytes / 4e6;
  return us;
}
inline Plan plan_product(const PlanCost* costs, int shapes, int step, int cus, int64_t M, int64_t N, int64_t K) {
  Plan best{shapes - 1, 1, ceil_div(K, step) * step};
  double least = 1e30;
  for (int i = 0; i < shapes; ++i) {
    int64_t last = -1;
    for (int s = 1; s <= 64; s += s < 16 ? 1 : s < 32 ? 8 : 16) {
      const int64_t ks = ceil_div(ceil_div(K, s), step) * step;
      const int n = ks > 0 ? (int)ceil_div(K, ks) : 1;   // shares that are not empty
      if (ks == last) continue;
      last = ks;
      const double us = plan_us(costs[i], step, cus, M, N, ks, n);
      if (us < least) {
        least = us;
        best = {i, n, ks};
      }
    }
  }
  return best;
}

}  // namespace

// gemm_linear.hip: C [M, N] = A B for bf16 matrices A and B whose rows are whole 16-byte chunks
// (zeros past the end of K in them), at multiples of 16.  A [M, K] of rows lda (a_k) or [K, M]; B [N, K] (b_k) or [K, N].
struct LinearOut {
  bf16_t* out;
  bf16_t* z;
  const bf16_t* bias;
  const bf16_t* add;
  int act;
  bool wide;   // N a multiple of 8 and every pointer at one of 16
};
size_t linear_part_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_linear_tiles(const char* name, const bf16_t* a, int64_t lda, bool a_k, const bf16_t* b, int64_t ldb,
                               bool b_k, int64_t M, int64_t N, int64_t K, const LinearOut& o, float* part,
                               hipStream_t st);
}  // namespace moe
