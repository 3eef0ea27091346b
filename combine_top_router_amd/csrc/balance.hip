// The router's load-balance loss with the per-expert counts, forward and backward.
//
// Over the N tokens that count (mask != 0, or all), with p_t = softmax(logits[t]),
// c_e the number of their slots that chose expert e and P_e the mean of p_te:
//   loss = coef E / (k N) sum_e c_e P_e
//   d_logits[t, j] = d_in[t, j] + d_loss coef E / (k N^2) p_tj (c_j - sum_e c_e p_te)
// The counts are piecewise constant and carry no gradient.
//
// Bound: the forward reads the logits once and the backward reads them once more beside
// d_in and writes d_logits, 12 bytes an entry in all; at a layer's sizes (2 to 8 MB of
// logits) they sit in the caches and the launches are what counts.  A row is held in
// registers by 16 lanes (E <= 256) or a wave, so its softmax is one read; each lane keeps
// its columns' sums of p over the rows it sees.  Per-workgroup shares are added in a fixed
// order, in fp64 (a few adds per expert), so results do not change from run to run; the
// counts are integers, whose atomics in LDS commute.
#include "common.h"

namespace moe {

namespace {

typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

constexpr int BT = 256;   // threads of a workgroup

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
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = e + j < E ? row[e + j] : fill;
    }
  }
}

template <int LPR>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// v -> exp(v - max), and 1 / their sum (0 for a row of -inf alone: it has no probabilities).
// A NaN or +inf logit makes its whole row NaN.
template <int LPR, int NV>
__device__ __forceinline__ float softmax_row(float (&v)[NV][4]) {
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, v[i][j]);
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if (m == -__builtin_inff()) m = 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[i][j] = expf(v[i][j] - m);
      s += v[i][j];
    }
  s = group_sum<LPR>(s);
  return s == 0.f ? 0.f : 1.f / s;
}

// The loss and the outputs from the sums: thread e of the workgroup holds expert e's
// (and e + BT's, ...) in sp and sc, the counted tokens in sc[E]
__device__ __forceinline__ void balance_out(const double* sp, const int* sc, int E, int k, float coef, float* loss,
                                            int32_t* counts, float* prob, double* red) {
  const int n = sc[E];
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double a = 0.0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const double p = sp[e] * inv;
    prob[e] = (float)p;
    counts[e] = sc[e];
    a += p * sc[e];
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) a += __shfl_xor(a, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < (int)(blockDim.x >> 6); ++i) a += red[i];
    loss[0] = (float)(a * coef * E / k * inv);
    counts[E] = n;
  }
}

// Sums of p and counts of this workgroup's rows into part_p[wg][E], part_c[wg][E + 1]; a
// grid of one workgroup writes the outputs itself.
template <int LPR, int NV>
__global__ __launch_bounds__(BT) void k_balance_sum(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                                                    const uint8_t* __restrict__ mask, int T, int E, int k,
                                                    float* __restrict__ part_p, int32_t* __restrict__ part_c,
                                                    float coef, float* loss, int32_t* counts, float* prob) {
  constexpr int GROUPS = BT / LPR, COLS = 4 * LPR * NV;
  __shared__ float fold[GROUPS][COLS];
  __shared__ int hist[COLS + 1];
  __shared__ double sp[COLS];
  __shared__ double red[BT / 64];
  const int sub = threadIdx.x % LPR, group = threadIdx.x / LPR;
  for (int e = threadIdx.x; e <= E; e += BT) hist[e] = 0;
  __syncthreads();
  float acc[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  int rows = 0;
  for (int64_t t = (int64_t)blockIdx.x * GROUPS + group; t < T; t += (int64_t)gridDim.x * GROUPS) {
    if (mask && mask[t] == 0) continue;   // not read: its logits may hold anything
    ++rows;
    if (sub < k) {
      const int e = idx[t * k + sub];
      if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
    }
    float v[NV][4];
    load_row<LPR, NV>(logits + (size_t)t * E, sub, E, -__builtin_inff(), v);
    const float inv = softmax_row<LPR, NV>(v);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] += v[i][j] * inv;
  }
  if (sub == 0) atomicAdd(&hist[E], rows);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) fold[group][4 * (sub + LPR * i) + j] = acc[i][j];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += BT) {
    double a = 0.0;
    for (int g = 0; g < GROUPS; ++g) a += fold[g][e];
    if (gridDim.x == 1) sp[e] = a;
    else part_p[(size_t)blockIdx.x * E + e] = (float)a;
  }
  if (gridDim.x == 1) {
    __syncthreads();
    balance_out(sp, hist, E, k, coef, loss, counts, prob, red);
  } else {
    for (int e = threadIdx.x; e <= E; e += BT) part_c[(size_t)blockIdx.x * (E + 1) + e] = hist[e];
  }
}

// The W workgroups' shares, added in a fixed order, and the outputs (one workgroup)
constexpr int FT = 1024;
__global__ __launch_bounds__(FT) void k_balance_out(const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                                                    int W, int E, int k, float coef, float* loss, int32_t* counts,
                                                    float* prob) {
  __shared__ double sp[1024];
  __shared__ int sc[1025];
  __shared__ double red[FT / 64];
  __shared__ double fp[FT];
  __shared__ int fc[FT];
  // threads: `lanes` experts (a power of two) by FT / lanes slices of the workgroups
  int lanes = 64;
  while (lanes < E && lanes < FT) lanes <<= 1;
  const int slices = FT / lanes, e = threadIdx.x % lanes, sl = threadIdx.x / lanes;
  double a = 0.0;
  int c = 0;
  if (e < E)
#pragma unroll 4
    for (int w = sl; w < W; w += slices) {
      a += part_p[(size_t)w * E + e];
      c += part_c[(size_t)w * (E + 1) + e];
    }
  fp[threadIdx.x] = a;
  fc[threadIdx.x] = c;
  if (threadIdx.x == 0) sc[E] = 0;
  __syncthreads();
  if (sl == 0 && e < E) {
    for (int o = 1; o < slices; ++o) {
      a += fp[o * lanes + e];
      c += fc[o * lanes + e];
    }
    sp[e] = a;
    sc[e] = c;
  }
  for (int w = threadIdx.x; w < W; w += FT) atomicAdd(&sc[E], part_c[(size_t)w * (E + 1) + E]);
  __syncthreads();
  balance_out(sp, sc, E, k, coef, loss, counts, prob, red);
}

// d_in may be d_logits: a lane reads its entries before it writes them.
template <int LPR, int NV>
__global__ __launch_bounds__(BT) void k_balance_bwd(const float* __restrict__ logits,
                                                    const int32_t* __restrict__ counts,
                                                    const uint8_t* __restrict__ mask, int T, int E, int k, float coef,
                                                    const float* __restrict__ d_loss, const float* d_in, float* d_out) {
  constexpr int GROUPS = BT / LPR;
  const int sub = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int n = counts[E];
  // counts about their mean k N / E: the probabilities of a row sum to 1, so the constant
  // drops out of c_j - sum c p, and what is left keeps its digits when the load is balanced
  const double mid = (double)k * n / E;
  const float scale =
      n > 0 ? (float)((double)(d_loss ? d_loss[0] : 1.f) * coef * E / k / ((double)n * (double)n)) : 0.f;
  float c[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * (sub + LPR * i) + j;
      c[i][j] = e < E ? (float)(counts[e] - mid) : 0.f;
    }
  for (int64_t t = (int64_t)blockIdx.x * GROUPS + group; t < T; t += (int64_t)gridDim.x * GROUPS) {
    float v[NV][4], d[NV][4];
    if (d_in) {
      load_row<LPR, NV>(d_in + (size_t)t * E, sub, E, 0.f, d);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[i][j] = 0.f;
    }
    if (!mask || mask[t] != 0) {
      load_row<LPR, NV>(logits + (size_t)t * E, sub, E, -__builtin_inff(), v);
      const float inv = softmax_row<LPR, NV>(v);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][j] *= inv;
          s += v[i][j] * c[i][j];
        }
      s = group_sum<LPR>(s);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[i][j] += scale * (v[i][j] * (c[i][j] - s));
    }
    float* row = d_out + (size_t)t * E;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 4 * (sub + LPR * i);
      if (e + 4 <= E) {
        f32x4 u;
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = d[i][j];
        *reinterpret_cast<f32x4_a4*>(row + e) = u;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e + j < E) row[e + j] = d[i][j];
      }
    }
  }
}

// lanes of a row and vectors of four columns a lane
#define BALANCE_DISPATCH(E, CALL)          \
  do {                                     \
    if ((E) <= 64) { CALL(16, 1); }        \
    else if ((E) <= 128) { CALL(16, 2); }  \
    else if ((E) <= 256) { CALL(16, 4); }  \
    else if ((E) <= 512) { CALL(64, 2); }  \
    else { CALL(64, 4); }                  \
  } while (0)

inline int rows_per_wg(int E) { return E <= 256 ? 16 : 4; }

}  // namespace

// Workgroups of the forward: four rows of each lane group, at most 128 (the second launch
// reads all their shares with one workgroup)
int balance_parts(int T, int E) {
  const int64_t w = ceil_div(T, 4 * rows_per_wg(E));
  return (int)(w < 1 ? 1 : w > 128 ? 128 : w);
}

hipError_t launch_balance_fwd(const moe_shape& s, const float* logits, const int32_t* idx, const uint8_t* mask,
                              float coef, float* loss, int32_t* counts, float* prob, float* part_p, int32_t* part_c,
                              hipStream_t st) {
  const int W = balance_parts(s.T, s.E);
#define CALL(LPR, NV)                                                                                               \
  MOE_LAUNCH("balance_sum", (k_balance_sum<LPR, NV>), dim3((unsigned)W), dim3(BT), 0, st, logits, idx, mask, s.T, s.E, \
             s.k, part_p, part_c, coef, loss, counts, prob)
  BALANCE_DISPATCH(s.E, CALL);
#undef CALL
  if (W > 1)
    MOE_LAUNCH("balance_out", k_balance_out, dim3(1), dim3(FT), 0, st, part_p, part_c, W, s.E, s.k, coef, loss, counts,
               prob);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const moe_shape& s, const float* logits, const int32_t* counts, const uint8_t* mask,
                              float coef, const float* d_loss, const float* d_in, float* d_out, hipStream_t st) {
  const int64_t want = ceil_div(s.T, rows_per_wg(s.E));
  const unsigned grid = (unsigned)(want < 1024 ? want : 1024);
#define CALL(LPR, NV)                                                                                             \
  MOE_LAUNCH("balance_bwd", (k_balance_bwd<LPR, NV>), dim3(grid), dim3(BT), 0, st, logits, counts, mask, s.T, s.E, s.k, \
             coef, d_loss, d_in, d_out)
  BALANCE_DISPATCH(s.E, CALL);
#undef CALL
  return hipGetLastError();
}

}  // namespace moe
