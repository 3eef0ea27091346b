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
// registers by 16 lanes (E <= 256; fewer for few experts) or a wave, so its softmax is one
// read; each lane keeps its columns' sums of p over the rows it sees.  Per-workgroup shares
// are added in a fixed order, in fp64 (a few adds per expert), so results do not change from
// run to run; the counts are integers, whose atomics in LDS commute.  Measured on one MI355X, forward and
// backward: 64 x 8 4.0 + 2.7 us, 4096 x 128 9.8 + 3.9 us, 16384 x 128 12.5 + 6.1 us.
#include "common.h"

namespace moe {

namespace {

typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

constexpr int BT = 256;   // threads of a workgroup of the backward

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
      v[i][j] = exp_neg(v[i][j] - m);
      s += v[i][j];
    }
  s = group_sum<LPR>(s);
  return s == 0.f ? 0.f : 1.f / s;
}

// The loss and the outputs from the sums: thread e of the workgroup holds expert e's
// (and e + blockDim's, ...) in sp and sc; n: the counted tokens
__device__ __forceinline__ void balance_out(const double* sp, const int* sc, int n, int E, int k, float coef,
                                            float* loss, int32_t* counts, float* prob, double* red) {
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
  if (threadIdx.x < 64) {
    a = threadIdx.x < (blockDim.x >> 6) ? red[threadIdx.x] : 0.0;
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) a += __shfl_xor(a, off, 64);   // at most 16 waves
    if (threadIdx.x == 0) {
      loss[0] = (float)(a * coef * E / k * inv);
      counts[E] = n;
    }
  }
}

// Sums of p and counts of this workgroup's rows into part_p[wg][E], part_c[wg][E + 1]; a
// grid of one workgroup writes the outputs itself.  Two rows are in flight at a time where
// there are that many.
constexpr int ST = 512;
template <int LPR, int NV>
__global__ __launch_bounds__(ST) void k_balance_sum(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                                                    const uint8_t* __restrict__ mask, int T, int E, int k,
                                                    float* __restrict__ part_p, int32_t* __restrict__ part_c,
                                                    float coef, float* loss, int32_t* counts, float* prob) {
  constexpr int GROUPS = ST / LPR, COLS = 4 * LPR * NV, WAVES = ST / 64;
  __shared__ float fold[WAVES][COLS];
  __shared__ int hist[COLS + 1];
  __shared__ double sp[COLS];
  __shared__ double red[WAVES];
  const int sub = threadIdx.x % LPR, group = threadIdx.x / LPR;
  for (int e = threadIdx.x; e <= E; e += ST) hist[e] = 0;
  __syncthreads();
  const bool two = (int64_t)gridDim.x * GROUPS < T;
  float acc[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  int rows = 0;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  for (int64_t t0 = (int64_t)blockIdx.x * GROUPS + group; t0 < T; t0 += 2 * step) {
    float v[2][NV][4];
    bool on[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      on[u] = false;
      if (u == 1 && !two) break;
      const int64_t t = t0 + u * step < T ? t0 + u * step : t0;
      on[u] = t0 + u * step < T && (!mask || mask[t] != 0);
      load_row<LPR, NV>(logits + (size_t)t * E, sub, E, -__builtin_inff(), v[u]);
      if (on[u])
        for (int j = sub; j < k; j += LPR) {
          const int e = idx[t * k + j];
          if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
        }
      rows += on[u];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u == 1 && !two) break;
      const float inv = softmax_row<LPR, NV>(v[u]);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += on[u] ? v[u][i][j] * inv : 0.f;   // others may hold anything
    }
  }
  if (sub == 0) atomicAdd(&hist[E], rows);
  // the wave's groups by shuffles, the waves through LDS
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int off = 32; off >= LPR; off >>= 1) acc[i][j] += __shfl_xor(acc[i][j], off, 64);
      if ((threadIdx.x & 63) < LPR) fold[threadIdx.x >> 6][4 * (sub + LPR * i) + j] = acc[i][j];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += ST) {
    double a = 0.0;
    for (int w = 0; w < WAVES; ++w) a += fold[w][e];
    if (gridDim.x == 1) sp[e] = a;
    else part_p[(size_t)blockIdx.x * E + e] = (float)a;
  }
  if (gridDim.x == 1) {
    __syncthreads();
    balance_out(sp, hist, hist[E], E, k, coef, loss, counts, prob, red);
  } else {
    for (int e = threadIdx.x; e <= E; e += ST) part_c[(size_t)blockIdx.x * (E + 1) + e] = hist[e];
  }
}

// The W workgroups' shares, added in a fixed order, and the outputs (one workgroup).  Kept
// short: such a launch waits for its loads and its cold instructions alone.
constexpr int FT = 1024;
__global__ __launch_bounds__(FT) void k_balance_out(const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                                                    int W, int E, int k, float coef, float* loss, int32_t* counts,
                                                    float* prob) {
  __shared__ double sp[FT];
  __shared__ int sc[FT + 1];
  __shared__ double red[FT / 64];
  // threads: `lanes` experts (a power of two) by FT / lanes slices of the workgroups
  int lanes = 64;
  while (lanes < E) lanes <<= 1;
  const int slices = FT / lanes, e = threadIdx.x & (lanes - 1), sl = (int)threadIdx.x / lanes;
  double a = 0.0;
  int c = 0, n = 0;
  if (sl == 0)
    for (int w = e; w < W; w += lanes) n += part_c[(size_t)w * (E + 1) + E];
  if (e < E)
#pragma unroll 8
    for (int w = sl; w < W; w += slices) {
      a += part_p[(size_t)w * E + e];
      c += part_c[(size_t)w * (E + 1) + e];
    }
  if (threadIdx.x == 0) sc[FT] = 0;
  sp[threadIdx.x] = a;
  sc[threadIdx.x] = c;
  __syncthreads();
  if (n) atomicAdd(&sc[FT], n);
  for (int h = slices >> 1; h > 0; h >>= 1) {   // slices are a power of two
    if (sl < h) {
      sp[threadIdx.x] += sp[threadIdx.x + h * lanes];
      sc[threadIdx.x] += sc[threadIdx.x + h * lanes];
    }
    __syncthreads();
  }
  if (slices == 1) __syncthreads();
  balance_out(sp, sc, sc[FT], E, k, coef, loss, counts, prob, red);
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
    if ((E) <= 16) { CALL(4, 1); }         \
    else if ((E) <= 32) { CALL(8, 1); }    \
    else if ((E) <= 64) { CALL(16, 1); }   \
    else if ((E) <= 128) { CALL(16, 2); }  \
    else if ((E) <= 256) { CALL(16, 4); }  \
    else if ((E) <= 512) { CALL(64, 2); }  \
    else { CALL(64, 4); }                  \
  } while (0)

inline int lanes_of(int E) { return E <= 16 ? 4 : E <= 32 ? 8 : E <= 256 ? 16 : 64; }

}  // namespace

// Workgroups of the forward: at most 128, whose shares the second launch reads with one
// workgroup
int balance_parts(int T, int E) {
  const int64_t w = ceil_div(T, ST / lanes_of(E));
  return (int)(w < 1 ? 1 : w > 128 ? 128 : w);
}

hipError_t launch_balance_fwd(const moe_shape& s, const float* logits, const int32_t* idx, const uint8_t* mask,
                              float coef, float* loss, int32_t* counts, float* prob, float* part_p, int32_t* part_c,
                              hipStream_t st) {
  const int W = balance_parts(s.T, s.E);
#define CALL(LPR, NV)                                                                                               \
  MOE_LAUNCH("balance_sum", (k_balance_sum<LPR, NV>), dim3((unsigned)W), dim3(ST), 0, st, logits, idx, mask, s.T, s.E, \
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
  const int64_t want = ceil_div(s.T, BT / lanes_of(s.E));
  const unsigned grid = (unsigned)(want < 1024 ? want : 1024);
#define CALL(LPR, NV)                                                                                             \
  MOE_LAUNCH("balance_bwd", (k_balance_bwd<LPR, NV>), dim3(grid), dim3(BT), 0, st, logits, counts, mask, s.T, s.E, s.k, \
             coef, d_loss, d_in, d_out)
  BALANCE_DISPATCH(s.E, CALL);
#undef CALL
  return hipGetLastError();
}

}  // namespace moe
