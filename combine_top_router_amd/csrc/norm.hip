// Layer norm and root-mean-square norm in front of the MoE layer, forward and backward.
//
//   s = x + res;  layer: mu = mean(s), xh = (s - mu) rstd, rstd = 1 / sqrt(mean((s - mu)^2) + eps)
//                 rms:   mu = 0
//   y = xh w + b
//   g = dy w;  dx = ds_in + rstd (g - mean(g) [layer only] - xh mean(g xh))
//   dw = sum_t dy xh,  db = sum_t dy
//
// Both passes are bound by HBM: about ten flops an element against 8 bytes (forward with a
// residual, bf16) or 8 to 10 (backward).  So a row is read once and held in registers, as
// EPT fp32 values in each of the TPR threads that share it: the statistics are two passes
// over registers (the variance about the mean itself, not E[s^2] - mu^2, which cancels),
// and the backward keeps each thread's columns of dw and db in registers over all its rows.
#include "common.h"

namespace moe {

namespace {

// 16 bytes at an address of any element: gfx950 global loads and stores run in unaligned
// mode, so rows of an odd width take the same wide accesses as aligned ones
typedef i32x4 i32x4_a2 __attribute__((aligned(2)));
typedef i32x4 i32x4_a4 __attribute__((aligned(4)));

template <typename T> struct rowvec;
template <> struct rowvec<bf16_t> {
  static constexpr int V = 8;
  __device__ __forceinline__ static void load(const bf16_t* p, float (&v)[8]) {
    const i32x4 u = *reinterpret_cast<const i32x4_a2*>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float((uint32_t)u[q] << 16);
      v[2 * q + 1] = __uint_as_float((uint32_t)u[q] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static void store(bf16_t* p, const float (&v)[8]) {
    i32x4 u;
#pragma unroll
    for (int q = 0; q < 4; ++q) u[q] = (int)pk_bf16(v[2 * q], v[2 * q + 1]);
    *reinterpret_cast<i32x4_a2*>(p) = u;
  }
};
template <> struct rowvec<float> {
  static constexpr int V = 4;
  __device__ __forceinline__ static void load(const float* p, float (&v)[4]) {
    const i32x4 u = *reinterpret_cast<const i32x4_a4*>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = __uint_as_float((uint32_t)u[q]);
  }
  __device__ __forceinline__ static void store(float* p, const float (&v)[4]) {
    i32x4 u;
#pragma unroll
    for (int q = 0; q < 4; ++q) u[q] = (int)__float_as_uint(v[q]);
    *reinterpret_cast<i32x4_a4*>(p) = u;
  }
};

// V elements at column c of a row of H: whole vectors where they fit, element by element in
// the row's last, partial one; columns at or past H read as 0 and are not written
template <typename T>
__device__ __forceinline__ void load_cols(const T* row, int c, int H, float (&v)[rowvec<T>::V]) {
  constexpr int V = rowvec<T>::V;
  if (c + V <= H) {
    rowvec<T>::load(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = c + j < H ? elem<T>::load(row + c + j) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store_cols(T* row, int c, int H, const float (&v)[rowvec<T>::V]) {
  constexpr int V = rowvec<T>::V;
  if (c + V <= H) {
    rowvec<T>::store(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c + j < H) elem<T>::store(row + c + j, v[j]);
  }
}

// Sums of a and b over the TPR threads of a row, in every one of them.  TPR = 64 is one
// wave; larger groups are the whole workgroup and meet in red, which the caller gives anew
// (another slot) for each call between two barriers.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float (*red)[2]) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    a += __shfl_xor(a, off, 64);
    b += __shfl_xor(b, off, 64);
  }
  if constexpr (TPR > 64) {
    constexpr int NWV = TPR / 64;
    const int wv = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      red[wv][0] = a;
      red[wv][1] = b;
    }
    __syncthreads();
    a = 0.f;
    b = 0.f;
#pragma unroll
    for (int i = 0; i < NWV; ++i) {
      a += red[i][0];
      b += red[i][1];
    }
  }
}

template <int TPR>
constexpr int wg_threads() { return TPR > 64 ? TPR : 256; }

// Forward, a row in the registers of TPR threads (H <= TPR EPT).  The norm is taken of the
// fp32 sum, not of the sum rounded to the stored type: y then carries one rounding instead
// of two.
template <typename T, int TPR, int EPT, bool RMS>
__global__ __launch_bounds__(wg_threads<TPR>()) void k_norm_fwd(const T* x, const T* res,
                                                               const T* __restrict__ w, const T* __restrict__ b,
                                                               int T_, int H, float eps, T* sum, T* y, float* mean,
                                                               float* rstd) {
  constexpr int V = rowvec<T>::V, NV = EPT / V, GROUPS = wg_threads<TPR>() / TPR;
  __shared__ float red[4][TPR / 64][2];
  const int lane = threadIdx.x % TPR;
  int par = 0;   // the row's slots in red: those of the row before may still be read
  for (int64_t t = (int64_t)blockIdx.x * GROUPS + threadIdx.x / TPR; t < T_; t += (int64_t)gridDim.x * GROUPS, par ^= 2) {
    const size_t off = (size_t)t * H;
    float v[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) load_cols(x + off, (lane + i * TPR) * V, H, v[i]);
    if (res) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float r[V];
        load_cols(res + off, (lane + i * TPR) * V, H, r);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] += r[j];
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) store_cols(sum + off, (lane + i * TPR) * V, H, v[i]);
    }
    float mu = 0.f;
    if constexpr (!RMS) {
      float s = 0.f, unused = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) s += v[i][j];
      row_sum2<TPR>(s, unused, red[par]);
      mu = s / (float)H;
    }
    float q = 0.f, unused = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[i][j] -= mu;
        if ((lane + i * TPR) * V + j < H) q += v[i][j] * v[i][j];
      }
    row_sum2<TPR>(q, unused, red[par + 1]);
    const float rs = 1.f / sqrtf(q / (float)H + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * TPR) * V;
      float wv[V];
      load_cols(w, c, H, wv);
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] *= rs * wv[j];
      if (b) {
        float bv[V];
        load_cols(b, c, H, bv);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] += bv[j];
      }
      store_cols(y + off, c, H, v[i]);
    }
    if (lane == 0) {
      if constexpr (!RMS) mean[t] = mu;
      rstd[t] = rs;
    }
  }
}

// Forward for rows past the registers of a workgroup: the row is read again (from the L2)
// for each pass over it.
constexpr int LONG_T = 1024;
template <typename T, bool RMS>
__global__ __launch_bounds__(LONG_T) void k_norm_fwd_long(const T* x, const T* res,
                                                          const T* __restrict__ w, const T* __restrict__ b, int T_,
                                                          int H, float eps, T* sum, T* y, float* mean, float* rstd) {
  constexpr int V = rowvec<T>::V;
  __shared__ float red[4][LONG_T / 64][2];
  int par = 0;
  for (int64_t t = blockIdx.x; t < T_; t += gridDim.x, par ^= 2) {
    const size_t off = (size_t)t * H;
    auto row = [&](int c, float (&v)[V]) {
      load_cols(x + off, c, H, v);
      if (res) {
        float r[V];
        load_cols(res + off, c, H, r);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += r[j];
      }
    };
    float mu = 0.f, unused = 0.f;
    if constexpr (!RMS) {
      float s = 0.f;
      for (int c = threadIdx.x * V; c < H; c += LONG_T * V) {
        float v[V];
        row(c, v);
#pragma unroll
        for (int j = 0; j < V; ++j) s += v[j];
      }
      row_sum2<LONG_T>(s, unused, red[par]);
      mu = s / (float)H;
    }
    float q = 0.f;
    unused = 0.f;
    for (int c = threadIdx.x * V; c < H; c += LONG_T * V) {
      float v[V];
      row(c, v);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c + j < H) q += (v[j] - mu) * (v[j] - mu);
    }
    row_sum2<LONG_T>(q, unused, red[par + 1]);
    const float rs = 1.f / sqrtf(q / (float)H + eps);
    for (int c = threadIdx.x * V; c < H; c += LONG_T * V) {
      float v[V], wv[V];
      row(c, v);
      if (res) store_cols(sum + off, c, H, v);
      load_cols(w, c, H, wv);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = (v[j] - mu) * (rs * wv[j]);
      if (b) {
        float bv[V];
        load_cols(b, c, H, bv);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += bv[j];
      }
      store_cols(y + off, c, H, v);
    }
    if (threadIdx.x == 0) {
      if constexpr (!RMS) mean[t] = mu;
      rstd[t] = rs;
    }
  }
}

// Backward, rows in registers: workgroup g takes rows g, g + gridDim.x, ... (times the rows
// it holds at once) and leaves its share of dw and db in part[g] and part[G + g].
template <typename T, int TPR, int EPT, bool RMS, bool HAS_B>
__global__ __launch_bounds__(wg_threads<TPR>()) void k_norm_bwd(const T* __restrict__ dy, const T* __restrict__ s,
                                                               const T* __restrict__ res, const T* __restrict__ w,
                                                               const float* __restrict__ mean,
                                                               const float* __restrict__ rstd, const T* ds_in, int T_,
                                                               int H, T* dx, float* __restrict__ part) {
  constexpr int V = rowvec<T>::V, NV = EPT / V, GROUPS = wg_threads<TPR>() / TPR;
  __shared__ float red[2][TPR / 64][2];
  __shared__ float fold[GROUPS > 1 ? GROUPS * TPR * EPT : 1];
  const int group = (int)threadIdx.x / TPR, lane = threadIdx.x % TPR;
  float wv[NV][V], dwa[NV][V], dba[HAS_B ? NV : 1][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_cols(w, (lane + i * TPR) * V, H, wv[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      dwa[i][j] = 0.f;
      if (HAS_B) dba[i][j] = 0.f;
    }
  }
  const float inv_h = 1.f / (float)H;
  int par = 0;
  for (int64_t t = (int64_t)blockIdx.x * GROUPS + group; t < T_; t += (int64_t)gridDim.x * GROUPS, par ^= 1) {
    const size_t off = (size_t)t * H;
    float xh[NV][V], g[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_cols(s + off, (lane + i * TPR) * V, H, xh[i]);
      load_cols(dy + off, (lane + i * TPR) * V, H, g[i]);
    }
    const float mu = RMS ? 0.f : mean[t], rs = rstd[t];
    if (res) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float r[V];
        load_cols(res + off, (lane + i * TPR) * V, H, r);
#pragma unroll
        for (int j = 0; j < V; ++j) xh[i][j] += r[j];
      }
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {   // columns at or past H hold dy = 0
        xh[i][j] = (xh[i][j] - mu) * rs;
        dwa[i][j] += g[i][j] * xh[i][j];
        if (HAS_B) dba[i][j] += g[i][j];
        g[i][j] *= wv[i][j];
        s1 += g[i][j];
        s2 += g[i][j] * xh[i][j];
      }
    row_sum2<TPR>(s1, s2, red[par]);
    s1 = RMS ? 0.f : s1 * inv_h;
    s2 *= inv_h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * TPR) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) g[i][j] = rs * (g[i][j] - s1 - xh[i][j] * s2);
      if (ds_in) {
        float d[V];
        load_cols(ds_in + off, c, H, d);
#pragma unroll
        for (int j = 0; j < V; ++j) g[i][j] += d[j];
      }
      store_cols(dx + off, c, H, g[i]);
    }
  }
  // the row groups' shares, added in group order
  auto leave = [&](float (&a)[NV][V], float* out) {
    if constexpr (GROUPS > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) fold[((group * NV + i) * V + j) * TPR + lane] = a[i][j];
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j)
            for (int o = 1; o < GROUPS; ++o) a[i][j] += fold[((o * NV + i) * V + j) * TPR + lane];
      }
    }
    if (group == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < V; q += 4)
          store_cols<float>(out, (lane + i * TPR) * V + q, H, *reinterpret_cast<float(*)[4]>(&a[i][q]));
    }
  };
  leave(dwa, part + (size_t)blockIdx.x * H);
  if constexpr (HAS_B) leave(dba, part + ((size_t)gridDim.x + blockIdx.x) * H);
}

// Backward of the long rows: dx row by row, then dw and db column by column over slices of
// the rows.
template <typename T, bool RMS>
__global__ __launch_bounds__(LONG_T) void k_norm_dx_long(const T* __restrict__ dy, const T* __restrict__ s,
                                                         const T* __restrict__ res, const T* __restrict__ w, const float* __restrict__ mean,
                                                         const float* __restrict__ rstd, const T* ds_in, int T_, int H,
                                                         T* dx) {
  constexpr int V = rowvec<T>::V;
  __shared__ float red[2][LONG_T / 64][2];
  int par = 0;
  for (int64_t t = blockIdx.x; t < T_; t += gridDim.x, par ^= 1) {
    const size_t off = (size_t)t * H;
    const float mu = RMS ? 0.f : mean[t], rs = rstd[t];
    auto row = [&](int c, float (&v)[V]) {
      load_cols(s + off, c, H, v);
      if (res) {
        float r[V];
        load_cols(res + off, c, H, r);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += r[j];
      }
    };
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x * V; c < H; c += LONG_T * V) {
      float xv[V], g[V], wv[V];
      row(c, xv);
      load_cols(dy + off, c, H, g);
      load_cols(w, c, H, wv);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        g[j] *= wv[j];
        s1 += g[j];
        s2 += g[j] * ((xv[j] - mu) * rs);
      }
    }
    row_sum2<LONG_T>(s1, s2, red[par]);
    s1 = RMS ? 0.f : s1 / (float)H;
    s2 /= (float)H;
    for (int c = threadIdx.x * V; c < H; c += LONG_T * V) {
      float xv[V], g[V], wv[V];
      row(c, xv);
      load_cols(dy + off, c, H, g);
      load_cols(w, c, H, wv);
#pragma unroll
      for (int j = 0; j < V; ++j) g[j] = rs * (g[j] * wv[j] - s1 - (xv[j] - mu) * rs * s2);
      if (ds_in) {
        float d[V];
        load_cols(ds_in + off, c, H, d);
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] += d[j];
      }
      store_cols(dx + off, c, H, g);
    }
  }
}

template <typename T, bool RMS>
__global__ __launch_bounds__(256) void k_norm_dw_long(const T* __restrict__ dy, const T* __restrict__ s,
                                                      const T* __restrict__ res,
                                                      const float* __restrict__ mean, const float* __restrict__ rstd,
                                                      int T_, int H, float* __restrict__ part, int has_b) {
  const int c = (int)blockIdx.x * 256 + (int)threadIdx.x;
  if (c >= H) return;
  float a = 0.f, d = 0.f;
  for (int64_t t = blockIdx.y; t < T_; t += gridDim.y) {
    const float g = elem<T>::load(dy + (size_t)t * H + c);
    const float v = elem<T>::load(s + (size_t)t * H + c) + (res ? elem<T>::load(res + (size_t)t * H + c) : 0.f);
    a += g * ((v - (RMS ? 0.f : mean[t])) * rstd[t]);
    d += g;
  }
  part[(size_t)blockIdx.y * H + c] = a;
  if (has_b) part[((size_t)gridDim.y + blockIdx.y) * H + c] = d;
}

// dw (and db, blockIdx.y = 1): the G shares added in a fixed order, rounded once
constexpr int FOLD_COLS = 64, FOLD_GROUPS = 16;
template <typename T>
__global__ __launch_bounds__(FOLD_COLS* FOLD_GROUPS) void k_norm_fold(const float* __restrict__ part, int G, int H,
                                                                     T* __restrict__ dw, T* __restrict__ db) {
  __shared__ float sh[FOLD_GROUPS][FOLD_COLS];
  const int cl = threadIdx.x % FOLD_COLS, gr = threadIdx.x / FOLD_COLS;
  const int c = (int)blockIdx.x * FOLD_COLS + cl;
  const float* p = part + (size_t)blockIdx.y * G * H;
  float a = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int g = gr; g < G; g += FOLD_GROUPS) a += p[(size_t)g * H + c];
  }
  sh[gr][cl] = a;
  __syncthreads();
  if (gr == 0 && c < H) {
    for (int o = 1; o < FOLD_GROUPS; ++o) a += sh[o][cl];
    elem<T>::store((blockIdx.y ? db : dw) + c, a);
  }
}

constexpr int NORM_REG_COLS = 16384;   // the widest row held in registers
// one workgroup a row (or four rows), as far as a grid goes; the kernels loop over the rest
inline unsigned row_grid(int64_t wgs) { return (unsigned)(wgs < (1 << 20) ? wgs : (1 << 20)); }

}  // namespace

// Shares of dw: workgroups of the backward, or row slices of the long rows.  1024 (512 of
// four times the threads): at 16384 x 4096 bf16 with a residual 256 / 512 / 1024 / 2048 take
// 320 / 198 / 136 / 145 us, too few rows in flight on one side and more shares than rows are
// worth on the other.
int norm_parts(const moe_norm_shape& s) {
  if (s.T == 0) return 0;
  const int rows = s.H <= 1024 ? 4 : 1;   // rows a workgroup holds at once
  const int64_t most = s.H > NORM_REG_COLS ? 16 : s.H > 4096 ? 512 : 1024;
  const int64_t g = ceil_div(s.T, rows);
  return (int)(g < most ? g : most);
}

// Threads and registers of a row: 16 values a thread at most, so that the backward's rows,
// weights and two sums (5 x 16) fit without spilling; one wave up to 1024 columns, then 256
// threads to 4096 and 1024 threads to 16384.  32 values in fewer threads, with fewer barriers,
// lose: 16384 x 4096 with 128 threads takes 109 us forward and 195 backward, against 95 and
// 136.  The forward holds less and takes 512 threads from 2048 to 4096 columns: 95 us against
// 100 with 256.
#define NORM_BWD_DISPATCH(H, CALL)             \
  do {                                         \
    if ((H) <= 512) { CALL(64, 8); }           \
    else if ((H) <= 1024) { CALL(64, 16); }    \
    else if ((H) <= 2048) { CALL(256, 8); }    \
    else if ((H) <= 4096) { CALL(256, 16); }   \
    else if ((H) <= 8192) { CALL(1024, 8); }   \
    else { CALL(1024, 16); }                   \
  } while (0)
#define NORM_FWD_DISPATCH(H, CALL)             \
  do {                                         \
    if ((H) <= 512) { CALL(64, 8); }           \
    else if ((H) <= 1024) { CALL(64, 16); }    \
    else if ((H) <= 2048) { CALL(256, 8); }    \
    else if ((H) <= 4096) { CALL(512, 8); }    \
    else if ((H) <= 8192) { CALL(1024, 8); }   \
    else { CALL(1024, 16); }                   \
  } while (0)

template <typename T, bool RMS>
static hipError_t norm_fwd(const moe_norm_shape& s, const void* x_, const void* res_, const void* w_, const void* b_,
                           void* sum_, void* y_, float* mean, float* rstd, hipStream_t st) {
  const T *x = (const T*)x_, *res = (const T*)res_, *w = (const T*)w_, *b = (const T*)b_;
  T *sum = (T*)sum_, *y = (T*)y_;
  if (s.H > NORM_REG_COLS) {
    MOE_LAUNCH("norm_fwd", (k_norm_fwd_long<T, RMS>), dim3(row_grid(s.T)), dim3(LONG_T), 0, st, x, res, w, b, s.T,
               s.H, s.eps, sum, y, mean, rstd);
    return hipGetLastError();
  }
#define CALL(TPR, EPT)                                                                                          \
  MOE_LAUNCH("norm_fwd", (k_norm_fwd<T, TPR, EPT, RMS>), dim3(row_grid(ceil_div(s.T, wg_threads<TPR>() / TPR))), \
             dim3(wg_threads<TPR>()), 0, st, x, res, w, b, s.T, s.H, s.eps, sum, y, mean, rstd)
  NORM_FWD_DISPATCH(s.H, CALL);
#undef CALL
  return hipGetLastError();
}

template <typename T, bool RMS, bool HAS_B>
static hipError_t norm_bwd(const moe_norm_shape& s, const void* dy_, const void* sum_, const void* res_,
                           const void* w_, const float* mean, const float* rstd, const void* ds_in_, void* dx_,
                           void* dw, void* db, float* part, hipStream_t st) {
  const T *dy = (const T*)dy_, *sum = (const T*)sum_, *res = (const T*)res_, *w = (const T*)w_, *ds_in = (const T*)ds_in_;
  T* dx = (T*)dx_;
  const int G = norm_parts(s);
  if (s.T > 0 && s.H > NORM_REG_COLS) {
    MOE_LAUNCH("norm_dx", (k_norm_dx_long<T, RMS>), dim3(row_grid(s.T)), dim3(LONG_T), 0, st, dy, sum, res, w, mean,
               rstd, ds_in, s.T, s.H, dx);
    MOE_LAUNCH("norm_dw", (k_norm_dw_long<T, RMS>), dim3((unsigned)ceil_div(s.H, 256), (unsigned)G), dim3(256), 0, st,
               dy, sum, res, mean, rstd, s.T, s.H, part, HAS_B);
  } else if (s.T > 0) {
#define CALL(TPR, EPT)                                                                                              \
  MOE_LAUNCH("norm_bwd", (k_norm_bwd<T, TPR, EPT, RMS, HAS_B>), dim3((unsigned)G), dim3(wg_threads<TPR>()), 0, st, dy, \
             sum, res, w, mean, rstd, ds_in, s.T, s.H, dx, part)
    NORM_BWD_DISPATCH(s.H, CALL);
#undef CALL
  }
  MOE_LAUNCH("norm_fold", k_norm_fold<T>, dim3((unsigned)ceil_div(s.H, FOLD_COLS), HAS_B ? 2u : 1u),
             dim3(FOLD_COLS * FOLD_GROUPS), 0, st, part, G, s.H, (T*)dw, (T*)db);
  return hipGetLastError();
}

hipError_t launch_norm_fwd(const moe_norm_shape& s, const void* x, const void* res, const void* w, const void* b,
                           void* sum, void* y, float* mean, float* rstd, hipStream_t st) {
  const bool rms = s.kind == MOE_NORM_RMS;
  if (s.dtype == MOE_BF16)
    return rms ? norm_fwd<bf16_t, true>(s, x, res, w, b, sum, y, mean, rstd, st)
               : norm_fwd<bf16_t, false>(s, x, res, w, b, sum, y, mean, rstd, st);
  return rms ? norm_fwd<float, true>(s, x, res, w, b, sum, y, mean, rstd, st)
             : norm_fwd<float, false>(s, x, res, w, b, sum, y, mean, rstd, st);
}

template <typename T, bool RMS, class... A>
static hipError_t norm_bwd_b(bool has_b, A... a) {
  return has_b ? norm_bwd<T, RMS, true>(a...) : norm_bwd<T, RMS, false>(a...);
}
hipError_t launch_norm_bwd(const moe_norm_shape& s, const void* dy, const void* sum, const void* res, const void* w,
                           const float* mean, const float* rstd, const void* ds_in, void* dx, void* dw, void* db,
                           float* part, hipStream_t st) {
  const bool rms = s.kind == MOE_NORM_RMS, b = db != nullptr;
  if (s.dtype == MOE_BF16)
    return rms ? norm_bwd_b<bf16_t, true>(b, s, dy, sum, res, w, mean, rstd, ds_in, dx, dw, db, part, st)
               : norm_bwd_b<bf16_t, false>(b, s, dy, sum, res, w, mean, rstd, ds_in, dx, dw, db, part, st);
  return rms ? norm_bwd_b<float, true>(b, s, dy, sum, res, w, mean, rstd, ds_in, dx, dw, db, part, st)
             : norm_bwd_b<float, false>(b, s, dy, sum, res, w, mean, rstd, ds_in, dx, dw, db, part, st);
}

}  // namespace moe
