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
// EPT fp32 values in each of the threads that share it: the statistics are two passes
// over registers (the variance about the mean itself, not E[s^2] - mu^2, which cancels),
// and the backward keeps each thread's columns of dw and db in registers over all its rows.
// Measured on one MI355X, in a graph: 16384 x 4096 bf16 with a residual forward 94 us for 537 MB,
// backward 134 us for 671 MB (x, res, dy, ds_in, dx), 5.7 and 5.0 TB/s beside the 5.1 TB/s of a
// large copy, the same over four sets of tensors in turn; 4096 x 2048 forward 13.4 us; one row 2.5
// us, a launch.  Rows past the registers (16384 columns) are read again for each pass: 8192 x
// 20000 bf16 forward 181 us for 655 MB, backward 540 us for 983, of which dw and db, column by
// column, are the larger part.
#include "common.h"

namespace moe {

namespace {

// 16 bytes at an address of any element: gfx950 global loads and stores run in unaligned
// mode, so rows of an odd width take wide accesses too
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

// V elements at column c of a row of H: whole vectors where they fit, element by element
// over the row's end (the kernels of long and of very short rows)
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

// The same for the rows held in registers: columns c .. c + V - 1, c >= -1; columns outside
// [0, H) read as 0 and are not written.  EDGE: H is no multiple of V.  A vector over a row's
// end is then read whole, with the neighbour rows' elements (which may be changing: they are
// dropped); at the tensor's own ends the vector is moved to columns lo .. hi, inside it, and
// its elements moved back.  (Element by element, the ends made the rows of 4095 bf16 take three
// times as long as those of 4096.)  What a row's end asks for is the same for all of its
// threads (the vector over it holds `tail` of the row's elements), so it is decided by scalar
// branches, and moving back is left to the last row.
struct RowEnds {
  int lo, hi, tail;
};
// of row t of T, V <= H, with vectors that start `shift` columns early
template <int V>
__device__ __forceinline__ RowEnds row_ends(int64_t t, int64_t T, int H, int shift) {
  const int64_t left = (T - t) * H - V;
  return {t > 0 ? -1 : 0, left < (1 << 30) ? (int)left : 1 << 30, (H + shift) & (V - 1)};
}
template <bool EDGE, typename T>
__device__ __forceinline__ void load_row(const T* row, RowEnds ends, int c, int H, float (&v)[rowvec<T>::V]) {
  constexpr int V = rowvec<T>::V;
  if (c < H) {
    if constexpr (EDGE) {
      rowvec<T>::load(row + min(max(c, ends.lo), ends.hi), v);
      if (c + V > H) {
        if (ends.hi < H) {   // the last row: moved by V - tail
#pragma unroll
          for (int b = V / 2; b >= 1; b >>= 1)
            if ((V - ends.tail) & b) {
#pragma unroll
              for (int j = 0; j + b < V; ++j) v[j] = v[j + b];
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j >= ends.tail) v[j] = 0.f;
      }
      if (sizeof(T) == 2 && c < 0) {
        if (ends.lo == 0) {
#pragma unroll
          for (int j = V - 1; j > 0; --j) v[j] = v[j - 1];
        }
        v[0] = 0.f;
      }
    } else {
      rowvec<T>::load(row + c, v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 0.f;
  }
}
template <bool EDGE, typename T>
__device__ __forceinline__ void store_row(T* row, int c, int H, int tail, const float (&v)[rowvec<T>::V]) {
  constexpr int V = rowvec<T>::V;
  if (!EDGE || (c >= 0 && c + V <= H)) {
    if (c < H) rowvec<T>::store(row + c, v);
  } else if (c < 0) {
#pragma unroll
    for (int j = 1; j < V; ++j) elem<T>::store(row + c + j, v[j]);
  } else if (c < H) {
#pragma unroll
    for (int j = 0; j < V - 1; ++j)
      if (j < tail) elem<T>::store(row + c + j, v[j]);
  }
}

// Columns by which a row's vectors start early, so that a bf16 row at an odd element is read
// at whole words (16 bytes at an odd one cost twice as much).  Any value gives the same
// results up to the order of the row's sums; cap: the columns that the row's threads hold.
template <bool EDGE, typename T>
__device__ __forceinline__ int col_shift(const T* row, int H, int cap) {
  return EDGE && sizeof(T) == 2 && H < cap ? (int)(((uintptr_t)row >> 1) & 1) : 0;
}

// The threads of a row: one wave (WAVE; four rows a workgroup) or the whole workgroup, of
// as many waves as the row fills.
template <bool WAVE>
__device__ __forceinline__ int row_threads() { return WAVE ? 64 : (int)blockDim.x; }

// Sums of a and b over the threads of a row, in every one of them.  Workgroups meet in red,
// of which the caller gives another slot for each call between two barriers.
template <bool WAVE>
__device__ __forceinline__ void row_sum2(float& a, float& b, float (*red)[2]) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    a += __shfl_xor(a, off, 64);
    b += __shfl_xor(b, off, 64);
  }
  if constexpr (!WAVE) {
    const int wv = threadIdx.x >> 6, nw = (int)(blockDim.x >> 6);
    if ((threadIdx.x & 63) == 0) {
      red[wv][0] = a;
      red[wv][1] = b;
    }
    __syncthreads();
    a = red[0][0];
    b = red[0][1];
#pragma unroll 4
    for (int i = 1; i < nw; ++i) {
      a += red[i][0];
      b += red[i][1];
    }
  }
}

constexpr int MAX_WAVES = 16;
template <bool WAVE>
constexpr int wg_most() { return WAVE ? 256 : 64 * MAX_WAVES; }

// Forward, a row in registers.  The norm is taken of the fp32 sum, not of the sum rounded to
// the stored type: y then carries one rounding instead of two.
template <typename T, bool WAVE, int EPT, bool EDGE, bool RMS>
__global__ __launch_bounds__(wg_most<WAVE>()) void k_norm_fwd(const T* x, const T* res, const T* __restrict__ w,
                                                             const T* __restrict__ b, int T_, int H, float eps,
                                                             T* sum, T* y, float* mean, float* rstd) {
  constexpr int V = rowvec<T>::V, NV = EPT / V, GROUPS = WAVE ? 4 : 1;
  __shared__ float red[4][MAX_WAVES][2];
  const int tpr = row_threads<WAVE>(), lane = WAVE ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  int par = 0;   // the row's slots in red: those of the row before may still be read
  for (int64_t t = (int64_t)blockIdx.x * GROUPS + (WAVE ? __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) : 0); t < T_;
       t += (int64_t)gridDim.x * GROUPS, par ^= 2) {
    const size_t off = (size_t)t * H;
    const int shift = col_shift<EDGE>(x + off, H, tpr * EPT);
    const RowEnds ends = row_ends<V>(t, T_, H, shift), vec = row_ends<V>(0, 1, H, shift);   // vec: w and b
    const int c0 = lane * V - shift;
    float v[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) load_row<EDGE>(x + off, ends, c0 + i * tpr * V, H, v[i]);
    if (res) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float r[V];
        load_row<EDGE>(res + off, ends, c0 + i * tpr * V, H, r);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] += r[j];
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) store_row<EDGE>(sum + off, c0 + i * tpr * V, H, ends.tail, v[i]);
    }
    float mu = 0.f;
    if constexpr (!RMS) {
      float s = 0.f, unused = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) s += v[i][j];
      row_sum2<WAVE>(s, unused, red[par]);
      mu = s / (float)H;
    }
    float q = 0.f, unused = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = c0 + i * tpr * V + (EDGE ? j : 0);   // else vectors lie inside or outside whole
        v[i][j] -= mu;
        if (RMS || (c >= 0 && c < H)) q += v[i][j] * v[i][j];
      }
    row_sum2<WAVE>(q, unused, red[par + 1]);
    const float rs = 1.f / sqrtf(q / (float)H + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * tpr * V;
      float wv[V];
      load_row<EDGE>(w, vec, c, H, wv);
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] *= rs * wv[j];
      if (b) {
        float bv[V];
        load_row<EDGE>(b, vec, c, H, bv);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] += bv[j];
      }
      store_row<EDGE>(y + off, c, H, ends.tail, v[i]);
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
  __shared__ float red[4][MAX_WAVES][2];
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
      row_sum2<false>(s, unused, red[par]);
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
    row_sum2<false>(q, unused, red[par + 1]);
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
template <typename T, bool WAVE, int EPT, bool EDGE, bool RMS, bool HAS_B>
__global__ __launch_bounds__(wg_most<WAVE>()) void k_norm_bwd(const T* __restrict__ dy, const T* __restrict__ s,
                                                             const T* __restrict__ res, const T* __restrict__ w,
                                                             const float* __restrict__ mean,
                                                             const float* __restrict__ rstd, const T* ds_in, int T_,
                                                             int H, T* dx, float* __restrict__ part) {
  constexpr int V = rowvec<T>::V, NV = EPT / V, GROUPS = WAVE ? 4 : 1;
  __shared__ float red[2][MAX_WAVES][2];
  __shared__ float fold[WAVE ? GROUPS * 64 * EPT : 1];
  const int tpr = row_threads<WAVE>(), lane = WAVE ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int group = WAVE ? __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) : 0;
  // one shift for all the rows of the group, whose columns stay with their threads (their
  // parities agree: the rows of a step are a multiple of 4, or the grid is even)
  const int shift = col_shift<EDGE>(s + ((size_t)blockIdx.x * GROUPS + group) * H, H, tpr * EPT);
  const int c0 = lane * V - shift;
  const RowEnds vec = row_ends<V>(0, 1, H, shift);   // of w
  float wv[NV][V], dwa[NV][V], dba[HAS_B ? NV : 1][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_row<EDGE>(w, vec, c0 + i * tpr * V, H, wv[i]);
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
    const RowEnds ends = row_ends<V>(t, T_, H, shift);
    float xh[NV][V], g[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_row<EDGE>(s + off, ends, c0 + i * tpr * V, H, xh[i]);
      load_row<EDGE>(dy + off, ends, c0 + i * tpr * V, H, g[i]);
    }
    const float mu = RMS ? 0.f : mean[t], rs = rstd[t];
    if (res) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float r[V];
        load_row<EDGE>(res + off, ends, c0 + i * tpr * V, H, r);
#pragma unroll
        for (int j = 0; j < V; ++j) xh[i][j] += r[j];
      }
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {   // columns outside the row hold dy = 0
        xh[i][j] = (xh[i][j] - mu) * rs;
        dwa[i][j] += g[i][j] * xh[i][j];
        if (HAS_B) dba[i][j] += g[i][j];
        g[i][j] *= wv[i][j];
        s1 += g[i][j];
        s2 += g[i][j] * xh[i][j];
      }
    row_sum2<WAVE>(s1, s2, red[par]);
    s1 = RMS ? 0.f : s1 * inv_h;
    s2 *= inv_h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * tpr * V;
#pragma unroll
      for (int j = 0; j < V; ++j) g[i][j] = rs * (g[i][j] - s1 - xh[i][j] * s2);
      if (ds_in) {
        float d[V];
        load_row<EDGE>(ds_in + off, ends, c, H, d);
#pragma unroll
        for (int j = 0; j < V; ++j) g[i][j] += d[j];
      }
      store_row<EDGE>(dx + off, c, H, ends.tail, g[i]);
    }
  }
  // the row groups' shares, added in group order
  auto leave = [&](float (&a)[NV][V], float* out) {
    if constexpr (WAVE) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = c0 + i * tpr * V + j;
          if (c >= 0 && c < H) fold[group * 64 * EPT + c] = a[i][j];
        }
      __syncthreads();
      for (int c = threadIdx.x; c < H; c += 256) {
        float sum = fold[c];
#pragma unroll
        for (int o = 1; o < GROUPS; ++o) sum += fold[o * 64 * EPT + c];
        out[c] = sum;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < V; q += 4)
          store_row<EDGE>(out, c0 + i * tpr * V + q, H, (H + shift) & 3, *reinterpret_cast<float(*)[4]>(&a[i][q]));
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
  __shared__ float red[2][MAX_WAVES][2];
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
    row_sum2<false>(s1, s2, red[par]);
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
constexpr int FOLD_COLS = 32, FOLD_GROUPS = 32;
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

// Threads of a row.  One wave up to 1024 columns (8 or 16 values a thread); then a workgroup
// of as many waves as 8 values a thread fill, to 8192 columns, and 1024 threads of 16 to
// 16384.  More values in fewer threads, with fewer barriers, lose: 16384 x 4096 bf16 with 128
// threads of 32 takes 107 us forward and 345 backward, with 512 of 8 94 and 134.
inline int norm_threads(int H) {
  return H <= 1024 ? 256 : H > 8192 ? 1024 : (int)(ceil_div(ceil_div(H, 8), 64) * 64);
}

// Shares of dw: workgroups of the backward, or row slices of the long rows.  One for every four
// of the rows (groups of four up to 1024 columns) that a workgroup takes at a time, but 256 where
// there are rows for them, and no more than 256 K threads hold, or 512: at 16384 x 4096 bf16 with
// a residual, 512 threads, 256 / 512 / 1024 / 2048 shares take 212 / 135 / 153 / 142 us, too few
// rows in flight on one side and more shares than rows are worth on the other.
int norm_parts(const moe_norm_shape& s) {
  if (s.T == 0) return 0;
  const int rows = s.H <= 1024 ? 4 : 1;   // rows a workgroup holds at once
  int64_t most = s.H > NORM_REG_COLS ? 16 : 262144 / norm_threads(s.H);
  if (s.H <= NORM_REG_COLS && most < 512) most = 512;
  const int64_t all = ceil_div(s.T, rows), want = ceil_div(all, 4) > 256 ? ceil_div(all, 4) : 256;
  int64_t g = all < want ? all : want;
  if (g > most) g = most;
  if (g < all && (g & 1)) ++g;   // even: see k_norm_bwd's columns
  return (int)g;
}

// rows held in registers: at least one vector, at most 1024 threads of 16 values
template <typename T>
inline bool in_registers(int H) { return H >= rowvec<T>::V && H <= NORM_REG_COLS; }

#define NORM_DISPATCH(H, EDGE, CALL)               \
  do {                                             \
    if ((H) <= 512) { CALL(true, 8, EDGE); }       \
    else if ((H) <= 1024) { CALL(true, 16, EDGE); } \
    else if ((H) <= 8192) { CALL(false, 8, EDGE); } \
    else { CALL(false, 16, EDGE); }                \
  } while (0)

template <typename T, bool RMS>
static hipError_t norm_fwd(const moe_norm_shape& s, const void* x_, const void* res_, const void* w_, const void* b_,
                           void* sum_, void* y_, float* mean, float* rstd, hipStream_t st) {
  const T *x = (const T*)x_, *res = (const T*)res_, *w = (const T*)w_, *b = (const T*)b_;
  T *sum = (T*)sum_, *y = (T*)y_;
  if (!in_registers<T>(s.H)) {
    MOE_LAUNCH("norm_fwd", (k_norm_fwd_long<T, RMS>), dim3(row_grid(s.T)), dim3(LONG_T), 0, st, x, res, w, b, s.T,
               s.H, s.eps, sum, y, mean, rstd);
    return hipGetLastError();
  }
#define CALL(WAVE, EPT, EDGE)                                                                                        \
  MOE_LAUNCH("norm_fwd", (k_norm_fwd<T, WAVE, EPT, EDGE, RMS>), dim3(row_grid(WAVE ? ceil_div(s.T, 4) : s.T)),          \
             dim3((unsigned)norm_threads(s.H)), 0, st, x, res, w, b, s.T, s.H, s.eps, sum, y, mean, rstd)
  if (s.H % rowvec<T>::V) NORM_DISPATCH(s.H, true, CALL);
  else NORM_DISPATCH(s.H, false, CALL);
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
  if (s.T > 0 && !in_registers<T>(s.H)) {
    MOE_LAUNCH("norm_dx", (k_norm_dx_long<T, RMS>), dim3(row_grid(s.T)), dim3(LONG_T), 0, st, dy, sum, res, w, mean,
               rstd, ds_in, s.T, s.H, dx);
    MOE_LAUNCH("norm_dw", (k_norm_dw_long<T, RMS>), dim3((unsigned)ceil_div(s.H, 256), (unsigned)G), dim3(256), 0, st,
               dy, sum, res, mean, rstd, s.T, s.H, part, HAS_B);
  } else if (s.T > 0) {
#define CALL(WAVE, EPT, EDGE)                                                                                          \
  MOE_LAUNCH("norm_bwd", (k_norm_bwd<T, WAVE, EPT, EDGE, RMS, HAS_B>), dim3((unsigned)G), dim3((unsigned)norm_threads(s.H)), \
             0, st, dy, sum, res, w, mean, rstd, ds_in, s.T, s.H, dx, part)
    if (s.H % rowvec<T>::V) NORM_DISPATCH(s.H, true, CALL);
    else NORM_DISPATCH(s.H, false, CALL);
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
