// Orthogonalising weight updates by Newton-Schulz products (the Muon optimiser's step), a
// batch of equal matrices (one per expert) in one call.
//
// With m = min(rows, cols), l = max(rows, cols) and X [m, l] the matrix (or its transpose)
// divided by its Frobenius norm, every step is
//   A = X X^T,  X <- a X + (b A + c A^2) X,   (a, b, c) = (3.4445, -4.7750, 2.0315),
// which maps each singular value by p(s) = a s + b s^3 + c s^5.  p takes [0, 1.2025] into
// itself (its peak there is 1.2025), so every |entry| and every eigenvalue below is bounded.
//
// Precision.  The products run on fp16 MFMAs with fp32 sums; fp16 has three more bits than
// bf16 at the same rate, and the bounds above fix scales that keep it in range:
//   X * 2^15 (<= 39400), A * 2^14 (<= 23700), (b A + c A^2) * 2^14 (<= 46000).
// An early rounding is what hurts: a singular value far below the largest is multiplied by
// a = 3.4 a step, and so is the rounding noise that lands beside it.  So
// * the step's a X is added in fp32 outside the matrix product (with a I inside the fp16
//   factor, its rounded diagonal leaks the large directions into the small ones);
// * X is kept as a pair hi + lo of fp16 through the first steps (the product reads hi, a X
//   both), and enters as the exact bf16 values scaled by a power of two;
// * from step 3 on, when the singular values are near 1, A is kept as D = A - I:
//   b A + c A^2 = (b + c) I + (b + 2c) D + c D^2, so the diagonal's rounding enters times
//   b + 2c = -0.71 instead of b = -4.8.
// Against fp64 that is 0.7 to 2e-3 of the result's norm over spectra from flat to a
// thousandfold spread, next to 1.7e-3 for the output's own rounding to bf16 (plain fp16
// iterates: up to 4e-2, bf16 ones: up to 3e-1, on the same matrices).
#include "common.h"

namespace moe {

namespace {

typedef _Float16 f16;
typedef f16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float NS_A = 3.4445f, NS_B = -4.7750f, NS_C = 2.0315f;
constexpr double NS_EPS = 1e-7;
constexpr int X_LOG2 = 15, D_LOG2 = 14, B_LOG2 = 14;
constexpr float X_SCALE = 32768.f, D_SCALE = 16384.f, B_SCALE = 16384.f;
constexpr int LO_STEPS = 3;      // the first iterates that are kept as hi + lo
constexpr int SHIFT_STEP = 3;    // from this step on, D = A - I

// ---- norm and entry ----
constexpr int NORM_CHUNKS = 64;   // workgroups a matrix at most

// sums of squares of chunk blockIdx.x of matrix blockIdx.y, in fp64: neither a gradient of
// 1e-30 nor one of 1e30 leaves the range
template <typename T>
__global__ __launch_bounds__(256) void k_orth_sumsq(const T* __restrict__ g, int64_t count, int64_t chunk,
                                                    double* __restrict__ part) {
  const T* p = g + (int64_t)blockIdx.y * count;
  const int64_t b = (int64_t)blockIdx.x * chunk, e = b + chunk < count ? b + chunk : count;
  double a = 0.0;
  for (int64_t i = b + threadIdx.x; i < e; i += 256) {
    const double v = (double)elem<T>::load(p + i);
    a += v * v;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) a += __shfl_xor(a, off, 64);
  __shared__ double red[4];
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
  __syncthreads();
  if (threadIdx.x == 0) part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// X0 (hi, and lo for fp32 input) [m_p, l_p] of each matrix, padded with zeros, from g
// [rows, cols] (transposed when rows > cols) times 2^e, where 2^e brings the norm into
// [2^14, 2^15); factor[matrix] = 2^-e / (norm + eps) turns stored values into X0.
template <typename T, bool TR>
__global__ __launch_bounds__(256) void k_orth_enter(const T* __restrict__ g, int rows, int cols,
                                                    const double* __restrict__ part, int chunks, int mp, int lp,
                                                    f16* __restrict__ hi, f16* __restrict__ lo,
                                                    float* __restrict__ factor) {
  __shared__ float tile[64][65];
  double ss = 0.0;
  for (int i = 0; i < chunks; ++i) ss += part[(size_t)blockIdx.z * chunks + i];
  const double norm = sqrt(ss);
  int e = 0;
  if (norm > 0.0 && norm < 1e300) {
    frexp(norm, &e);   // norm = f 2^e, f in [1/2, 1)
    e = X_LOG2 - e;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    factor[blockIdx.z] = (float)(ldexp(1.0, -e) / (norm + NS_EPS));
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;   // of X
  const T* p = g + (size_t)blockIdx.z * rows * cols;
  const int m = TR ? cols : rows, l = TR ? rows : cols;
  if (TR) {
    for (int i = ty; i < 64; i += 4) {   // g row = X column c0 + i, g column = X row r0 + tx
      const int r = c0 + i, c = r0 + tx;
      tile[tx][i] = r < l && c < m ? elem<T>::load(p + (size_t)r * cols + c) : 0.f;
    }
    __syncthreads();
  }
  for (int i = ty; i < 64; i += 4) {
    const int r = r0 + i, c = c0 + tx;
    float v = TR ? tile[i][tx] : r < m && c < l ? elem<T>::load(p + (size_t)r * cols + c) : 0.f;
    v = ldexpf(v, e);
    const size_t o = ((size_t)blockIdx.z * mp + r) * lp + c;
    const f16 h = (f16)v;
    hi[o] = h;
    if (lo) lo[o] = (f16)(v - (float)h);
  }
}

// ---- the products ----
// C = P Q^T (NT) or P Q, one 64 x 64 tile a workgroup of four waves
constexpr int TB = 64, TK = 64, TLD = TK + 8;

enum { ORTH_GRAM = 0, ORTH_POLY = 1, ORTH_APPLY = 2, ORTH_LAST = 3 };

struct OrthArgs {
  int mp, lp;             // padded sizes, multiples of 64
  int m, l, rows, cols;
  int step;
  const f16* x;           // X hi [n, mp, lp]
  const f16* xlo;         // X lo, or null
  const float* factor;    // stored X -> X, per matrix (step 0)
  f16* d;                 // D [n, mp, mp]
  f16* b;                 // B = beta D + c D^2 [n, mp, mp]
  f16* xn;                // the next X
  f16* xnlo;              // its lo, or null
  bf16_t* out;            // the last step's result [n, rows, cols]
  float scale;
};

struct StepCoef {
  float t, alpha, beta;   // D = A - t I;  X' = alpha X + (beta D + c D^2) X
};
__host__ __device__ inline StepCoef step_coef(int step) {
  const float t = step >= SHIFT_STEP ? 1.f : 0.f;
  return {t, NS_A + NS_B * t + NS_C * t * t, NS_B + 2.f * NS_C * t};
}

template <int OP>
__global__ __launch_bounds__(256) void k_orth_tile(OrthArgs a) {
  __shared__ __attribute__((aligned(16))) f16 ps[TB * TLD];
  __shared__ __attribute__((aligned(16))) f16 qs[TB * TLD];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int z = blockIdx.z;
  int i0, j0;
  if (OP == ORTH_GRAM || OP == ORTH_POLY) {   // lower triangle of tiles
    int ti = 0, rem = blockIdx.x;
    while (rem > ti) rem -= ++ti;
    i0 = ti * TB;
    j0 = rem * TB;
  } else {
    i0 = blockIdx.y * TB;
    j0 = blockIdx.x * TB;
  }
  const int K = OP == ORTH_GRAM ? a.lp : a.mp;
  const size_t xo = (size_t)z * a.mp * a.lp, so = (size_t)z * a.mp * a.mp;
  const f16* P = OP == ORTH_GRAM ? a.x + xo : OP == ORTH_POLY ? a.d + so : a.b + so;
  const f16* Q = OP == ORTH_GRAM ? a.x + xo : OP == ORTH_POLY ? a.d + so : a.x + xo;
  f32x16 acc;
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = 0.f;
  const int wi = (wv & 1) * 32, wj = (wv >> 1) * 32;
  for (int k0 = 0; k0 < K; k0 += TK) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = (tid >> 3) + 32 * q, c = (tid & 7) * 8;
      *reinterpret_cast<f16x8*>(&ps[r * TLD + c]) = *reinterpret_cast<const f16x8*>(P + (size_t)(i0 + r) * K + k0 + c);
      if (OP <= ORTH_POLY) {
        *reinterpret_cast<f16x8*>(&qs[r * TLD + c]) =
            *reinterpret_cast<const f16x8*>(Q + (size_t)(j0 + r) * K + k0 + c);
      } else {
        const f16x8 v = *reinterpret_cast<const f16x8*>(Q + (size_t)(k0 + r) * a.lp + j0 + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) qs[(c + j) * TLD + r] = v[j];
      }
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < TK / 16; ++kk) {
      const int kt = kk * 16 + (lane >> 5) * 8;
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(
          *reinterpret_cast<const f16x8*>(&ps[(wi + (lane & 31)) * TLD + kt]),
          *reinterpret_cast<const f16x8*>(&qs[(wj + (lane & 31)) * TLD + kt]), acc, 0, 0, 0);
    }
  }
  const StepCoef co = step_coef(a.step);
  const float f = a.step == 0 ? a.factor[z] : 1.f / X_SCALE;
  const int j = j0 + wj + (lane & 31);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int i = i0 + wi + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
    if (OP == ORTH_GRAM) {
      const f16 v = (f16)(acc[r] * (f * f * D_SCALE) - (i == j ? co.t * D_SCALE : 0.f));
      a.d[so + (size_t)i * a.mp + j] = v;
      if (i0 != j0) a.d[so + (size_t)j * a.mp + i] = v;
    } else if (OP == ORTH_POLY) {
      const float dv = (float)a.d[so + (size_t)i * a.mp + j];
      const f16 v = (f16)(acc[r] * (NS_C * B_SCALE / (D_SCALE * D_SCALE)) + dv * (co.beta * B_SCALE / D_SCALE));
      a.b[so + (size_t)i * a.mp + j] = v;
      if (i0 != j0) a.b[so + (size_t)j * a.mp + i] = v;
    } else {
      const size_t o = xo + (size_t)i * a.lp + j;
      float xv = (float)a.x[o];
      if (a.xlo) xv += (float)a.xlo[o];
      const float v = xv * (co.alpha * f) + acc[r] * (f / B_SCALE);
      if (OP == ORTH_APPLY) {
        const float s = v * X_SCALE;
        const f16 h = (f16)s;
        a.xn[o] = h;
        if (a.xnlo) a.xnlo[o] = (f16)(s - (float)h);
      } else if (i < a.m && j < a.l) {
        const size_t base = (size_t)z * a.rows * a.cols;
        const size_t oo = a.rows > a.cols ? (size_t)j * a.cols + i : (size_t)i * a.cols + j;
        a.out[base + oo] = f2bf(v * a.scale);
      }
    }
  }
}

inline int pad64(int v) { return (v + 63) & ~63; }

}  // namespace

// Scratch: norm shares and factors, then X (two iterates, hi and lo), D and B
struct OrthLayout {
  int m, l, mp, lp, chunks;
  size_t off_part, off_factor, off_x[2], off_lo[2], off_d, off_b, bytes;
};
static OrthLayout orth_layout(const moe_orth_shape& s) {
  OrthLayout L{};
  L.m = s.rows < s.cols ? s.rows : s.cols;
  L.l = s.rows < s.cols ? s.cols : s.rows;
  L.mp = pad64(L.m);
  L.lp = pad64(L.l);
  const int64_t count = (int64_t)s.rows * s.cols;
  const int64_t ch = ceil_div(count, 16384);
  L.chunks = (int)(ch < NORM_CHUNKS ? ch : NORM_CHUNKS);
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off += (n + 255) / 256 * 256;
    return at;
  };
  const size_t xb = (size_t)s.n * L.mp * L.lp * 2, db = (size_t)s.n * L.mp * L.mp * 2;
  L.off_part = take((size_t)s.n * L.chunks * 8);
  L.off_factor = take((size_t)s.n * 4);
  for (int i = 0; i < 2; ++i) {
    L.off_x[i] = take(xb);
    L.off_lo[i] = take(xb);
  }
  L.off_d = take(db);
  L.off_b = take(db);
  L.bytes = off;
  return L;
}
size_t orth_scratch_bytes(const moe_orth_shape& s) { return orth_layout(s).bytes; }

template <typename T>
static void orth_enter(const moe_orth_shape& s, const OrthLayout& L, const T* g, char* ws, hipStream_t st) {
  const int64_t count = (int64_t)s.rows * s.cols;
  const int64_t chunk = ceil_div(count, L.chunks);
  double* part = reinterpret_cast<double*>(ws + L.off_part);
  float* factor = reinterpret_cast<float*>(ws + L.off_factor);
  f16* hi = reinterpret_cast<f16*>(ws + L.off_x[0]);
  f16* lo = s.dtype == MOE_F32 ? reinterpret_cast<f16*>(ws + L.off_lo[0]) : nullptr;
  MOE_LAUNCH("orth_sumsq", k_orth_sumsq<T>, dim3((unsigned)L.chunks, (unsigned)s.n), dim3(256), 0, st, g, count, chunk,
             part);
  const dim3 grid((unsigned)(L.lp / 64), (unsigned)(L.mp / 64), (unsigned)s.n);
  if (s.rows > s.cols)
    MOE_LAUNCH("orth_enter", (k_orth_enter<T, true>), grid, dim3(256), 0, st, g, s.rows, s.cols, part, L.chunks, L.mp,
               L.lp, hi, lo, factor);
  else
    MOE_LAUNCH("orth_enter", (k_orth_enter<T, false>), grid, dim3(256), 0, st, g, s.rows, s.cols, part, L.chunks, L.mp,
               L.lp, hi, lo, factor);
}

hipError_t launch_orthogonalize(const moe_orth_shape& s, const void* g, void* o, float scale, void* scratch,
                                hipStream_t st) {
  const OrthLayout L = orth_layout(s);
  char* ws = reinterpret_cast<char*>(scratch);
  if (s.dtype == MOE_BF16) orth_enter(s, L, (const bf16_t*)g, ws, st);
  else orth_enter(s, L, (const float*)g, ws, st);
  const int tm = L.mp / TB, tl = L.lp / TB;
  for (int i = 0; i < s.steps; ++i) {
    OrthArgs a{};
    a.mp = L.mp; a.lp = L.lp; a.m = L.m; a.l = L.l; a.rows = s.rows; a.cols = s.cols;
    a.step = i;
    a.x = reinterpret_cast<const f16*>(ws + L.off_x[i & 1]);
    const bool lo_in = i == 0 ? s.dtype == MOE_F32 : i <= LO_STEPS, last = i == s.steps - 1;
    a.xlo = lo_in ? reinterpret_cast<const f16*>(ws + L.off_lo[i & 1]) : nullptr;
    a.factor = reinterpret_cast<const float*>(ws + L.off_factor);
    a.d = reinterpret_cast<f16*>(ws + L.off_d);
    a.b = reinterpret_cast<f16*>(ws + L.off_b);
    a.xn = reinterpret_cast<f16*>(ws + L.off_x[(i + 1) & 1]);
    a.xnlo = i < LO_STEPS ? reinterpret_cast<f16*>(ws + L.off_lo[(i + 1) & 1]) : nullptr;
    a.out = (bf16_t*)o;
    a.scale = scale;
    const dim3 sym((unsigned)(tm * (tm + 1) / 2), 1, (unsigned)s.n), full((unsigned)tl, (unsigned)tm, (unsigned)s.n);
    MOE_LAUNCH("orth_gram", k_orth_tile<ORTH_GRAM>, sym, dim3(256), 0, st, a);
    MOE_LAUNCH("orth_poly", k_orth_tile<ORTH_POLY>, sym, dim3(256), 0, st, a);
    if (last) MOE_LAUNCH("orth_last", k_orth_tile<ORTH_LAST>, full, dim3(256), 0, st, a);
    else MOE_LAUNCH("orth_apply", k_orth_tile<ORTH_APPLY>, full, dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace moe
