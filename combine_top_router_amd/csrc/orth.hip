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
#define MOE_GEMM_FW 256
#include "gemm_engine.h"

namespace moe {

namespace {

typedef _Float16 f16;
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef i32x4 i32x4_a2 __attribute__((aligned(2)));   // 16 bytes at any element of bf16

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

// ---- the products on 256 x 256 tiles: jobs of the persistent tile stream ----
__device__ __forceinline__ f16x8 as_f16(bf16x8 v) { return __builtin_bit_cast(f16x8, v); }

// 8 fp32 values of one row <-> 16 bytes of fp16
__device__ __forceinline__ f16x8 half8(const float (&v)[8]) {
  f16x8 h;
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = (f16)v[j];
  return h;
}

struct OrthTile {
  int z, i0, j0, nk;
  int cnt, ncols;   // rows and columns of the product in the tile
  float f;          // stored X -> X
};

struct OrthLd {
  static constexpr bool GATHER = false;
  int nk, pw;
  const bf16_t* a[A_LP];   // the lane's chunk of its rows at K step 0 (K-major)
  const bf16_t* b[B_LP];   // K-major rows, or MN-major k-rows
  size_t bstep;            // elements from one K step of B to the next
  __device__ __forceinline__ void fetch(int, int) const {}
  template <class F>
  __device__ __forceinline__ void issue(int kt, bf16_t* st, int, int, F&&) const {
#pragma unroll
    for (int q = 0; q < A_LP; ++q) dma16(a[q] + kt * BK, a_dst(st, q, pw));
#pragma unroll
    for (int q = 0; q < B_LP; ++q) dma16(b[q] + (size_t)kt * bstep, b_dst(st, q, pw));
  }
};

template <int OP>
struct JOrth {
  using Tile = OrthTile;
  using Ld = OrthLd;
  static constexpr bool SYM = OP == ORTH_GRAM || OP == ORTH_POLY;
  static constexpr bool A_KMAJ = true, B_KMAJ = SYM;
  static constexpr bool DYN = false, TRANS = false, EPI_LDS = true, NSPLIT = false, SIDE = false;
  OrthArgs a;
  int n, tm, tn;   // matrices; tiles along the rows and columns of a product
  __device__ __forceinline__ static int ncol(int wn, int ni) { return wn * WCOLS + ni * 32; }
  __device__ __forceinline__ int per() const { return SYM ? tm * (tm + 1) / 2 : tm * tn; }
  __device__ __forceinline__ int items() const { return n * per(); }
  __device__ __forceinline__ void tile(int v, Tile& p) const {
    p.z = uni(v / per());
    int rem = uni(v - p.z * per()), ti = 0;
    if (SYM) {
      while (rem > ti) rem -= ++ti;   // the lower triangle, row by row
    } else {
      ti = uni(rem % tm);             // down a column of tiles, which shares the tiles of X
      rem = uni(rem / tm);
    }
    p.i0 = uni(ti * BM);
    p.j0 = uni(rem * BN);
    p.nk = uni((OP == ORTH_GRAM ? a.lp : a.mp) / BK);
    p.cnt = uni(min(BM, a.mp - p.i0));
    p.ncols = uni(min(BN, (SYM ? a.mp : a.lp) - p.j0));
    p.f = a.step == 0 ? sload(a.factor + p.z) : 1.f / X_SCALE;
  }
  __device__ __forceinline__ WaveRows rows(const Tile& p, int wm) const { return wave_rows(p.cnt, wm); }
  __device__ __forceinline__ void setup(int v, Ld& p, int pw, int lane) const {
    Tile t;
    tile(v, t);
    p.pw = pw;
    p.nk = t.nk;
    const int K = OP == ORTH_GRAM ? a.lp : a.mp;
    const size_t xo = (size_t)t.z * a.mp * a.lp, so = (size_t)t.z * a.mp * a.mp;
    const bf16_t* pa = reinterpret_cast<const bf16_t*>(OP == ORTH_GRAM ? a.x + xo : OP == ORTH_POLY ? a.d + so : a.b + so);
    const bf16_t* pb = reinterpret_cast<const bf16_t*>(OP == ORTH_POLY ? a.d + so : a.x + xo);
#pragma unroll
    for (int q = 0; q < A_LP; ++q) {
      int r, c;
      kmaj_slot(load_slot(q, pw, lane), r, c);
      p.a[q] = pa + (size_t)min(t.i0 + r, a.mp - 1) * K + c * 8;
    }
#pragma unroll
    for (int q = 0; q < B_LP; ++q) {
      int r, c;
      if (SYM) {
        kmaj_slot(load_slot(q, pw, lane), r, c);
        p.b[q] = pb + (size_t)min(t.j0 + r, a.mp - 1) * K + c * 8;
      } else {
        mnmaj_slot<BN>(load_slot(q, pw, lane), r, c);
        const int col = t.j0 + c * 8;
        p.b[q] = pb + (size_t)r * a.lp + (col < a.lp ? col : t.j0);   // past the edge: any column, not stored
      }
    }
    p.bstep = SYM ? (size_t)BK : (size_t)BK * a.lp;
  }
  __device__ __forceinline__ void compute(const bf16_t* st, int, Acc& acc, int lane, const WaveRows& w, int wn) const {
    const bf16_t* As = st;
    const bf16_t* Bs = st + A_ELEMS;
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      bf16x8 af[MI], bf[NI];
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) af[mi] = frag_kmaj(As, w.base + mi * 32, kk, lane);
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        bf[ni] = B_KMAJ ? frag_kmaj(Bs, ncol(wn, ni), kk, lane) : frag_mnmaj<BN>(Bs, ncol(wn, ni), kk, lane);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          acc[mi][ni] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_f16(af[mi]), as_f16(bf[ni]), acc[mi][ni], 0, 0, 0);
    }
  }
  // 16 rows at a time through the wave's fp32 staging: rows leave as they are, 8 columns a
  // lane; a mirrored tile (or a transposed result) leaves as columns too, 16 rows a lane,
  // from the finished values put back into the staging.
  __device__ __forceinline__ void epilogue(const Tile& p, const Acc& acc, float* stage) const {
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int wm = (int)((unsigned)wv % WM), wn = (int)((unsigned)wv / WM);
    float* wsm = stage + wv * EP_ROWS * EP_LD;
    const StepCoef co = step_coef(a.step);
    const size_t xo = (size_t)p.z * a.mp * a.lp, so = (size_t)p.z * a.mp * a.mp;
    const bool tr = a.rows > a.cols;
    const bool cols_out = SYM ? p.i0 != p.j0 : OP == ORTH_LAST && tr;
    const int jw = p.j0 + wn * WCOLS;   // the wave's first column
    if (jw - p.j0 >= p.ncols) return;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int rt = wm * WROWS + mi * 32 + h * 16;   // the piece's first row in the tile
        if (rt < p.cnt) {
          stage_quarter(wsm, acc, mi, h, lane);
#pragma unroll
          for (int jj = 0; jj < EP_ROWS / EP_RPP; ++jj) {
            const int rr = lane / EP_LPR + EP_RPP * jj, cc = (lane % EP_LPR) * 8;
            const int i = p.i0 + rt + rr, j = jw + cc;
            float* const q = wsm + rr * EP_LD + cc;
            float v[8];
            read8(q, rr, v);
            if constexpr (OP == ORTH_GRAM) {
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = v[e] * (p.f * p.f * D_SCALE) - (i == j + e ? co.t * D_SCALE : 0.f);
              *reinterpret_cast<f16x8*>(a.d + so + (size_t)i * a.mp + j) = half8(v);
            } else if constexpr (OP == ORTH_POLY) {
              const f16x8 d = *reinterpret_cast<const f16x8*>(a.d + so + (size_t)i * a.mp + j);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[e] = v[e] * (NS_C * B_SCALE / (D_SCALE * D_SCALE)) + (float)d[e] * (co.beta * B_SCALE / D_SCALE);
              *reinterpret_cast<f16x8*>(a.b + so + (size_t)i * a.mp + j) = half8(v);
            } else {
              const size_t o = xo + (size_t)i * a.lp + j;
              const f16x8 xh = *reinterpret_cast<const f16x8*>(a.x + o);
              float xv[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) xv[e] = (float)xh[e];
              if (a.xlo) {
                const f16x8 xl = *reinterpret_cast<const f16x8*>(a.xlo + o);
#pragma unroll
                for (int e = 0; e < 8; ++e) xv[e] += (float)xl[e];
              }
              const float ca = co.alpha * p.f, cb = p.f / B_SCALE;
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = xv[e] * ca + v[e] * cb;
              if constexpr (OP == ORTH_APPLY) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= X_SCALE;
                const f16x8 hi = half8(v);
                *reinterpret_cast<f16x8*>(a.xn + o) = hi;
                if (a.xnlo) {
#pragma unroll
                  for (int e = 0; e < 8; ++e) v[e] -= (float)hi[e];
                  *reinterpret_cast<f16x8*>(a.xnlo + o) = half8(v);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= a.scale;
                if (!tr && i < a.m) {
                  bf16_t* const out = a.out + (size_t)p.z * a.rows * a.cols + (size_t)i * a.cols + j;
                  if (j + 8 <= a.l) {
                    *reinterpret_cast<i32x4_a2*>(out) = pack8(v);
                  } else {
                    for (int e = 0; e < 8; ++e)
                      if (j + e < a.l) out[e] = f2bf(v[e]);
                  }
                }
              }
            }
            if (cols_out) {
#pragma unroll
              for (int e = 0; e < 8; ++e) q[e] = v[e];
            }
          }
          staging_done();
          if (cols_out) {
            const int i = p.i0 + rt, j = jw + lane;   // rows i .. i + 15 of column j
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = wsm[e * EP_LD + lane];
            if constexpr (SYM) {
              f16* const d = (OP == ORTH_GRAM ? a.d : a.b) + so + (size_t)j * a.mp + i;
              f16x8 lo, hi;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                lo[e] = (f16)v[e];
                hi[e] = (f16)v[8 + e];
              }
              *reinterpret_cast<f16x8*>(d) = lo;
              *reinterpret_cast<f16x8*>(d + 8) = hi;
            } else if (j < a.l) {
              bf16_t* const out = a.out + (size_t)p.z * a.rows * a.cols + (size_t)j * a.cols + i;
              float lo[8], hi[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                lo[e] = v[e];
                hi[e] = v[8 + e];
              }
              if (i + 16 <= a.m) {
                *reinterpret_cast<i32x4_a2*>(out) = pack8(lo);
                *reinterpret_cast<i32x4_a2*>(out + 8) = pack8(hi);
              } else {
                for (int e = 0; e < 16; ++e)
                  if (i + e < a.m) out[e] = f2bf(v[e]);
              }
            }
            staging_done();
          }
        }
      }
  }
};

template <int OP>
__global__ __launch_bounds__(NTHR, 1) void k_orth_stream(OrthArgs a, int n, int tm, int tn) {
  __shared__ __attribute__((aligned(16))) bf16_t lds[LDS_ELEMS];
  JOrth<OP> job{a, n, tm, tn};
  run_stream(job, lds);
}

template <int OP>
static void orth_product(const char* name, const OrthArgs& a, int n, bool wide, hipStream_t st) {
  constexpr bool SYM = OP == ORTH_GRAM || OP == ORTH_POLY;
  if (wide) {
    const int tm = (int)ceil_div(a.mp, BM), tn = (int)ceil_div(a.lp, BN);
    const int64_t items = (int64_t)n * (SYM ? tm * (tm + 1) / 2 : tm * tn);
    MOE_LAUNCH(name, k_orth_stream<OP>, dim3((unsigned)grid_for(items)), dim3(NTHR), 0, st, a, n, tm, tn);
  } else {
    const int tm = a.mp / TB, tn = a.lp / TB;
    const dim3 grid = SYM ? dim3((unsigned)(tm * (tm + 1) / 2), 1, (unsigned)n) : dim3((unsigned)tn, (unsigned)tm, (unsigned)n);
    MOE_LAUNCH(name, k_orth_tile<OP>, grid, dim3(256), 0, st, a);
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
  const bool wide = L.mp >= 256;
  for (int i = 0; i < s.steps; ++i) {
    OrthArgs a{};
    a.mp = L.mp; a.lp = L.lp; a.m = L.m; a.l = L.l; a.rows = s.rows; a.cols = s.cols;
    a.step = i;
    a.x = reinterpret_cast<const f16*>(ws + L.off_x[i & 1]);
    const bool lo_in = i == 0 ? s.dtype == MOE_F32 : i <= LO_STEPS;
    a.xlo = lo_in ? reinterpret_cast<const f16*>(ws + L.off_lo[i & 1]) : nullptr;
    a.factor = reinterpret_cast<const float*>(ws + L.off_factor);
    a.d = reinterpret_cast<f16*>(ws + L.off_d);
    a.b = reinterpret_cast<f16*>(ws + L.off_b);
    a.xn = reinterpret_cast<f16*>(ws + L.off_x[(i + 1) & 1]);
    a.xnlo = i < LO_STEPS ? reinterpret_cast<f16*>(ws + L.off_lo[(i + 1) & 1]) : nullptr;
    a.out = (bf16_t*)o;
    a.scale = scale;
    orth_product<ORTH_GRAM>("orth_gram", a, s.n, wide, st);
    orth_product<ORTH_POLY>("orth_poly", a, s.n, wide, st);
    if (i == s.steps - 1) orth_product<ORTH_LAST>("orth_last", a, s.n, wide, st);
    else orth_product<ORTH_APPLY>("orth_apply", a, s.n, wide, st);
  }
  return hipGetLastError();
}

}  // namespace moe
