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
//   X * 2^15 (<= 39400), A * 2^14 (<= 23700), (b A + c A^2) * 2^14 (<= 46000);
// a matrix whose norm is next to eps or below, and its iterates as small, takes another power of
// two on X, so that they keep their bits.
// An early rounding is what hurts: a singular value far below the largest is multiplied by
// a = 3.4 a step, and so is the rounding noise that lands beside it.  So
// * the step's a X is added to the fp32 sums by itself (with a I inside the fp16 factor, the
//   rounded diagonal leaks the large directions into the small ones); where matrix
//   instructions add it, a times the factor's scale is made an fp16 number by that scale;
// * the first iterates are kept as a pair, hi in fp16 and lo = the rest times 16 in E4M3 (a
//   byte: 15 bits together; the product reads hi, a X both), and X enters as the exact bf16
//   values scaled by a power of two;
// * from step 3 on, when the singular values are near 1, A is kept as D = A - I:
//   b A + c A^2 = (b + c) I + (b + 2c) D + c D^2, so the diagonal's rounding enters times
//   b + 2c = -0.71 instead of b = -4.8.
// Against fp64, five steps, that is 0.7 to 2e-3 of the result's norm over spectra from flat to
// a thousandfold spread, next to 1.7e-3 for the output's own rounding (plain fp16 iterates: up
// to 4e-2, bf16 ones: up to 3e-1, on the same matrices).  Gradients of few tokens, of rank 1 to
// 64 with a few rows or columns 30 to 1000 times the others, usually cost 1 to 3e-3 and up to
// 5e-3, most of it the rounding of b A + c A^2 where a few rows hold it all; of rank 1 in fp32,
// which enters in 15 bits, up to 8e-3.
// The first two steps as one, in the square matrices (A_1 = a^2 R + 2a B_0 R + B_0^2 R and so on),
// would save 9% of the large updates below and up to a quarter of those of few rows, but its
// roundings cost up to 2e-2 on such gradients.
//
// Cost.  A step is 3 m^2 l + m^3 multiply-adds (A and A^2 by halves), which binds from a few
// matrices of some hundred rows on; below, launches and latencies do.  Measured on one MI355X,
// five steps, bf16, one call after another: 128 of 2048 x 768 3.65 ms, 16 of 1536 x 4096 3.22
// (2.6 PFLOP of such work each, 2.4 ms at the 1.08 PFLOP/s of a large library fp16 product;
// both run at the clock that their power leaves).  Of the former 0.23 read g twice and write X
// (5.1 TB/s).
#define MOE_GEMM_FW 256
#include <math.h>

#include "gemm_engine.h"

namespace moe {

namespace {

typedef _Float16 f16;
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef i32x4 i32x4_a2 __attribute__((aligned(2)));   // 16 bytes at any element of bf16
typedef i32x4 i32x4_a4 __attribute__((aligned(4)));   // or of fp32

constexpr float NS_A = 3.4445f, NS_B = -4.7750f, NS_C = 2.0315f;
constexpr double NS_EPS = 1e-7;
constexpr int X_LOG2 = 15;
constexpr float X_SCALE = 32768.f, D_SCALE = 16384.f, B_SCALE = 16384.f;
constexpr float LO_SCALE = 16.f;  // |lo| <= 16, half a step of fp16 at its top: 256 of E4M3's 448
constexpr int LO_STEPS = 2;      // the first iterates that are kept as hi + lo
constexpr int SHIFT_STEP = 3;    // from this step on, D = A - I

__device__ __forceinline__ uint8_t lo_code(float rest) {
  return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(rest * LO_SCALE, 0.f, 0, false);
}
__device__ __forceinline__ float lo_value(uint8_t code) {
  return __builtin_amdgcn_cvt_f32_fp8(code, 0) * (1.f / LO_SCALE);
}

// ---- norm and entry ----
constexpr int NORM_CHUNKS = 64;   // workgroups a matrix at most

// 8 elements at p, of which `left` are there (the rest read as 0); p at any element
__device__ __forceinline__ void load8_any(const bf16_t* p, int left, float (&v)[8]) {
  if (left >= 8) {
    unpack8(*reinterpret_cast<const i32x4_a2*>(p), v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? bf2f(p[e]) : 0.f;
  }
}
__device__ __forceinline__ void load8_any(const float* p, int left, float (&v)[8]) {
  if (left >= 8) {
    const i32x4 a = *reinterpret_cast<const i32x4_a4*>(p), b = *reinterpret_cast<const i32x4_a4*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __uint_as_float((uint32_t)a[e]);
      v[4 + e] = __uint_as_float((uint32_t)b[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? p[e] : 0.f;
  }
}

__device__ __forceinline__ double wave_sum_f64(double a) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) a += __shfl_xor(a, off, 64);
  return a;
}

// Norms next to eps or below make iterates as small, X_i <= |X_0| a^i: stored times 2^-s besides
// their usual scale, s <= 0 with 2^-s |X_0| grow in [1/2, 1) (grow = a^(steps - 1)), they stay in
// range and keep their bits.  0 for all other norms.
__device__ __forceinline__ int small_shift(double norm, double grow) {
  const double most = norm / (norm + NS_EPS) * grow;
  int s = 0;
  if (most > 0.0 && most < 1.0) frexp(most, &s);
  return s;
}

// sums of squares of chunk blockIdx.x of matrix blockIdx.y, in fp64: neither a gradient of
// 1e-30 nor one of 1e30 leaves the range
template <typename T>
__global__ __launch_bounds__(256) void k_orth_sumsq(const T* __restrict__ g, int64_t count, int64_t chunk,
                                                    double* __restrict__ part) {
  const T* p = g + (int64_t)blockIdx.y * count;
  const int64_t b = (int64_t)blockIdx.x * chunk, e = b + chunk < count ? b + chunk : count;
  double a = 0.0;
#pragma unroll 4
  for (int64_t i = b + threadIdx.x * 8; i < e; i += 256 * 8) {
    float v[8];
    load8_any(p + i, (int)(e - i < 8 ? e - i : 8), v);
#pragma unroll
    for (int q = 0; q < 8; ++q) a += (double)v[q] * (double)v[q];
  }
  a = wave_sum_f64(a);
  __shared__ double red[4];
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
  __syncthreads();
  if (threadIdx.x == 0) part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// X0 (hi, and lo for fp32 input) [m_p, l_p] of each matrix, padded with zeros, from g
// [rows, cols] (transposed when rows > cols) times 2^e, where 2^e brings the norm into
// [2^14, 2^15).  factor [3, n]: f0 = 2^-e / (norm + eps) turns stored values into X0, fi =
// 2^(s - 15) the later iterates' into X, and fx = f0 / fi those of X0 into those (s: small_shift).
// One workgroup makes 64 rows by `tiles` tiles of 64 columns.
template <typename T, bool TR>
__global__ __launch_bounds__(256) void k_orth_enter(const T* __restrict__ g, int rows, int cols,
                                                    const double* __restrict__ part, int chunks, double grow,
                                                    int mp, int lp, int tiles, f16* __restrict__ hi, uint8_t* __restrict__ lo,
                                                    float* __restrict__ factor) {
  __shared__ float tile[TR ? 64 : 1][65];
  static_assert(NORM_CHUNKS <= 64, "one lane a share");
  const int lane = threadIdx.x & 63;
  const double norm = sqrt(wave_sum_f64(lane < chunks ? part[(size_t)blockIdx.z * chunks + lane] : 0.0));
  int e = 0;
  if (norm > 0.0 && norm < 1e300) {
    frexp(norm, &e);   // norm = f 2^e, f in [1/2, 1)
    e = X_LOG2 - e;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    const double f = ldexp(1.0, -e) / (norm + NS_EPS);
    const int s = small_shift(norm, grow);
    factor[blockIdx.z] = (float)f;
    factor[gridDim.z + blockIdx.z] = (float)ldexp(f, X_LOG2 - s);
    factor[2 * gridDim.z + blockIdx.z] = (float)ldexp(1.0, s - X_LOG2);
  }
  const int tr = threadIdx.x >> 3, tc = (threadIdx.x & 7) * 8;   // rows tr, tr + 32; 8 columns
  const int r0 = blockIdx.y * 64;   // of X
  const T* p = g + (size_t)blockIdx.z * rows * cols;
  for (int ct = 0; ct < tiles; ++ct) {
    const int c0 = ((int)blockIdx.x * tiles + ct) * 64;
    if (c0 >= lp) break;
    float v[2][8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      // TR: row c0 + .. of g is column c0 + .. of X, its columns r0 + .. are X's rows
      const int r = (TR ? c0 : r0) + tr + 32 * q, c = (TR ? r0 : c0) + tc;
      load8_any(p + (size_t)r * cols + c, r < rows ? cols - c : 0, v[q]);
    }
    if (TR) {
      __syncthreads();   // the tile before has been read
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int x = 0; x < 8; ++x) tile[tc + x][tr + 32 * q] = v[q][x];
      __syncthreads();
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int x = 0; x < 8; ++x) v[q][x] = tile[tr + 32 * q][tc + x];
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const size_t o = ((size_t)blockIdx.z * mp + r0 + tr + 32 * q) * lp + c0 + tc;
      f16x8 h;
      uint64_t codes = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float s = ldexpf(v[q][x], e);
        h[x] = (f16)s;
        if (lo) codes |= (uint64_t)lo_code(s - (float)h[x]) << (8 * x);
      }
      *reinterpret_cast<f16x8*>(hi + o) = h;
      if (lo) *reinterpret_cast<uint64_t*>(lo + o) = codes;
    }
  }
}

// ---- the products ----
// What a product is for.  GRAM and POLY: a symmetric one, of which the lower triangle of tiles
// is computed and mirrored: C = c0 P P^T - diag I, and c0 P P^T + c1 P.  APPLY: X' = c0 P X +
// c1 X; LAST: the same into the result.
enum { ORTH_GRAM = 0, ORTH_POLY = 1, ORTH_APPLY = 2, ORTH_LAST = 3 };
constexpr bool orth_sym(int op) { return op <= ORTH_POLY; }

struct OrthArgs {
  int mp, lp;             // padded sizes, multiples of 64
  int K;                  // the contraction: rows of P are K long
  int m, l, rows, cols;
  const f16* p;           // [n, mp, K]
  const f16* q;           // symmetric: P; else X hi [n, mp, lp]
  float c0, c1, diag;
  f16 r1;                 // c1 / c0, which the scales make an fp16 number
  const float* factor;    // per matrix, times c0 and c1 (symmetric: its square times c0); null: 1
  f16* c;                 // symmetric: C [n, mp, mp]
  const uint8_t* xlo;     // X lo, or null
  f16* xn;                // X'
  uint8_t* xnlo;          // its lo, or null
  bf16_t* out;            // the result [n, rows, cols]
};

struct StepCoef {
  float t, alpha, beta;   // D = A - t I;  X' = alpha X + (beta D + c D^2) X
};
__host__ __device__ inline StepCoef step_coef(int step) {
  const float t = step >= SHIFT_STEP ? 1.f : 0.f;
  return {t, NS_A + NS_B * t + NS_C * t * t, NS_B + 2.f * NS_C * t};
}

// ---- the products on 256 x 256 tiles: jobs of the persistent tile stream ----
__device__ __forceinline__ f16x8 as_f16(bf16x8 v) { return __builtin_bit_cast(f16x8, v); }

typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef f16 f16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pk_f16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, (f16x2){(f16)lo, (f16)hi});
}
// trans_chunks in fp16: 16 values of a transposed accumulator block (columns 8q + 4 (l / 32)
// .. + 3 of row l % 32 in v[4q] .. v[4q + 3]) -> the row's chunks s = columns 16 s + 8 (l / 32)
// .. + 7
__device__ __forceinline__ void trans_chunks_f16(const float (&v)[16], i32x4 (&out)[2]) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    uint32_t d[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const auto r = __builtin_amdgcn_permlane32_swap(pk_f16(v[8 * s + 2 * c], v[8 * s + 2 * c + 1]),
                                                      pk_f16(v[8 * s + 4 + 2 * c], v[8 * s + 5 + 2 * c]), false, false);
      d[0][c] = r[0];
      d[1][c] = r[1];
    }
    out[s] = i32x4{(int)d[0][0], (int)d[0][1], (int)d[1][0], (int)d[1][1]};
  }
}
// and back (the swap undoes itself)
__device__ __forceinline__ void untrans_chunks_f16(const i32x4 (&ch)[2], float (&v)[16]) {
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const auto r = __builtin_amdgcn_permlane32_swap((uint32_t)ch[s][c], (uint32_t)ch[s][2 + c], false, false);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f16x2 p = __builtin_bit_cast(f16x2, (uint32_t)r[h]);
        v[8 * s + 4 * h + 2 * c] = (float)p[0];
        v[8 * s + 4 * h + 2 * c + 1] = (float)p[1];
      }
    }
}
// The lo codes of such a block: 16 codes of row l % 32, columns 16 (l / 32) .. + 15, from the
// lanes' values and back
__device__ __forceinline__ i32x4 trans_codes(const float (&rest)[16]) {
  uint32_t e[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(rest[4 * q] * LO_SCALE, rest[4 * q + 1] * LO_SCALE, 0, false);
    e[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(rest[4 * q + 2] * LO_SCALE, rest[4 * q + 3] * LO_SCALE, lo, true);
  }
  const auto s02 = __builtin_amdgcn_permlane32_swap(e[0], e[2], false, false);
  const auto s13 = __builtin_amdgcn_permlane32_swap(e[1], e[3], false, false);
  return i32x4{(int)s02[0], (int)s02[1], (int)s13[0], (int)s13[1]};
}
__device__ __forceinline__ void add_codes(const i32x4& c, float (&v)[16]) {
  const auto s02 = __builtin_amdgcn_permlane32_swap((uint32_t)c[0], (uint32_t)c[1], false, false);
  const auto s13 = __builtin_amdgcn_permlane32_swap((uint32_t)c[2], (uint32_t)c[3], false, false);
  const uint32_t e[4] = {s02[0], s13[0], s02[1], s13[1]};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)e[q], false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)e[q], true);
    v[4 * q] += a[0] * (1.f / LO_SCALE);
    v[4 * q + 1] += a[1] * (1.f / LO_SCALE);
    v[4 * q + 2] += b[0] * (1.f / LO_SCALE);
    v[4 * q + 3] += b[1] * (1.f / LO_SCALE);
  }
}

// The columns of the 32 x 64 band that band_store has just passed through the wave's LDS
// region, as rows of the transposed tile: store(column, row, chunk) gets rows row .. row + 7
// of a column.  The transposing read hands a lane four rows of its column.
template <class F>
__device__ __forceinline__ void band_columns(const bf16_t* wreg, F&& store) {
  const int lane = threadIdx.x & 63, g = lane >> 4, j = (lane >> 2) & 3, q = lane & 3;
  i32x4 v[4];
#pragma unroll
  for (int ni = 0; ni < 2; ++ni)
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int col = 32 * ni + 16 * (g & 1) + 4 * q;
      s16x4 t[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = kk * 16 + 8 * (g >> 1) + 4 * h + j;
        t[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (MOE_LDS s16x4*)(wreg + r * WCOLS + (((col >> 3) ^ band_swz<8>(r)) << 3) + (col & 7)));
      }
      __builtin_memcpy(&v[ni * 2 + kk], t, 16);
    }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the region is free for the next band
#pragma unroll
  for (int ni = 0; ni < 2; ++ni)
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) store(32 * ni + (lane & 31), kk * 16 + 8 * (lane >> 5), v[ni * 2 + kk]);
}

struct OrthTile {
  int z, i0, j0, nk;
  int cnt, ncols;   // rows and columns of the product in the tile
  float f;          // the matrix's factor
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

// TALL: the last step of matrices that were transposed on entry, whose accumulators hold C,
// so that the blocks leave as rows of C^T; all others hold C^T and leave as rows of C.
// LO: X comes with its lo.
template <int OP, bool TALL, bool LO>
struct JOrth {
  using Tile = OrthTile;
  using Ld = OrthLd;
  static constexpr bool SYM = orth_sym(OP);
  static constexpr bool A_KMAJ = true, B_KMAJ = SYM;
  static constexpr bool DYN = false, TRANS = !TALL, EPI_LDS = true, NSPLIT = false, SIDE = false;
  static constexpr bool DIAG = OP != ORTH_GRAM;
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
    p.nk = uni(a.K / BK);
    p.cnt = uni(min(BM, a.mp - p.i0));
    p.ncols = uni(min(BN, (SYM ? a.mp : a.lp) - p.j0));
    p.f = a.factor ? sload(a.factor + p.z) : 1.f;
  }
  // A diagonal tile's waves that lie above the diagonal: mirrored from those below it, which
  // leaves out two of eight (all of them computed: 3740 and 3200 us for the two batches above,
  // 3650 and 3220 so)
  __device__ __forceinline__ static bool above(const Tile& p, int wm, int wn) {
    return SYM && p.i0 == p.j0 && wn * WCOLS >= (wm + 1) * WROWS;
  }
  __device__ __forceinline__ WaveRows rows(const Tile& p, int wm) const {
    WaveRows w = wave_rows(p.cnt, wm);
    if (above(p, wm, (int)((unsigned)uni(threadIdx.x >> 6) / WM))) w.nblk = 0;
    return w;
  }
  __device__ __forceinline__ void setup(int v, Ld& p, int pw, int lane) const {
    Tile t;
    tile(v, t);
    p.pw = pw;
    p.nk = t.nk;
    const int K = a.K;
    const bf16_t* pa = reinterpret_cast<const bf16_t*>(a.p + (size_t)t.z * a.mp * K);
    const bf16_t* pb = reinterpret_cast<const bf16_t*>(a.q + (size_t)t.z * a.mp * (SYM ? K : a.lp));
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
    // Each k-step's fragments are read while the step before multiplies, one read after one
    // product: the compiler's own order read a step's fragments together and waited, 2% of the
    // whole update at 128 x 2048 x 768 (3730 us, 3650 so) and up to 1% at 16 x 1536 x 4096. Raising
    // the wave's priority around the products cost 2 to 4%.
    bf16x8 af[2][MI], bf[2][NI];
    auto frags = [&](int kk) {
#pragma unroll
      for (int ni = 0; ni < NI; ++ni)
        bf[kk & 1][ni] = B_KMAJ ? frag_kmaj(Bs, ncol(wn, ni), kk, lane) : frag_mnmaj<BN>(Bs, ncol(wn, ni), kk, lane);
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) af[kk & 1][mi] = frag_kmaj(As, w.base + mi * 32, kk, lane);
    };
    frags(0);
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      if (kk + 1 < BK / 16) frags(kk + 1);
      const bf16x8 *const fa = af[kk & 1], *const fb = bf[kk & 1];
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          acc[mi][ni] = TRANS ? __builtin_amdgcn_mfma_f32_32x32x16_f16(as_f16(fb[ni]), as_f16(fa[mi]), acc[mi][ni], 0, 0, 0)
                              : __builtin_amdgcn_mfma_f32_32x32x16_f16(as_f16(fa[mi]), as_f16(fb[ni]), acc[mi][ni], 0, 0, 0);
    }
    constexpr int READS = MI + (B_KMAJ ? NI : 2 * NI);   // of a k-step; the transposing read takes two
    constexpr int MFMA = 0x008, DS_READ = 0x100;
    __builtin_amdgcn_sched_group_barrier(DS_READ, READS, 0);
#pragma unroll
    for (int kk = 0; kk + 1 < BK / 16; ++kk)
#pragma unroll
      for (int q = 0; q < MI * NI; ++q) {
        __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
        if (q < READS) __builtin_amdgcn_sched_group_barrier(DS_READ, 1, 0);
      }
    __builtin_amdgcn_sched_group_barrier(MFMA, MI * NI, 0);
  }
  // c1 Q (P itself, or X) is part of the product: the tile's own block of Q passes through LDS
  // as the K steps of the tile's rows, where a fragment of r1 I multiplies it (P is symmetric).
  // r1 = c1 / c0 is fp16 and the sums are fp32, so nothing is rounded that an addition in the
  // epilogue would not round.  Read and added there, the block costs 8% of a product with X at
  // K = 768 (433 and 405 us, 128 of 768 x 2048) and 3% at 1536, 6% of a symmetric one.
  __device__ __forceinline__ static f16x8 scaled_identity(f16 r, int half, int lane) {   // 16 of 32 rows
    const int at = (lane & 31) - 16 * half - 8 * (lane >> 5);
    f16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e == at ? r : (f16)0.f;
    return v;
  }
  __device__ __forceinline__ void diagonal(const bf16_t* st, const Tile& p, int kc, Acc& acc, int lane, const WaveRows& w,
                                           int wn) const {
    const bf16_t* Bs = st + A_ELEMS;
    const int k0 = kc * BK;
#pragma unroll
    for (int half = 0; half < MI / 2; ++half) {   // 64 of the wave's rows
      if (k0 != p.i0 + w.base + 64 * half) continue;
      int ln = lane;
      asm volatile("" : "+v"(ln));   // its addresses are not kept in registers over the K steps
#pragma unroll
      for (int kk = 0; kk < BK / 16; ++kk) {
        const f16x8 e = scaled_identity(a.r1, kk & 1, ln);
        const int mi = 2 * half + (kk >> 1);
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
          const f16x8 b = as_f16(B_KMAJ ? frag_kmaj(Bs, ncol(wn, ni), kk, ln) : frag_mnmaj<BN>(Bs, ncol(wn, ni), kk, ln));
          acc[mi][ni] = TRANS ? __builtin_amdgcn_mfma_f32_32x32x16_f16(b, e, acc[mi][ni], 0, 0, 0)
                              : __builtin_amdgcn_mfma_f32_32x32x16_f16(e, b, acc[mi][ni], 0, 0, 0);
        }
      }
    }
  }
  __device__ __forceinline__ void epilogue(const Tile& p, const Acc& acc, float* stage) const {
    const int tid = threadIdx.x, wv = tid >> 6, wm = (int)((unsigned)wv % WM), wn = (int)((unsigned)wv / WM);
    if (wn * WCOLS >= p.ncols || above(p, wm, wn)) return;   // the tile's sizes are multiples of 64
    bf16_t* const wreg = reinterpret_cast<bf16_t*>(stage) + wv * BAND_ELEMS;
    if constexpr (TALL) out_tall(p, acc, wreg, p.i0 + wm * WROWS, p.j0 + wn * WCOLS);
    else out_rows(p, acc, wreg, p.i0 + wm * WROWS, p.j0 + wn * WCOLS);
  }
  // C^T accumulators: lane l holds row l % 32 of each band.  What the products do not hold
  // (X lo) is loaded in that layout two bands ahead; finished bands leave through the wave's LDS
  // region as whole row segments, and those of an off-diagonal tile of a symmetric product once
  // more as columns.
  __device__ __forceinline__ void out_rows(const Tile& p, const Acc& acc, bf16_t* wreg, int i0, int j0) const {
    const int lane = threadIdx.x & 63;
    const size_t xo = (size_t)p.z * a.mp * a.lp, so = (size_t)p.z * a.mp * a.mp;
    const int ld = SYM ? a.mp : a.lp;
    constexpr int AHEAD = 2;
    i32x4 xl[AHEAD][NI];
    auto fetch = [&](int mi) {
      const size_t row = (size_t)min(i0 + mi * 32 + (lane & 31), a.mp - 1) * ld + j0;
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) xl[mi % AHEAD][ni] = *reinterpret_cast<const i32x4*>(a.xlo + xo + row + ni * 32 + 16 * (lane >> 5));
    };
    if constexpr (LO) {
      fetch(0);
      fetch(1);
    }
    const float c0 = SYM ? a.c0 * p.f * p.f : a.c0 * p.f, c1 = a.c1 * p.f;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      const int rb = i0 + mi * 32;
      if (rb >= p.i0 + p.cnt) {
        // the bands already on their way: a load that is never waited for here would be waited
        // for where its registers are next written, in the K loop
        if constexpr (LO) {
#pragma unroll
          for (int k = 0; k < AHEAD && mi + k < MI; ++k)
#pragma unroll
            for (int ni = 0; ni < NI; ++ni) asm volatile("" ::"v"(xl[(mi + k) % AHEAD][ni]));
        }
        break;
      }
      i32x4 ch[NI][2], codes[NI];
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        float v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = acc[mi][ni][r] * c0;
        if constexpr (OP == ORTH_GRAM) {
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (rb + (lane & 31) == j0 + ni * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) v[r] -= a.diag;
        }
        if constexpr (LO) {
          float u[16] = {};
          add_codes(xl[mi % AHEAD][ni], u);
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] += u[r] * c1;
        }
        if constexpr (OP == ORTH_LAST) {
          f32x16 b;
#pragma unroll
          for (int r = 0; r < 16; ++r) b[r] = v[r];
          trans_chunks(b, ch[ni]);
        } else {
          trans_chunks_f16(v, ch[ni]);
        }
        if (OP == ORTH_APPLY && a.xnlo) {
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] -= (float)(f16)v[r];
          codes[ni] = trans_codes(v);
        }
      }
      if (LO && mi + AHEAD < MI) fetch(mi + AHEAD);
      if (OP == ORTH_APPLY && a.xnlo) {
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
          *reinterpret_cast<i32x4*>(a.xnlo + xo + (size_t)(rb + (lane & 31)) * ld + j0 + ni * 32 + 16 * (lane >> 5)) = codes[ni];
      }
      if constexpr (OP == ORTH_LAST) {
        bf16_t* const out = a.out + (size_t)p.z * a.rows * a.cols;
        band_store(wreg, ch, [&](int rr, int cb_, i32x4 w) {
          const int i = rb + rr, j = j0 + cb_;
          if (i >= a.m || j >= a.l) return;
          bf16_t* const q = out + (size_t)i * a.cols + j;
          if (j + 8 <= a.l) {
            *reinterpret_cast<i32x4_a2*>(q) = w;
          } else {
            for (int e = 0; e < 8; ++e)
              if (j + e < a.l) q[e] = (bf16_t)((uint32_t)w[e >> 1] >> (16 * (e & 1)));
          }
        });
      } else {
        f16* const out = SYM ? a.c + so : a.xn + xo;
        band_store(wreg, ch, [&](int rr, int cb_, i32x4 w) {
          *reinterpret_cast<i32x4*>(out + (size_t)(rb + rr) * ld + j0 + cb_) = w;
        });
        if (SYM && i0 >= j0 + WCOLS)   // off the diagonal
          band_columns(wreg, [&](int c, int r, i32x4 w) {
            *reinterpret_cast<i32x4*>(out + (size_t)(j0 + c) * ld + rb + r) = w;
          });
      }
    }
  }
  // The last step of transposed matrices: lane l holds column l % 32 of each block, and rows of
  // C^T leave.
  __device__ __forceinline__ void out_tall(const Tile& p, const Acc& acc, bf16_t* wreg, int i0, int j0) const {
    const int lane = threadIdx.x & 63;
    const size_t xo = (size_t)p.z * a.mp * a.lp;
    const float c0 = a.c0 * p.f, c1 = a.c1 * p.f;
    bf16_t* const out = a.out + (size_t)p.z * a.rows * a.cols;
#pragma unroll
    for (int ni = 0; ni < NI; ++ni)
#pragma unroll
      for (int mh = 0; mh < MI; mh += 2) {
        i32x4 ch[2][2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          f32x16 v;
#pragma unroll
          for (int r = 0; r < 16; ++r) v[r] = acc[mh + b][ni][r] * c0;
          if constexpr (LO) {   // three steps or fewer
            int ln = lane;
            asm volatile("" : "+v"(ln) : : "memory");   // one block's addresses and loads at a time
            const uint8_t* q = a.xlo + xo + (size_t)(min(i0 + (mh + b) * 32, a.mp - 32) + 4 * (ln >> 5)) * a.lp + j0 +
                               ni * 32 + (ln & 31);
#pragma unroll
            for (int r = 0; r < 16; ++r) v[r] += lo_value(q[(size_t)(8 * (r >> 2) + (r & 3)) * a.lp]) * c1;
          }
          trans_chunks(v, ch[b]);
        }
        band_store(wreg, ch, [&](int rr, int cb_, i32x4 w) {
          const int r = j0 + ni * 32 + rr, c = i0 + mh * 32 + cb_;   // of the output
          if (r >= a.l || c >= a.m) return;
          bf16_t* const o = out + (size_t)r * a.cols + c;
          if (c + 8 <= a.m) {
            *reinterpret_cast<i32x4_a2*>(o) = w;
          } else {
            for (int e = 0; e < 8; ++e)
              if (c + e < a.m) o[e] = (bf16_t)((uint32_t)w[e >> 1] >> (16 * (e & 1)));
          }
        });
      }
  }
};

template <int OP, bool TALL, bool LO>
__global__ __launch_bounds__(NTHR, 1) void k_orth_stream(OrthArgs a, int n, int tm, int tn) {
  __shared__ __attribute__((aligned(16))) bf16_t lds[LDS_ELEMS];
  JOrth<OP, TALL, LO> job{a, n, tm, tn};
  run_stream(job, lds);
}

// ---- the products on 128 x 128 and 64 x 64 tiles: one tile a workgroup ----
// For matrices whose 256-row tiles leave CUs idle or mostly padding.  The K steps ring through
// NS stages of LDS, so NS - 1 steps of direct-to-LDS loads are in flight, with one barrier a
// step: four stages where a CU gets up to two tiles, two where several workgroups on a CU cover
// each other's waits.  A step of a lone workgroup is LDS reads, the issue of the loads and the
// products in turn (0.24 us for 64 rows, the same when its data are in the nearest cache, with
// half the bytes on 32 rows, or with eight stages; three and five stages cost a division).
// Eight stages, one workgroup a CU, take 122 us for 5 of 333 x 1000 where four take 105, and
// with two tiles a CU on four stages instead of two 4 of 700 x 1500 take 179 instead of 204.
template <int TILE> struct TileCfg;
template <> struct TileCfg<64> { static constexpr int WAVES = 4, TMI = 1; };    // 2 x 2 waves of 32 x 32
template <> struct TileCfg<128> { static constexpr int WAVES = 8, TMI = 2; };   // 2 x 4 waves of 64 x 32

// MN-major rows of 64 (8 chunks): rows two apart in other halves of a row's 128 bytes, so the
// four rows of a transposing read meet no bank twice; wider rows as in the engine
template <int W>
__device__ __forceinline__ int tile_mn_chunk(int r, int c) {
  return W == 64 ? c ^ (((r >> 1) & 1) << 2) : mnmaj_chunk(r, c);
}
template <int W>
__device__ __forceinline__ f16x8 tile_frag_mn(const bf16_t* s, int base, int kk, int lane) {
  const int g = lane >> 4, j = (lane >> 2) & 3, q = lane & 3, col = base + 16 * (g & 1) + 4 * q;
  s16x4 v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = kk * 16 + 8 * (g >> 1) + 4 * h + j;
    v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(s + r * W + (tile_mn_chunk<W>(r, col >> 3) << 3) + (col & 7)));
  }
  f16x8 out;
  __builtin_memcpy(&out, v, 16);
  return out;
}

// dma16 to an LDS address that is a scalar already: a third of the instructions, which these
// launches run cold
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)((MOE_LDS const void*)p));
}
__device__ __forceinline__ void dma16_to(const void* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(lds) : "memory", "m0");
}

template <int OP, int TILE, int NS>
__global__ __launch_bounds__(64 * TileCfg<TILE>::WAVES, NS == 2 ? 4 : 1) void k_orth_tile(OrthArgs a, int tm, int tn, int items) {
  using C = TileCfg<TILE>;
  constexpr bool SYM = orth_sym(OP);
  constexpr int OPER = TILE * BK, STAGE = 2 * OPER;                  // elements
  constexpr int LP = OPER * 2 / 1024 / C::WAVES;                     // 1 KB loads of one operand a wave and step
  static_assert(LP * C::WAVES * 512 == OPER, "wave loads divide among the waves");
  __shared__ __attribute__((aligned(16))) bf16_t lds[NS * STAGE];
  const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6);
  const int per = SYM ? tm * (tm + 1) / 2 : tm * tn;
  // workgroup b runs on XCD b % 8: contiguous ranges of tiles, so that an XCD's L2 holds the
  // matrices its tiles share
  const int share = (int)(gridDim.x >> 3), v = (int)(blockIdx.x & 7) * share + (int)(blockIdx.x >> 3);
  if (v >= items) return;
  const int z = uni(v / per);
  int rem = uni(v - z * per), ti = 0;
  if (SYM) {
    while (rem > ti) rem -= ++ti;
  } else {
    ti = uni(rem % tm);
    rem = uni(rem / tm);
  }
  const int i0 = ti * TILE, j0 = rem * TILE, ldn = SYM ? a.mp : a.lp;
  const int K = a.K, nk = K / BK;
  const size_t xo = (size_t)z * a.mp * a.lp, so = (size_t)z * a.mp * a.mp;
  const bf16_t* pa = reinterpret_cast<const bf16_t*>(a.p + (size_t)z * a.mp * K);
  const bf16_t* pb = reinterpret_cast<const bf16_t*>(a.q + (SYM ? (size_t)z * a.mp * K : xo));
  const bf16_t *la[LP], *lb[LP];
#pragma unroll
  for (int q = 0; q < LP; ++q) {
    const int slot = (q * C::WAVES + wv) * 64 + lane;
    int r, c;
    kmaj_slot(slot, r, c);
    la[q] = pa + (size_t)min(i0 + r, a.mp - 1) * K + c * 8;
    if (SYM) {
      lb[q] = pb + (size_t)min(j0 + r, a.mp - 1) * K + c * 8;
    } else {
      r = slot / (TILE / 8);
      c = tile_mn_chunk<TILE>(r, slot % (TILE / 8));
      lb[q] = pb + (size_t)r * a.lp + min(j0 + c * 8, a.lp - 8);   // past the edge: any columns, not stored
    }
  }
  const size_t bstep = SYM ? (size_t)BK : (size_t)BK * a.lp;
  const uint32_t l0 = lds_address(lds) + wv * 1024;
  auto issue = [&](int kt) {
    const uint32_t st = l0 + (kt % NS) * STAGE * 2;
#pragma unroll
    for (int q = 0; q < LP; ++q) {
      dma16_to(la[q] + kt * BK, st + q * C::WAVES * 1024);
      dma16_to(lb[q] + kt * bstep, st + OPER * 2 + q * C::WAVES * 1024);
    }
  };
  const int wm = wv & 1, wn = wv >> 1, ib = wm * 32 * C::TMI, jb = wn * 32;   // the wave's first row and column
  // above the diagonal: mirrored from below.  Not in the deep ring: lone workgroups have nothing
  // to do in the time, and the branch costs more than the products (5 of 333 x 1000 105 us, 120
  // with it; in the short ring it saves 2% of 128 of 320 x 640)
  const bool above = SYM && NS == 2 && i0 == j0 && jb >= ib + 32 * C::TMI;
  f32x16 acc[C::TMI];
#pragma unroll
  for (int mi = 0; mi < C::TMI; ++mi)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[mi][r] = 0.f;
#pragma unroll 1
  for (int kt = 0; kt < min(NS - 1, nk); ++kt) issue(kt);
#pragma unroll 1
  for (int kt = 0; kt < nk; ++kt) {
    // step kt has landed when at most the NS - 2 later steps' loads are out
    if (NS > 2 && nk - 1 - kt >= NS - 2) {
      static_assert(2 * LP * (NS - 2) < 64, "vmcnt counts to 63");
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(2 * LP * (NS - 2)) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    // in the deep ring the step's fragments are asked for before a later step's loads, whose issue
    // (16 KB at 64 a clock) then passes while they come: 1 of 1024 x 1024 130 us, 125 so; several
    // workgroups on a CU fill that time themselves, and lose by the longer loop
    if (NS == 2 && kt + NS - 1 < nk) issue(kt + NS - 1);   // into the stage read one step ago
    const bf16_t* const as = lds + (kt % NS) * STAGE;
    const bf16_t* const bs = as + OPER;
    if (above) continue;
    f16x8 fa[C::TMI][BK / 16], fb[BK / 16];
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      fb[kk] = SYM ? as_f16(frag_kmaj(bs, jb, kk, lane)) : tile_frag_mn<TILE>(bs, jb, kk, lane);
#pragma unroll
      for (int mi = 0; mi < C::TMI; ++mi) fa[mi][kk] = as_f16(frag_kmaj(as, ib + mi * 32, kk, lane));
    }
    if (NS > 2 && kt + NS - 1 < nk) issue(kt + NS - 1);
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk)
#pragma unroll
      for (int mi = 0; mi < C::TMI; ++mi)
        acc[mi] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[kk], fa[mi][kk], acc[mi], 0, 0, 0);
  }
  // lane l: row l % 32 of each block, columns 8q + 4 (l / 32) .. + 3
  if (j0 + jb >= ldn || above) return;
  const float f = a.factor ? a.factor[z] : 1.f;
  const float c0 = SYM ? a.c0 * f * f : a.c0 * f, c1 = SYM ? a.c1 : a.c1 * f;
#pragma unroll
  for (int mi = 0; mi < C::TMI; ++mi) {
    const int i = i0 + ib + mi * 32 + (lane & 31), j = j0 + jb;
    if (i0 + ib + mi * 32 >= a.mp) break;
    const size_t at = (size_t)i * ldn + j;
    float v[16];
    if constexpr (OP == ORTH_GRAM) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        v[r] = acc[mi][r] * c0;
        if (i == j + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) v[r] -= a.diag;
      }
    } else {
      i32x4 ch[2];
#pragma unroll
      for (int s = 0; s < 2; ++s)
        ch[s] = *reinterpret_cast<const i32x4*>(a.q + (SYM ? so : xo) + at + 16 * s + 8 * (lane >> 5));
      untrans_chunks_f16(ch, v);
      if (!SYM && a.xlo) add_codes(*reinterpret_cast<const i32x4*>(a.xlo + xo + at + 16 * (lane >> 5)), v);
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] = acc[mi][r] * c0 + v[r] * c1;
    }
    if constexpr (OP == ORTH_LAST) {
      bf16_t* const out = a.out + (size_t)z * a.rows * a.cols;
      if (a.rows > a.cols) {   // transposed back: 32 lanes write 64 bytes of a row
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int jj = j + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
          if (i < a.m && jj < a.l) out[(size_t)jj * a.cols + i] = f2bf(v[r]);
        }
      } else {
        f32x16 b;
#pragma unroll
        for (int r = 0; r < 16; ++r) b[r] = v[r];
        i32x4 ch[2];
        trans_chunks(b, ch);
        if (i < a.m) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int jj = j + 16 * s + 8 * (lane >> 5);
            bf16_t* const q = out + (size_t)i * a.cols + jj;
            if (jj + 8 <= a.l) {
              *reinterpret_cast<i32x4_a2*>(q) = ch[s];
            } else {
              for (int e = 0; e < 8; ++e)
                if (jj + e < a.l) q[e] = (bf16_t)((uint32_t)ch[s][e >> 1] >> (16 * (e & 1)));
            }
          }
        }
      }
    } else {
      f16* const out = SYM ? a.c + so : a.xn + xo;
      i32x4 ch[2];
      trans_chunks_f16(v, ch);
#pragma unroll
      for (int s = 0; s < 2; ++s) *reinterpret_cast<i32x4*>(out + at + 16 * s + 8 * (lane >> 5)) = ch[s];
      if (SYM && (NS == 2 ? i0 + ib >= j0 + jb + 32 : i0 != j0)) {   // what no wave computes
#pragma unroll
        for (int r = 0; r < 16; ++r)
          out[(size_t)(j + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * ldn + i] = (f16)v[r];
      }
      if (OP == ORTH_APPLY && a.xnlo) {
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] -= (float)(f16)v[r];
        *reinterpret_cast<i32x4*>(a.xnlo + xo + at + 16 * (lane >> 5)) = trans_codes(v);
      }
    }
  }
}

// The tile of a product, M x N over K in n matrices (M x M by halves when symmetric): the one
// of least estimated time, from what the four kernels were measured to take on one MI355X, in
// us, for t tiles a CU and k steps of 64:
//   64 rows, deep ring    3 + max(0.24 k, t (0.8 + 0.18 k))  two share a CU, for two tiles at most
//   64 rows               3 + max(0.40 k, t (0.8 + 0.18 k))  five workgroups share a CU
//   128 rows              4 + max(0.58 k, t (1.9 + 0.70 k))  two share a CU
//   256 rows              5 + ceil(t) (7 + c k)              c = 1.25 on few CUs, 2.15 on all
// Whole updates, bf16, by this rule and with 64 deep / 64 / 128 / 256 rows throughout: 11 of 362 x
// 362 93 us and 93 / 100 / 132 / 240; 1 of 1024 x 1024 125 and 125 / 171 / 226 / 465; 4 of 700 x
// 1500 179 and 180 / 204 / 251 / 450; 8 of 768 x 2048 311 and 370 / 348 / 338 / 535; 128 of 320 x
// 640 419 and 472 / 424 / 444 / 543.
enum OrthTileKind { TILE_64_DEEP, TILE_64, TILE_128, TILE_256 };
static OrthTileKind orth_tile_kind(bool sym, int n, int M, int N, int K, double* time = nullptr) {
  const double k = K / 64.0, cus = num_cus();
  auto load = [&](int t) {
    const int64_t tm = ceil_div(M, t), tn = ceil_div(N, t);
    return n * (sym ? tm * (tm + 1) / 2 : tm * tn) / cus;
  };
  const double t64 = load(64), t128 = load(128), t256 = load(256);
  const double us[4] = {t64 <= 2.0 ? 3.0 + fmax(0.24 * k, t64 * (0.8 + 0.18 * k)) : 1e30, 3.0 + fmax(0.40 * k, t64 * (0.8 + 0.18 * k)),
                        4.0 + fmax(0.58 * k, t128 * (1.9 + 0.70 * k)),
                        5.0 + ceil(t256) * (7.0 + (1.25 + 0.9 * fmin(t256, 1.0)) * k)};
  int best = TILE_256;
  for (int i = 0; i < 3; ++i)
    if (us[i] < us[best]) best = i;
  if (time) *time = us[best];
  return (OrthTileKind)best;
}

template <int OP, int TILE, int NS>
static void orth_tiles(const char* name, const OrthArgs& a, int n, hipStream_t st) {
  constexpr bool SYM = orth_sym(OP);
  const int tm = (int)ceil_div(a.mp, TILE), tn = (int)ceil_div(a.lp, TILE);
  const int items = n * (SYM ? tm * (tm + 1) / 2 : tm * tn);
  MOE_LAUNCH(name, (k_orth_tile<OP, TILE, NS>), dim3((unsigned)(items + 7) & ~7u), dim3(64 * TileCfg<TILE>::WAVES), 0, st,
             a, tm, tn, items);
}

template <int OP, bool TALL, bool LO>
static void orth_stream(const char* name, const OrthArgs& a, int n, hipStream_t st) {
  constexpr bool SYM = orth_sym(OP);
  const int tm = (int)ceil_div(a.mp, BM), tn = (int)ceil_div(a.lp, BN);
  const dim3 grid((unsigned)grid_for((int64_t)n * (SYM ? tm * (tm + 1) / 2 : tm * tn)));
  MOE_LAUNCH(name, (k_orth_stream<OP, TALL, LO>), grid, dim3(NTHR), 0, st, a, n, tm, tn);
}
template <int OP>
static void orth_stream(const char* name, const OrthArgs& a, int n, hipStream_t st) {
  if constexpr (orth_sym(OP)) {
    orth_stream<OP, false, false>(name, a, n, st);
  } else {
    if constexpr (OP == ORTH_LAST)
      if (a.rows > a.cols) return a.xlo ? orth_stream<OP, true, true>(name, a, n, st) : orth_stream<OP, true, false>(name, a, n, st);
    a.xlo ? orth_stream<OP, false, true>(name, a, n, st) : orth_stream<OP, false, false>(name, a, n, st);
  }
}

template <int OP>
static void orth_product(const char* name, const OrthArgs& a, int n, hipStream_t st) {
  constexpr bool SYM = orth_sym(OP);
  switch (orth_tile_kind(SYM, n, a.mp, SYM ? a.mp : a.lp, a.K)) {
    case TILE_64_DEEP: return orth_tiles<OP, 64, 4>(name, a, n, st);
    case TILE_64: return orth_tiles<OP, 64, 2>(name, a, n, st);
    case TILE_128: return orth_tiles<OP, 128, 2>(name, a, n, st);
    default: break;
  }
  orth_stream<OP>(name, a, n, st);
}
// ---- small matrices: the whole iteration in one workgroup ----
// X [MP, lp] (at most SMALL_ELEMS) stays in one CU: as fp32 in the accumulator layout of its
// eight waves (so no iterate is rounded but for the products), and as fp16 in LDS beside D and
// B.  One launch instead of 2 + 3 a step, which is what bounds matrices this small: eight of
// 128 x 64, five steps, take 12.7 us and took 84 in 17 launches.
constexpr int SMALL_ELEMS = 32768, SMALL_MP = 128;
constexpr int small_lds(int mp) {   // elements: X (rows of lp + 8), D and B (rows of mp + 8)
  return SMALL_ELEMS + 8 * mp + 2 * mp * (mp + 8);
}

// NB 32 x 32 blocks of P Q^T, K-major rows of ldp and ldq in LDS, transposed in the
// accumulators; the blocks lie qs columns of it apart in one row of blocks, so that a fragment
// of P serves all of them (LDS reads are what such a step waits for)
template <int NB>
__device__ __forceinline__ void small_blocks(const f16* p, int ldp, const f16* q, int ldq, int qs, int K, int lane,
                                             f32x16 (&acc)[NB]) {
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;
  const f16 *pa = p + (lane & 31) * ldp + 8 * (lane >> 5), *pb = q + (lane & 31) * ldq + 8 * (lane >> 5);
#pragma unroll 4
  for (int k = 0; k < K; k += 16) {
    const f16x8 pf = *reinterpret_cast<const f16x8*>(pa + k);
#pragma unroll
    for (int b = 0; b < NB; ++b)
      acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*reinterpret_cast<const f16x8*>(pb + b * qs * ldq + k), pf, acc[b], 0, 0, 0);
  }
}
// the same of B X, at xo[b] columns of it: X as it lies, [K][ldx], through the transposing
// read; TALL: not transposed in the accumulators
template <int NB, bool TALL>
__device__ __forceinline__ void small_blocks_x(const f16* p, int ldp, const f16* x, int ldx, const int (&xo)[NB], int K,
                                               int lane, f32x16 (&acc)[NB]) {
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;
  const f16* pa = p + (lane & 31) * ldp + 8 * (lane >> 5);
  const int g = lane >> 4, j = (lane >> 2) & 3, q = lane & 3;
  const f16* px = x + (8 * (g >> 1) + j) * ldx + 16 * (g & 1) + 4 * q;
#pragma unroll 2
  for (int k = 0; k < K; k += 16) {
    const f16x8 pf = *reinterpret_cast<const f16x8*>(pa + k);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      s16x4 t[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        t[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(px + (k + 4 * h) * ldx + xo[b]));
      f16x8 xf;
      __builtin_memcpy(&xf, t, 16);
      acc[b] = TALL ? __builtin_amdgcn_mfma_f32_32x32x16_f16(pf, xf, acc[b], 0, 0, 0)
                    : __builtin_amdgcn_mfma_f32_32x32x16_f16(xf, pf, acc[b], 0, 0, 0);
    }
  }
}
// four elements at p, at any element's address
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef i32x2 i32x2_a2 __attribute__((aligned(2)));
__device__ __forceinline__ f32x4 load4(const bf16_t* p) {
  const i32x2 u = *reinterpret_cast<const i32x2_a2*>(p);
  return f32x4{__uint_as_float((uint32_t)u[0] << 16), __uint_as_float((uint32_t)u[0] & 0xffff0000u),
               __uint_as_float((uint32_t)u[1] << 16), __uint_as_float((uint32_t)u[1] & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 load4(const float* p) {
  const i32x4 u = *reinterpret_cast<const i32x4_a4*>(p);
  return f32x4{__uint_as_float((uint32_t)u[0]), __uint_as_float((uint32_t)u[1]), __uint_as_float((uint32_t)u[2]),
               __uint_as_float((uint32_t)u[3])};
}

// 16 values in the transposed accumulator layout -> the block at dst, rows of ld
__device__ __forceinline__ void small_put(f16* dst, int ld, const float (&v)[16], int lane) {
  f16* const row = dst + (lane & 31) * ld + 4 * (lane >> 5);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<f16x4*>(row + 8 * q) = f16x4{(f16)v[4 * q], (f16)v[4 * q + 1], (f16)v[4 * q + 2], (f16)v[4 * q + 3]};
}

// ---- few rows: a step's square matrices in one workgroup ----
// With m at most 128 a matrix's squares fit in one CU's LDS, so one launch makes A of X, passed
// through a ring of K steps that serves as both factors, and of it B: 2 launches a step in place
// of 3.  What is left is the K steps of a lone CU (0.2 us a step of 64 rows, 0.4 of 128, most of
// it LDS reads) and 4 to 6 us a launch.  A by the lower triangle alone, a wave a 16-deep slice of
// K (a third of the LDS reads, but shares to join), was slower up to K = 4096 at 128 rows, and
// faster past 2048 at 64.
struct SquareArgs {
  const f16* x;          // [n, MP, K]
  int K;
  const float* factor;   // per matrix, stored X -> X
  float c0, diag;        // D = c0 X X^T - diag I
  float sq, lin;         // B = sq D^2 + lin D
  f16* out;              // B [n, MP, MP]
};
template <int MP>
__global__ __launch_bounds__(NTHR, 1) void k_orth_square(SquareArgs a) {
  constexpr int NS = 4, OPER = MP * BK, LP = OPER * 2 / 1024 / NW;   // 1 KB loads a wave and K step
  static_assert(LP * NW * 512 == OPER && LP * (NS - 2) < 64, "wave loads divide among the waves");
  constexpr int LDM = MP + 8, RB = MP / 32, BLOCKS = RB * RB;
  constexpr int SB = BLOCKS > NW ? BLOCKS / NW : 1;       // 32 x 32 blocks a wave
  constexpr int SPLIT = BLOCKS < NW ? NW / BLOCKS : 1;    // waves that share a block's K steps
  constexpr int MAT = MP * LDM, SHARES = BLOCKS * 1024 * 2 * (SPLIT - 1);   // fp32, behind D
  constexpr int ELEMS = NS * OPER > MAT + SHARES ? NS * OPER : MAT + SHARES;
  __shared__ __attribute__((aligned(16))) f16 lds[ELEMS];
  const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6), w = wv % BLOCKS, part = wv / BLOCKS;
  const int bi = w % RB * 32, bj0 = w / RB * 32;
  constexpr int BSTEP = NW / RB * 32;   // columns from one of a wave's blocks to the next
  const size_t z = blockIdx.x;
  const int K = a.K, nk = K / BK;
  const bf16_t* la[LP];
#pragma unroll
  for (int q = 0; q < LP; ++q) {
    int r, c;
    kmaj_slot((q * NW + wv) * 64 + lane, r, c);
    la[q] = reinterpret_cast<const bf16_t*>(a.x) + (z * MP + r) * K + c * 8;
  }
  const bf16_t* const ring = reinterpret_cast<const bf16_t*>(lds);
  const uint32_t l0 = lds_address(lds) + wv * 1024;
  auto issue = [&](int kt) {
#pragma unroll
    for (int q = 0; q < LP; ++q) dma16_to(la[q] + kt * BK, l0 + (kt % NS) * OPER * 2 + q * NW * 1024);
  };
  f32x16 acc[SB];
#pragma unroll
  for (int b = 0; b < SB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[b][r] = 0.f;
#pragma unroll 1
  for (int kt = 0; kt < min(NS - 1, nk); ++kt) issue(kt);
#pragma unroll 1
  for (int kt = 0; kt < nk; ++kt) {
    // step kt has landed when at most the NS - 2 later steps' loads are out
    if (nk - 1 - kt >= NS - 2) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LP * (NS - 2)) : "memory");
    else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const bf16_t* const st = ring + (kt % NS) * OPER;
    constexpr int KS = BK / 16 / SPLIT;
    f16x8 pf[KS], qf[SB][KS];   // before the loads at 64 rows, as in k_orth_tile; at 128, LDS is busy all the time
    if (MP == 128 && kt + NS - 1 < nk) issue(kt + NS - 1);   // into the stage read one step ago
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      pf[k] = as_f16(frag_kmaj(st, bi, part * KS + k, lane));
#pragma unroll
      for (int b = 0; b < SB; ++b) qf[b][k] = as_f16(frag_kmaj(st, bj0 + b * BSTEP, part * KS + k, lane));
    }
    if (MP == 64 && kt + NS - 1 < nk) issue(kt + NS - 1);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int b = 0; b < SB; ++b) acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(qf[b][k], pf[k], acc[b], 0, 0, 0);
  }
  __syncthreads();   // the ring's space is D's from here on
  if constexpr (SPLIT > 1) {
    float* const share = reinterpret_cast<float*>(lds + MAT) + w * 1024 + lane;
    static_assert(SPLIT == 2, "one share a block");
    if (part == 1) {
#pragma unroll
      for (int r = 0; r < 16; ++r) share[r * 64] = acc[0][r];
    }
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[0][r] += share[r * 64];
    }
  }
  // blocks in this wave's layout: lane l holds row bi + l % 32, columns 8 q + 4 (l / 32) .. + 3 of
  // each
  const bool on = part == 0;
  f16* const d = lds;
  const float f = a.factor[z], c0 = a.c0 * f * f;
  if (on) {
#pragma unroll
    for (int b = 0; b < SB; ++b) {
      const int bj = bj0 + b * BSTEP;
      float v[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] = acc[b][r] * c0;
      if (bi == bj) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if ((lane & 31) == 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) v[r] -= a.diag;
      }
      small_put(d + bi * LDM + bj, LDM, v, lane);
    }
  }
  __syncthreads();
  if (!on) return;
  small_blocks<SB>(d + bi * LDM, LDM, d + bj0 * LDM, LDM, BSTEP, MP, lane, acc);
#pragma unroll
  for (int b = 0; b < SB; ++b) {
    const int bj = bj0 + b * BSTEP;
    float v[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f16x4 u = *reinterpret_cast<const f16x4*>(d + (bi + (lane & 31)) * LDM + bj + 8 * q + 4 * (lane >> 5));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] = acc[b][4 * q + e] * a.sq + (float)u[e] * a.lin;
    }
    i32x4 ch[2];
    trans_chunks_f16(v, ch);
    f16* const o = a.out + (z * MP + bi + (lane & 31)) * MP + bj + 8 * (lane >> 5);
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<i32x4*>(o + 16 * h) = ch[h];
  }
}

// XB: 32 x 32 blocks of X a wave, 1, 2 or 4 (one launch runs its code cold: the instructions
// of blocks that are not there cost more than the work of those that are).  TALL: rows > cols.
// A lane holds 16 elements of one row of g in each block, four at a time side by side, so of a
// row of X or, TALL, of a column (read element by element across g, 128 x 64 took 13.4 us
// where 64 x 128 took 12.2).
template <typename T, int MP, int XB, bool TALL>
__global__ __launch_bounds__(NTHR, 1) void k_orth_small(const T* g, bf16_t* out, int rows, int cols, int lp,
                                                        int steps, double grow, float scale) {
  __shared__ __attribute__((aligned(16))) f16 small[small_lds(MP)];
  __shared__ double red[NW];
  constexpr int LDM = MP + 8, RB = MP / 32;
  constexpr int SB = RB * RB > NW ? RB * RB / NW : 1;   // blocks of D and B a wave
  const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6), ldx = lp + 8;
  f16* const xs = small;
  f16* const ds = xs + MP * ldx;
  f16* const bs = ds + MP * LDM;
  const int nb = RB * (lp / 32);
  // of block blk: the lane's row of g, and its first column
  auto g_row = [&](int blk) { return (TALL ? blk / RB : blk % RB) * 32 + (lane & 31); };
  auto g_col = [&](int blk) { return (TALL ? blk % RB : blk / RB) * 32 + 4 * (lane >> 5); };
  const size_t base = (size_t)blockIdx.x * rows * cols;
  float x[XB][16];
  double ss = 0.0;
#pragma unroll
  for (int b = 0; b < XB; ++b) {
    const int blk = wv + NW * b, i = g_row(blk), j0 = g_col(blk);
    const T* const row = g + base + (size_t)i * cols;
    const bool in = blk < nb && i < rows;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = j0 + 8 * q;
      if (in && j + 4 <= cols) {
        const f32x4 u = load4(row + j);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[b][4 * q + c] = u[c];
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) x[b][4 * q + c] = in && j + c < cols ? elem<T>::load(row + j + c) : 0.f;
      }
    }
  }
#pragma unroll
  for (int b = 0; b < XB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) ss += (double)x[b][r] * (double)x[b][r];
  ss = wave_sum_f64(ss);
  if (lane == 0) red[wv] = ss;
  __syncthreads();
  ss = 0.0;
#pragma unroll
  for (int w = 0; w < NW; ++w) ss += red[w];
  const double norm = sqrt(ss);
  int e = 0;
  if (norm > 0.0 && norm < 1e300) {
    frexp(norm, &e);
    e = -e;
  }
  // X 2^(15 - sh), as in LDS (sh: small norms, as in k_orth_enter); through 2^e: no factor leaves
  // fp32's range
  const int sh = small_shift(norm, grow);
  const float f = (float)ldexp(1.0 / (norm + NS_EPS), X_LOG2 - sh - e);
  const float dscale = ldexpf(D_SCALE, 2 * (sh - X_LOG2));
#pragma unroll
  for (int b = 0; b < XB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) x[b][r] = ldexpf(x[b][r], e) * f;
  for (int step = 0; step < steps; ++step) {
    const StepCoef co = step_coef(step);
#pragma unroll
    for (int b = 0; b < XB; ++b) {
      const int blk = wv + NW * b;
      f16* const dst = xs + (blk % RB) * 32 * ldx + (blk / RB) * 32;
      if (blk >= nb) continue;
      if constexpr (TALL) {
        int ln = lane;
        asm volatile("" : "+v"(ln));   // its 16 addresses are not kept over the steps
#pragma unroll
        for (int r = 0; r < 16; ++r) dst[(8 * (r >> 2) + 4 * (ln >> 5) + (r & 3)) * ldx + (ln & 31)] = (f16)x[b][r];
      } else {
        small_put(dst, ldx, x[b], lane);
      }
    }
    __syncthreads();
    // a wave's blocks of D and B, and of X, share a row of blocks: NW is a multiple of RB
    static_assert(NW % RB == 0, "block rows");
    const int bi = wv % RB * 32, bj0 = wv / RB * 32;
    if (wv < RB * RB) {
      f32x16 acc[SB];
      small_blocks<SB>(xs + bi * ldx, ldx, xs + bj0 * ldx, ldx, NW / RB * 32, lp, lane, acc);
#pragma unroll
      for (int b = 0; b < SB; ++b) {
        const int bj = bj0 + b * (NW / RB) * 32;
        float v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = acc[b][r] * dscale;
        if (bi == bj) {
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if ((lane & 31) == 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) v[r] -= co.t * D_SCALE;
        }
        small_put(ds + bi * LDM + bj, LDM, v, lane);
      }
    }
    __syncthreads();
    if (wv < RB * RB) {
      f32x16 acc[SB];
      small_blocks<SB>(ds + bi * LDM, LDM, ds + bj0 * LDM, LDM, NW / RB * 32, MP, lane, acc);
#pragma unroll
      for (int b = 0; b < SB; ++b) {
        const int bj = bj0 + b * (NW / RB) * 32;
        float v[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f16x4 d = *reinterpret_cast<const f16x4*>(ds + (bi + (lane & 31)) * LDM + bj + 8 * q + 4 * (lane >> 5));
#pragma unroll
          for (int c = 0; c < 4; ++c)
            v[4 * q + c] = acc[b][4 * q + c] * (NS_C * B_SCALE / (D_SCALE * D_SCALE)) + (float)d[c] * (co.beta * B_SCALE / D_SCALE);
        }
        small_put(bs + bi * LDM + bj, LDM, v, lane);
      }
    }
    __syncthreads();
    {
      f32x16 acc[XB];
      int xo[XB];   // a block past the last reads the wave's first again; its x goes nowhere
#pragma unroll
      for (int b = 0; b < XB; ++b) xo[b] = wv + NW * b < nb ? b * (NW / RB) * 32 : 0;
      if (wv < nb) {
        small_blocks_x<XB, TALL>(bs + bi * LDM, LDM, xs + wv / RB * 32, ldx, xo, MP, lane, acc);
#pragma unroll
        for (int b = 0; b < XB; ++b)
#pragma unroll
          for (int r = 0; r < 16; ++r) x[b][r] = x[b][r] * co.alpha + acc[b][r] * (1.f / B_SCALE);
      }
    }
    __syncthreads();   // xs, ds and bs have been read
  }
  scale *= ldexpf(1.f, sh - X_LOG2);
#pragma unroll
  for (int b = 0; b < XB; ++b) {
    const int blk = wv + NW * b, i = g_row(blk), j0 = g_col(blk);
    bf16_t* const row = out + base + (size_t)i * cols;
    if (blk >= nb || i >= rows) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = j0 + 8 * q;
      if (j + 4 <= cols) {
        *reinterpret_cast<i32x2_a2*>(row + j) =
            i32x2{(int)pk_bf16(x[b][4 * q] * scale, x[b][4 * q + 1] * scale),
                  (int)pk_bf16(x[b][4 * q + 2] * scale, x[b][4 * q + 3] * scale)};
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (j + c < cols) row[j + c] = f2bf(x[b][4 * q + c] * scale);
      }
    }
  }
}

// what the last stored iterate is of X_0 at most
inline double growth(int steps) { return pow((double)NS_A, steps - 1); }

inline bool orth_small(int mp, int lp) { return mp <= SMALL_MP && mp * lp <= SMALL_ELEMS; }

template <typename T, int MP, bool TALL>
static hipError_t launch_small(const moe_orth_shape& s, const T* g, bf16_t* o, int lp, float scale, hipStream_t st) {
  const dim3 grid((unsigned)s.n), block(NTHR);
  const int blocks = (int)ceil_div(MP / 32 * (lp / 32), NW);
  const double grow = growth(s.steps);
#define CALL(XB) \
  MOE_LAUNCH("orth_small", (k_orth_small<T, MP, XB, TALL>), grid, block, 0, st, g, o, s.rows, s.cols, lp, s.steps, grow, scale)
  if (blocks == 1) CALL(1);
  else if (blocks == 2) CALL(2);
  else CALL(4);
#undef CALL
  return hipGetLastError();
}
template <typename T>
static hipError_t launch_small(const moe_orth_shape& s, const T* g, bf16_t* o, int mp, int lp, float scale,
                               hipStream_t st) {
  if (s.rows > s.cols)
    return mp == 64 ? launch_small<T, 64, true>(s, g, o, lp, scale, st) : launch_small<T, 128, true>(s, g, o, lp, scale, st);
  return mp == 64 ? launch_small<T, 64, false>(s, g, o, lp, scale, st) : launch_small<T, 128, false>(s, g, o, lp, scale, st);
}

// The scale next to `scale` with which k * scale is an fp16 number
inline float fit_scale(float k, float scale) { return (float)(f16)(k * scale) / k; }

inline int pad64(int v) { return (v + 63) & ~63; }

}  // namespace

// Whether a step's squares are made by k_orth_square (mp <= 128).  A lone workgroup takes
// 0.2 or 0.42 us a K step, so the products by tiles win where K is long and matrices are few:
// whole updates of five steps, squares in one launch / by tiles, 5 of 64 x 1024 51 / 64 us, 100
// of them 89 / 105, 1 of 64 x 4096 93 / 112, 400 of 64 x 1024 212 / 228, 2 of 128 x 512 57 / 61,
// 1 of 128 x 1500 89 / 81, 16 of 128 x 768 77 / 68, 128 of 96 x 1024 163 / 174, 300 of 128 x 600
// 271 / 266, 520 of them 436 / 473, 1 of 96 x 4096 166 / 125; 128 of 128 x 4096, 687 / 729, is on
// the wrong side.  Estimated time of a step's squares, in us, with two workgroups a CU for 64
// rows and one for 128; the factor is the launch that the tiles need more.
static bool square_pays(int n, int mp, int lp) {
  if (mp > 128) return false;
  double gram, poly;
  orth_tile_kind(true, n, mp, mp, lp, &gram);
  orth_tile_kind(true, n, mp, mp, mp, &poly);
  const double k = lp / 64.0, rounds = ceil(n / ((mp == 64 ? 2.0 : 1.0) * num_cus()));
  return rounds * (mp == 64 ? 4.0 + 0.20 * k : 6.0 + 0.42 * k) <= 1.15 * (gram + poly);
}
// Scratch: norm shares and factors, then X (two iterates, hi and lo), and the square matrices, D
// and B of a step
struct OrthLayout {
  int m, l, mp, lp, chunks;
  bool square;   // k_orth_square, whose D stays in LDS
  size_t off_part, off_factor, off_x[2], off_lo[2], off_s[2], bytes;
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
  if (orth_small(L.mp, L.lp)) return L;   // no scratch
  L.off_part = take((size_t)s.n * L.chunks * 8);
  L.off_factor = take((size_t)s.n * 4 * 3);
  for (int i = 0; i < 2; ++i) {
    L.off_x[i] = take(xb);
    L.off_lo[i] = take(xb / 2);
  }
  L.square = square_pays(s.n, L.mp, L.lp);
  for (int i = 0; i < (L.square ? 1 : 2); ++i) L.off_s[i] = take(db);
  L.bytes = off;
  return L;
}
size_t orth_scratch_bytes(const moe_orth_shape& s) { return orth_layout(s).bytes; }

template <typename T>
static void orth_enter(const moe_orth_shape& s, const OrthLayout& L, const T* g, char* ws, hipStream_t st) {
  const int64_t count = (int64_t)s.rows * s.cols;
  const int64_t chunk = ceil_div(ceil_div(count, L.chunks), 8) * 8;
  double* part = reinterpret_cast<double*>(ws + L.off_part);
  float* factor = reinterpret_cast<float*>(ws + L.off_factor);
  f16* hi = reinterpret_cast<f16*>(ws + L.off_x[0]);
  uint8_t* lo = s.dtype == MOE_F32 ? reinterpret_cast<uint8_t*>(ws + L.off_lo[0]) : nullptr;
  MOE_LAUNCH("orth_sumsq", k_orth_sumsq<T>, dim3((unsigned)L.chunks, (unsigned)s.n), dim3(256), 0, st, g, count, chunk,
             part);
  const double grow = growth(s.steps);
  // up to 8 tiles a workgroup (the norm's shares are read once for them) where that leaves
  // 4096 workgroups
  const int64_t all = (int64_t)s.n * (L.lp / 64) * (L.mp / 64);
  const int tiles = (int)(all < 4096 ? 1 : all > 8 * 4096 ? 8 : all / 4096);
  const dim3 grid((unsigned)ceil_div(L.lp / 64, tiles), (unsigned)(L.mp / 64), (unsigned)s.n);
  if (s.rows > s.cols)
    MOE_LAUNCH("orth_enter", (k_orth_enter<T, true>), grid, dim3(256), 0, st, g, s.rows, s.cols, part, L.chunks, grow,
               L.mp, L.lp, tiles, hi, lo, factor);
  else
    MOE_LAUNCH("orth_enter", (k_orth_enter<T, false>), grid, dim3(256), 0, st, g, s.rows, s.cols, part, L.chunks, grow,
               L.mp, L.lp, tiles, hi, lo, factor);
}

hipError_t launch_orthogonalize(const moe_orth_shape& s, const void* g, void* o, float scale, void* scratch,
                                hipStream_t st) {
  const OrthLayout L = orth_layout(s);
  if (orth_small(L.mp, L.lp))
    return s.dtype == MOE_BF16 ? launch_small(s, (const bf16_t*)g, (bf16_t*)o, L.mp, L.lp, scale, st)
                               : launch_small(s, (const float*)g, (bf16_t*)o, L.mp, L.lp, scale, st);
  char* ws = reinterpret_cast<char*>(scratch);
  if (s.dtype == MOE_BF16) orth_enter(s, L, (const bf16_t*)g, ws, st);
  else orth_enter(s, L, (const float*)g, ws, st);
  f16* const x[2] = {reinterpret_cast<f16*>(ws + L.off_x[0]), reinterpret_cast<f16*>(ws + L.off_x[1])};
  uint8_t* const xlo[2] = {reinterpret_cast<uint8_t*>(ws + L.off_lo[0]), reinterpret_cast<uint8_t*>(ws + L.off_lo[1])};
  f16* const sq[2] = {reinterpret_cast<f16*>(ws + L.off_s[0]), reinterpret_cast<f16*>(ws + L.off_s[1])};
  OrthArgs base{};
  base.mp = L.mp; base.lp = L.lp; base.m = L.m; base.l = L.l; base.rows = s.rows; base.cols = s.cols;
  base.out = (bf16_t*)o;
  const float *f0 = reinterpret_cast<const float*>(ws + L.off_factor), *fx = f0 + s.n, *fi = fx + s.n;
  int cur = 0;                              // X's buffer
  bool has_lo = s.dtype == MOE_F32;
  int los = LO_STEPS;                       // iterates still to be kept with their lo
  // D = A - t I of the current X, and B = beta D + c D^2
  auto gram = [&](f16* d, float ds, float t, const float* f) {
    OrthArgs a = base;
    a.p = a.q = x[cur]; a.K = L.lp; a.c = d;
    a.c0 = ds;
    a.diag = t * ds;
    a.factor = f;
    orth_product<ORTH_GRAM>("orth_gram", a, s.n, st);
  };
  auto poly = [&](const f16* d, float ds, f16* b, float bs, float beta) {
    OrthArgs a = base;
    a.p = a.q = d; a.K = L.mp; a.c = b;
    a.c0 = NS_C * bs / (ds * ds);
    a.c1 = beta * bs / ds;
    a.r1 = (f16)(a.c1 / a.c0);
    orth_product<ORTH_POLY>("orth_poly", a, s.n, st);
  };
  // X <- alpha X + P X (P at p_scale); the last one into the result
  auto apply = [&](const f16* p, float p_scale, float alpha, const float* f, bool last) {
    OrthArgs a = base;
    const float out = last ? scale : 1.f;
    a.p = p; a.q = x[cur]; a.K = L.mp;
    a.c0 = out / p_scale;
    a.c1 = out * alpha;
    a.r1 = (f16)(alpha * p_scale);
    a.factor = f;
    a.xlo = has_lo ? xlo[cur] : nullptr;
    has_lo = los-- > 0;
    a.xn = x[cur ^ 1];
    a.xnlo = has_lo ? xlo[cur ^ 1] : nullptr;
    if (last) orth_product<ORTH_LAST>("orth_last", a, s.n, st);
    else orth_product<ORTH_APPLY>("orth_apply", a, s.n, st);
    cur ^= 1;
  };
  auto square = [&](f16* b, float ds, float t, float bs, float beta, const float* f) {
    SquareArgs a{};
    a.x = x[cur]; a.K = L.lp; a.factor = f; a.out = b;
    a.c0 = ds;
    a.diag = t * ds;
    a.sq = NS_C * bs / (ds * ds);
    a.lin = beta * bs / ds;
    const dim3 grid((unsigned)s.n), block(NTHR);
    if (L.mp == 64) {
      MOE_LAUNCH("orth_square", k_orth_square<64>, grid, block, 0, st, a);
    } else {
      MOE_LAUNCH("orth_square", k_orth_square<128>, grid, block, 0, st, a);
    }
  };
  for (int step = 0; step < s.steps; ++step) {
    const StepCoef co = step_coef(step);
    const bool last = step == s.steps - 1;
    const float* const f = step == 0 ? f0 : fi;   // the stored X -> X
    const float ds = fit_scale(co.beta / NS_C, D_SCALE), bs = fit_scale(co.alpha, B_SCALE);
    f16* const b = L.square ? sq[0] : sq[1];
    if (L.square) {
      square(b, ds, co.t, bs, co.beta, f);
    } else {
      gram(sq[0], ds, co.t, f);
      poly(sq[0], ds, b, bs, co.beta);
    }
    apply(b, bs, co.alpha, last ? f : step == 0 ? fx : nullptr, last);
  }
  return hipGetLastError();
}

}  // namespace moe
