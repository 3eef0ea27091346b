// Matrix product with bias, activation and residual in its epilogue, and its backward.
//
//   z = x W + b,  y = act(z) + res
//   dz = dy act'(z),  dx = dx_in + dz W^T,  dW = x^T dz,  db = sum_t dz
// with x [T, K], W [K, N] as the layer's weights are stored, sums in fp32.  z is kept in the
// data's type for the backward; y is formed from the fp32 sum.
#include "linear.h"

namespace moe {

namespace {

// ---------------- any size, any alignment ----------------
// 64 x 64 tiles of four waves, K steps of 32 staged element by element through registers: two
// steps' loads are under way while one is multiplied, one barrier a step.  With few tiles K is split, and the
// shares, fp32 [share, M, N], are added in order by a second launch with the epilogue.
constexpr int GTILE = 64, GSTEP = 32;

template <typename T> struct gstage;
template <> struct gstage<bf16_t> { static constexpr int LD = GSTEP + 8; };
template <> struct gstage<float> { static constexpr int LD = GSTEP + 1; };

// C [M, N] = A B over K.  A element (m, k) at m * am + k * ak, B element (k, n) at k * bk + n * bn;
// of each pair of strides one is 1.
template <typename T>
struct GeneralArgs {
  const T* a;
  const T* b;
  int64_t am, ak, bk, bn;
  int64_t M, N, K;
  int64_t ks;     // of K a share, a multiple of GSTEP
  float* part;    // or null: one share
  Epilogue<T> e;
};

template <typename T>
__global__ __launch_bounds__(256) void k_linear_any(GeneralArgs<T> g) {
  constexpr int LD = gstage<T>::LD;
  __shared__ __attribute__((aligned(16))) T as[2][GTILE][LD];   // [m][k]
  __shared__ __attribute__((aligned(16))) T bs[2][GTILE][LD];   // [n][k]
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t m0 = (int64_t)blockIdx.x * GTILE, n0 = (int64_t)blockIdx.y * GTILE, k0 = blockIdx.z * g.ks;
  const int64_t k1 = min(g.K, k0 + g.ks);
  const int wm = (wv & 1) * 32, wn = (wv >> 1) * 32;
  // neighbouring threads along the axis that is contiguous: the thread's first place, and what
  // each of its eight further ones adds
  const bool ka = g.ak == 1, kb = g.bk == 1;
  const int am = ka ? tid >> 5 : tid & 63, ak = ka ? tid & 31 : tid >> 6, dam = ka ? 8 : 0, dak = ka ? 0 : 4;
  const int bn = kb ? tid >> 5 : tid & 63, bk = kb ? tid & 31 : tid >> 6, dbn = kb ? 8 : 0, dbk = kb ? 0 : 4;
  // offsets within a step from its (uniform) first element; rows past the end give way to the
  // last one, their results are discarded
  const int mm = (int)min(g.M - 1 - m0, (int64_t)GTILE), nm = (int)min(g.N - 1 - n0, (int64_t)GTILE);
  uint32_t oa[8], ob[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    oa[q] = (uint32_t)min(am + q * dam, mm) * (uint32_t)g.am + (uint32_t)(ak + q * dak) * (uint32_t)g.ak;
    ob[q] = (uint32_t)min(bn + q * dbn, nm) * (uint32_t)g.bn + (uint32_t)(bk + q * dbk) * (uint32_t)g.bk;
  }
  const T* pa = g.a + m0 * g.am + k0 * g.ak;
  const T* pb = g.b + k0 * g.bk + n0 * g.bn;
  f32x16 acc;
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = 0.f;
  T ra[2][8], rb[2][8];   // of two steps ahead
  auto load = [&](int left, T (&a)[8], T (&b)[8]) {   // left: of K from the step on
    if (left >= GSTEP) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        a[q] = pa[oa[q]];
        b[q] = pb[ob[q]];
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        a[q] = ak + q * dak < left ? pa[oa[q]] : (T)0;
        b[q] = bk + q * dbk < left ? pb[ob[q]] : (T)0;
      }
    }
    pa += GSTEP * g.ak;
    pb += GSTEP * g.bk;
  };
  const int len = (int)(k1 - k0);
  if (len > 0) load(len, ra[0], rb[0]);
  if (len > GSTEP) load(len - GSTEP, ra[1], rb[1]);
  for (int k2 = 0; k2 < len; k2 += 2 * GSTEP)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = k2 + c * GSTEP;
      if (k >= len) break;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        as[c][am + q * dam][ak + q * dak] = ra[c][q];
        bs[c][bn + q * dbn][bk + q * dbk] = rb[c][q];
      }
      __syncthreads();   // the other stage's readers are past it: they have met this barrier since
      if (k + 2 * GSTEP < len) load(len - k - 2 * GSTEP, ra[c], rb[c]);
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int kk = 0; kk < GSTEP; kk += 16) {
          const int i = kk + (lane >> 5) * 8;
          acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8*>(&as[c][wm + (lane & 31)][i]),
                                                        *reinterpret_cast<const bf16x8*>(&bs[c][wn + (lane & 31)][i]),
                                                        acc, 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < GSTEP; kk += 2) {
          const int i = kk + (lane >> 5);
          acc = __builtin_amdgcn_mfma_f32_32x32x2f32(as[c][wm + (lane & 31)][i], bs[c][wn + (lane & 31)][i], acc, 0, 0,
                                                     0);
        }
      }
    }
  const int64_t n = n0 + wn + (lane & 31);
  if (n >= g.N) return;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int64_t m = m0 + wm + 8 * (j >> 2) + 4 * (lane >> 5) + (j & 3);
    if (m >= g.M) continue;
    if (g.part) g.part[(blockIdx.z * g.M + m) * g.N + n] = acc[j];
    else g.e.store(m, n, g.N, acc[j]);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_linear_any_join(GeneralArgs<T> g, int splits) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, size = g.M * g.N;
  if (i >= size) return;
  float s = 0.f;
#pragma unroll 4
  for (int sp = 0; sp < splits; ++sp) s += g.part[sp * size + i];
  g.e.store(i / g.N, i % g.N, g.N, s);
}

// shares of K: two workgroups for each CU, of four steps at least
int general_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ceil_div(M, GTILE) * ceil_div(N, GTILE);
  if (tiles == 0) return 1;
  int64_t s = 2 * gemm_cus() / tiles;
  s = s < K / (4 * GSTEP) ? s : K / (4 * GSTEP);
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}
size_t general_part_bytes(int64_t M, int64_t N, int64_t K) {
  const int s = general_splits(M, N, K);
  return s == 1 ? 0 : (size_t)s * M * N * 4;
}

template <typename T>
hipError_t general(const char* name, const T* a, const T* b, int64_t am, int64_t ak, int64_t bk, int64_t bn, int64_t M,
                   int64_t N, int64_t K, const Epilogue<T>& e, float* part, hipStream_t st) {
  if (M == 0 || N == 0) return hipSuccess;
  int splits = general_splits(M, N, K);
  const int64_t ks = ceil_div(ceil_div(K, splits), GSTEP) * GSTEP;
  splits = ks > 0 ? (int)ceil_div(K, ks) : 1;
  const GeneralArgs<T> g{a, b, am, ak, bk, bn, M, N, K, ks, splits > 1 ? part : nullptr, e};
  MOE_LAUNCH(name, k_linear_any<T>,
             dim3((unsigned)ceil_div(M, GTILE), (unsigned)ceil_div(N, GTILE), (unsigned)splits), dim3(256), 0, st, g);
  if (splits > 1)
    MOE_LAUNCH("linear_join", k_linear_any_join<T>, dim3((unsigned)ceil_div(M * N, 256)), dim3(256), 0, st, g, splits);
  return hipGetLastError();
}

// ---------------- few rows ----------------
// Up to FEW rows (the tokens of a decode step): W is read once, and that is what counts.  A
// workgroup takes 16 columns, two lanes of 8, and all of K, 256 of its rows at a time; its sums
// meet by lane exchanges and through LDS, so one launch does, without shares in memory.
constexpr int FEW = 4, FT = 512, FC = 16;

template <typename T, bool WIDE, int ROWS>
__global__ __launch_bounds__(FT) void k_linear_few(const T* __restrict__ x, const T* __restrict__ w, int rows, int K, int N,
                                                   Epilogue<T> e) {
  __shared__ float red[FT / 64][ROWS][FC];
  // neighbouring column blocks, which share lines of memory, on one XCD
  const int blocks = (N + FC - 1) / FC, xcd = blockIdx.x & 7;
  const int lo = (int)((int64_t)blocks * xcd >> 3), hi = (int)((int64_t)blocks * (xcd + 1) >> 3);
  const int block = lo + (int)(blockIdx.x >> 3);
  if (block >= hi) return;
  const int n0 = block * FC, c = (threadIdx.x & 1) * 8, n = n0 + c, kl = threadIdx.x >> 1;
  float acc[ROWS][8];
#pragma unroll
  for (int t = 0; t < ROWS; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[t][j] = 0.f;
  if (n < N)
#pragma unroll 8
    for (int k = kl; k < K; k += FT / 2) {
      float v[8];
      load8<T, WIDE>(w + (int64_t)k * N + n, N - n, v);
#pragma unroll
      for (int t = 0; t < ROWS; ++t) {
        const float xv = elem<T>::load(x + (int64_t)min(t, rows - 1) * K + k);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t][j] = fmaf(xv, v[j], acc[t][j]);
      }
    }
#pragma unroll
  for (int t = 0; t < ROWS; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int off = 2; off < 64; off <<= 1) acc[t][j] += __shfl_xor(acc[t][j], off, 64);
      if ((threadIdx.x & 63) < 2) red[threadIdx.x >> 6][t][c + j] = acc[t][j];
    }
  __syncthreads();
  const int t = threadIdx.x / FC, m = n0 + (int)threadIdx.x % FC;
  if (t < rows && t < ROWS && m < N) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < FT / 64; ++q) s += red[q][t][threadIdx.x % FC];
    e.store(t, m, N, s);
  }
}

template <typename T, bool WIDE>
void launch_few(const T* x, const T* w, int rows, int K, int N, const Epilogue<T>& e, hipStream_t st) {
  const dim3 grid((unsigned)(ceil_div(ceil_div(N, FC), 8) * 8));
#define CALL(R) MOE_LAUNCH("linear_fwd", (k_linear_few<T, WIDE, R>), grid, dim3(FT), 0, st, x, w, rows, K, N, e)
  if (rows == 1) CALL(1);
  else if (rows == 2) CALL(2);
  else CALL(4);
#undef CALL
}

// ---------------- dz and db ----------------
// dz = dy act'(z) and the workgroup's share of db.  WIDE: 32 lanes of 8 columns by 8 rows at a time;
// else a lane for each column, row by row.
constexpr int ZC = 256;   // columns of a workgroup
template <typename T, bool WIDE>
__global__ __launch_bounds__(256) void k_linear_dz(const T* __restrict__ dy, const T* __restrict__ z, int64_t rows,
                                                   int N, int act, int slab, T* __restrict__ dz,
                                                   float* __restrict__ part) {
  const int64_t t0 = (int64_t)blockIdx.x * slab, t1 = min(rows, t0 + slab);
  const int m = blockIdx.y * ZC + threadIdx.x;
  if constexpr (WIDE) {
    __shared__ float red[8][ZC];
    const int c = (threadIdx.x & 31) * 8, r = threadIdx.x >> 5, n = blockIdx.y * ZC + c;
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.f;
    if (n < N)
#pragma unroll 2
      for (int64_t t = t0 + r; t < t1; t += 8) {
        float d[8], v[8];
        load8<T, true>(dy + t * N + n, 8, d);
        if (dz) {
          load8<T, true>(z + t * N + n, 8, v);
          slope8(d, v, act);
          store8<T, true>(dz + t * N + n, 8, d);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += d[j];
      }
    if (!part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) red[r][c + j] = s[j];
    __syncthreads();
    if (m < N) {
      float a = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) a += red[q][threadIdx.x];
      part[(size_t)blockIdx.x * N + m] = a;
    }
  } else {
    if (m >= N) return;
    float s = 0.f;
    for (int64_t t = t0; t < t1; t += 8) {   // 8 rows in flight; past the end the last one, for nothing
      float d[8], v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t at = min(t + j, t1 - 1) * N + m;
        d[j] = elem<T>::load(dy + at);
        v[j] = dz ? elem<T>::load(z + at) : 0.f;
      }
      if (dz) slope8(d, v, act);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (t + j < t1) {
          if (dz) elem<T>::store(dz + (t + j) * N + m, d[j]);
          s += d[j];
        }
    }
    if (part) part[(size_t)blockIdx.x * N + m] = s;
  }
}

// db from its shares, added in a fixed order: 64 columns a workgroup, 16 slices of the shares
template <typename T>
__global__ __launch_bounds__(1024) void k_linear_db(const float* __restrict__ part, int W, int N, T* __restrict__ db) {
  __shared__ float red[16][64];
  const int c = threadIdx.x & 63, sl = threadIdx.x >> 6, n = blockIdx.x * 64 + c;
  float s = 0.f;
  if (n < N)
  #pragma unroll 8
    for (int w = sl; w < W; w += 16) s += part[(size_t)w * N + n];
  red[sl][c] = s;
  __syncthreads();
  if (sl == 0 && n < N) {
    for (int q = 1; q < 16; ++q) s += red[q][c];
    elem<T>::store(db + n, s);
  }
}

// rows of a share of db: about 1024 workgroups, of at least 16 rows
int dz_slab(const moe_linear_shape& s) {
  const int64_t blocks = ceil_div(s.N, ZC), want = ceil_div((int64_t)s.T * blocks, 1024);
  return (int)(ceil_div(want < 16 ? 16 : want > 65536 ? 65536 : want, 8) * 8);
}

inline bool at16(const void* p) { return ((uintptr_t)p & 15) == 0; }
// the tiles take bf16 rows of whole 16-byte chunks, the general kernel the rest
template <typename T>
bool tiled(const moe_linear_shape& s) { return sizeof(T) == 2 && s.K % 8 == 0 && s.N % 8 == 0; }

template <typename T>
hipError_t fwd(const moe_linear_shape& s, const T* x, const T* w, const T* b, const T* res, T* z, T* y, void* scratch,
               hipStream_t st) {
  float* const part = (float*)((char*)scratch + linear_layout(s).off_part);
  Epilogue<T> e{};
  e.out = y; e.z = z; e.bias = b; e.add = res; e.act = s.act;
  if (s.T <= FEW) {
    if (s.N % 8 == 0 && at16(w)) launch_few<T, true>(x, w, s.T, s.K, s.N, e, st);
    else launch_few<T, false>(x, w, s.T, s.K, s.N, e, st);
    return hipGetLastError();
  }
  if constexpr (sizeof(T) == 2)
    if (tiled<T>(s) && at16(x) && at16(w) && at16(b) && at16(res) && at16(z) && at16(y))
      return launch_linear_tiles("linear_fwd", x, s.K, true, w, s.N, false, s.T, s.N, s.K, {y, z, b, res, s.act}, part,
                                 st);
  return general<T>("linear_fwd", x, w, s.K, 1, s.N, 1, s.T, s.N, s.K, e, part, st);
}

template <typename T>
hipError_t bwd(const moe_linear_shape& s, const T* dy, const T* x, const T* w, const T* z, const T* dx_in, T* dx,
               T* dw, T* db, void* scratch, hipStream_t st) {
  const LinearLayout L = linear_layout(s);
  T* const dzbuf = s.act == MOE_ACT_NONE ? nullptr : (T*)scratch;
  float* const dbp = (float*)((char*)scratch + L.off_db);
  float* const part = (float*)((char*)scratch + L.off_part);
  const T* dz = dzbuf ? dzbuf : dy;
  const int slab = dz_slab(s), W = (int)ceil_div(s.T, slab);
  if ((dzbuf || db) && s.T > 0) {
    const dim3 grid((unsigned)W, (unsigned)ceil_div(s.N, ZC));
    if (s.N % 8 == 0 && at16(dy) && at16(z))
      MOE_LAUNCH("linear_dz", (k_linear_dz<T, true>), grid, dim3(256), 0, st, dy, z, (int64_t)s.T, s.N, s.act, slab,
                 dzbuf, db ? dbp : nullptr);
    else
      MOE_LAUNCH("linear_dz", (k_linear_dz<T, false>), grid, dim3(256), 0, st, dy, z, (int64_t)s.T, s.N, s.act, slab,
                 dzbuf, db ? dbp : nullptr);
  }
  if (db)
    MOE_LAUNCH("linear_db", k_linear_db<T>, dim3((unsigned)ceil_div(s.N, 64)), dim3(1024), 0, st, dbp, W, s.N, db);
  hipError_t err = hipGetLastError();
  if constexpr (sizeof(T) == 2)
    if (tiled<T>(s) && at16(dy) && at16(x) && at16(w) && at16(dx_in) && at16(dx) && at16(dw)) {
      if (err == hipSuccess && dx && s.T > 0)
        err = launch_linear_tiles("linear_dx", dz, s.N, true, w, s.N, true, s.T, s.K, s.N,
                                  {dx, nullptr, nullptr, dx_in, MOE_ACT_NONE}, part, st);
      if (err == hipSuccess)
        err = launch_linear_tiles("linear_dw", x, s.K, false, dz, s.N, false, s.K, s.N, s.T,
                                  {dw, nullptr, nullptr, nullptr, MOE_ACT_NONE}, part, st);
      return err;
    }
  if (err == hipSuccess && dx) {
    Epilogue<T> e{};
    e.out = dx; e.add = dx_in; e.act = MOE_ACT_NONE;
    err = general<T>("linear_dx", dz, w, s.N, 1, 1, s.N, s.T, s.K, s.N, e, part, st);
  }
  if (err == hipSuccess) {
    Epilogue<T> e{};
    e.out = dw; e.act = MOE_ACT_NONE;
    err = general<T>("linear_dw", x, dz, 1, s.K, s.N, 1, s.K, s.N, s.T, e, part, st);
  }
  return err;
}

}  // namespace

LinearLayout linear_layout(const moe_linear_shape& s) {
  const size_t es = s.dtype == MOE_BF16 ? 2 : 4;
  LinearLayout L{};
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  L.off_part = s.act == MOE_ACT_NONE ? 0 : up((size_t)s.T * s.N * es);
  size_t part = 0;   // of the largest of the three products, on the tiles or on the general kernel
  const bool tiles = s.dtype == MOE_BF16 && tiled<bf16_t>(s);
  const int64_t of[3][3] = {{s.T, s.N, s.K}, {s.T, s.K, s.N}, {s.K, s.N, s.T}};
  for (const auto& d : of) {
    const size_t a = tiles ? linear_part_bytes(d[0], d[1], d[2]) : 0, b = general_part_bytes(d[0], d[1], d[2]);
    part = a > part ? a : part;
    part = b > part ? b : part;
  }
  L.off_db = L.off_part + up(part);
  L.bytes = L.off_db + up((size_t)ceil_div(s.T, dz_slab(s)) * s.N * 4);
  return L;
}

hipError_t launch_linear_fwd(const moe_linear_shape& s, const void* x, const void* w, const void* b, const void* res,
                             void* z, void* y, void* scratch, hipStream_t st) {
  if (s.dtype == MOE_BF16)
    return fwd<bf16_t>(s, (const bf16_t*)x, (const bf16_t*)w, (const bf16_t*)b, (const bf16_t*)res, (bf16_t*)z,
                       (bf16_t*)y, scratch, st);
  return fwd<float>(s, (const float*)x, (const float*)w, (const float*)b, (const float*)res, (float*)z, (float*)y,
                    scratch, st);
}

hipError_t launch_linear_bwd(const moe_linear_shape& s, const void* dy, const void* x, const void* w, const void* z,
                             const void* dx_in, void* dx, void* dw, void* db, void* scratch, hipStream_t st) {
  if (s.dtype == MOE_BF16)
    return bwd<bf16_t>(s, (const bf16_t*)dy, (const bf16_t*)x, (const bf16_t*)w, (const bf16_t*)z,
                       (const bf16_t*)dx_in, (bf16_t*)dx, (bf16_t*)dw, (bf16_t*)db, scratch, st);
  return bwd<float>(s, (const float*)dy, (const float*)x, (const float*)w, (const float*)z, (const float*)dx_in,
                    (float*)dx, (float*)dw, (float*)db, scratch, st);
}

}  // namespace moe
