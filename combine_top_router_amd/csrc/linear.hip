// Matrix product with bias, activation and residual in its epilogue, and its backward.
//
//   z = x W + b,  y = act(z) + res
//   dz = dy act'(z),  dx = dx_in + dz W^T,  dW = x^T dz,  db = sum_t dz
// with x [T, K], W [K, N] as the layer's weights are stored, sums in fp32.  z is kept in the
// data's type for the backward; y is formed from the fp32 sum.
//
// Three ways to a product: up to four rows by k_linear_few, bf16 by matrix-core tiles
// (gemm_linear.hip), fp32 and what is left by k_linear_any.
#include <type_traits>

#include "linear.h"

namespace moe {

namespace {

// ---------------- relu's corner ----------------
// Where z is within its sum's rounding of 0, that rounding takes the side, and dz is off by all of dy: one
// in 10^7 elements of fp32's products, which in a matrix of 1003 x 333 leaves 2.7e-3 of a gradient's norm where
// all other roundings leave 3e-7.  So in fp32 (in bf16 it stays below the type's own steps) such a z is
// formed again in fp64 before it is kept; y, off by |z| at most, stays.  Which: a rounding is 2^-24 of a partial sum at
// most.  One over the first k of K is at most |x_1..k| |W_1..k|, and as the sum is near -b, at most
// |b| + |x_k+1..K| |W_k+1..K| too; the two products together are |x| |W| at most, so the smaller is
// (|x| |W| + |b|) / 2.  With K such roundings, taken as independent, 3 sqrt(K) of them are five standard deviations.
// The squares of both norms are added up beside the products.  Ordinary data have one such z in ten thousand
// or so; with all of it the forward of 1003 x 769 x 333 takes 18.8 us (16.5 without), of 8192 x 1024 x 2048 333 (312), of
// one row of 2048 x 768 4.6 (4.1).  Where sums cancel in bulk (rows far off 0, one-hot rows and pruned weights),
// whole blocks are formed again by the matrix cores in fp64 (8192 x 1024 x 2048 of nothing else: 1.4 ms).
struct Corner {
  const float* a;
  const float* b;
  const float* bias;   // or null
  float* z;
  int64_t am, ak, bk, bn, M, N, K;
};

// whether that z has to be formed again; b: its bias, norms: |x_t| |W_n| (3 2^-24 / 2 and 1 % for the norms'
// own rounding; where their squares leave fp32's range, above 10^19 or below 10^-20, the sum stays)
__device__ __forceinline__ bool corner_near(const Corner& c, float z, float b, float norms) {
  const float bound = 0x1.84p-24f * sqrtf((float)c.K + 64.f) * (norms + fabsf(b));
  return fabsf(z) < bound && bound < __builtin_inff();
}
// One element by a whole wave, U products of a lane under way; lane src has it
template <int U>
__device__ __forceinline__ void settle_one(const Corner& c, int m, int n, int src) {
  const float *const pa = c.a + m * c.am, *const pb = c.b + n * c.bn;
  const int lane = threadIdx.x & 63, K = (int)c.K;
  double s = 0.0;
  for (int k = lane; k - lane < K; k += 64 * U) {
    float u[U], v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {   // past the end the last again, for nothing
      const int at = min(k + 64 * j, K - 1);
      u[j] = pa[at * c.ak];
      v[j] = pb[at * c.bk];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) s = fma((double)(k + 64 * j < K ? u[j] : 0.f), (double)v[j], s);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
  if (lane == src) c.z[m * c.N + n] = (float)(c.bias ? s + (double)c.bias[n] : s);
}
// Each lane its own element, if it has one (any of the matrices' for the others)
__device__ __forceinline__ void settle_each(const Corner& c, bool near, int m, int n) {
  const float *pa = c.a + m * c.am, *pb = c.b + n * c.bn;
  double s = 0.0;
#pragma unroll 8
  for (int k = 0; k < (int)c.K; ++k, pa += c.ak, pb += c.bk) s = fma((double)*pa, (double)*pb, s);
  if (near) c.z[m * c.N + n] = (float)(c.bias ? s + (double)c.bias[n] : s);
}
// One element (m, n) a lane
__device__ __forceinline__ void settle_wave(const Corner& c, bool near, int m, int n) {
  uint64_t lanes = __ballot(near);
  if (__popcll(lanes) > 16) {
    settle_each(c, near, m, n);
    return;
  }
  for (; lanes != 0; lanes &= lanes - 1) {
    const int src = __builtin_ctzll(lanes);
    settle_one<16>(c, __shfl(m, src, 64), __shfl(n, src, 64), src);
  }
}
// All of a block of 32 x 32 from (m0, n0) on, in fp64 by the matrix cores
typedef double f64x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void settle_block(const Corner& c, int64_t m0, int64_t n0) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4, K = (int)c.K;
  const float *pa[2], *pb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {   // past the end the last row and column again, for nothing
    pa[i] = c.a + min(m0 + 16 * i + r, c.M - 1) * c.am;
    pb[i] = c.b + min(n0 + 16 * i + r, c.N - 1) * c.bn;
  }
  f64x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i / 2][i % 2] = f64x4{0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
  for (int k = q; k - q < K; k += 4) {
    const int at = min(k, K - 1);
    double u[2], v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float x = pa[i][at * c.ak], y = pb[i][at * c.bk];
      u[i] = k < K ? x : 0.f;
      v[i] = k < K ? y : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[i / 2][i % 2] = __builtin_amdgcn_mfma_f64_16x16x4f64(u[i / 2], v[i % 2], acc[i / 2][i % 2], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = n0 + 16 * (i % 2) + r;
    if (n >= c.N) continue;
    const double b = c.bias ? (double)c.bias[n] : 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + 16 * (i / 2) + 4 * j + q;
      if (m < c.M) c.z[m * c.N + n] = (float)(acc[i / 2][i % 2][j] + b);
    }
  }
}

// ---------------- any size, any alignment ----------------
// Tiles of 64 or 128 square, four waves, K steps of 32 staged through registers, 8 consecutive
// elements a thread, several steps' loads under way while one is multiplied, one barrier a step.
// With few tiles K is split, and the shares, fp32 [share, M, N], are added in order by a second launch with
// the epilogue.  In fp32 the matrix cores bound it (busy 77 % of the time: 8192 x 1024 x 2048 dx 290
// us, 118 TFLOP/s with tiles of 128, 98 with tiles of 64); for small products, the loads' latency.
constexpr int GSTEP = 32;

// rows of K in LDS, whole 16-byte pieces that 16 rows spread over all the banks
template <typename T> struct gstage;
template <> struct gstage<bf16_t> { static constexpr int LD = GSTEP + 8; };
template <> struct gstage<float> { static constexpr int LD = GSTEP + 4; };

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
  float* squares; // with shares and relu's corner: [share, M + N], the squares of A's rows and of B's columns
  Epilogue<T> e;
};
inline __device__ Corner corner_of(const GeneralArgs<float>& g) {
  return {g.a, g.b, g.e.bias, g.e.z, g.am, g.ak, g.bk, g.bn, g.M, g.N, g.K};
}

// One operand's part of a thread: H times 8 elements along the axis that is contiguous, 64 rows or
// columns apart
template <typename T, int H>
struct GeneralLd {
  const T* p;        // the step's first element (uniform)
  int64_t step;
  uint32_t off[H];   // the thread's places from there
  int row[H], k;     // the first in the tile: row of LDS, and in the step
  int some;          // of the 8 (uniform)
  bool km;           // K is contiguous
  __device__ __forceinline__ void setup(const T* m, int64_t xs, int64_t ks, int64_t x0, int64_t X, int64_t k0, int tid) {
    km = ks == 1;
    // K contiguous: 4 threads a row.  Else 4 threads of 8 columns by 16 of K in a wave, whose
    // writes into LDS then meet in no bank more than twice.
    const int x = km ? tid >> 2 : ((tid & 3) | (tid >> 6 & 1) << 2) * 8;
    k = km ? (tid & 3) * 8 : (tid >> 2 & 15) | (tid >> 7) << 4;
    p = m + x0 * xs + k0 * ks;
    step = GSTEP * ks;
    const int left = (int)min(X - x0, (int64_t)(64 * H));   // rows or columns there are
    some = km ? 8 : min(8, left);
    // past the end: the last row, or the last 8 columns, loaded again; what stays unwritten in LDS
    // goes into results that are discarded
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int y = min(x + 64 * h, km ? left - 1 : max(0, left - 8));
      row[h] = km ? x + 64 * h : y;
      off[h] = (uint32_t)y * (uint32_t)xs + (uint32_t)k * (uint32_t)ks;
    }
  }
  // The step with `left` of K to its end.  What lies past it is loaded from the last place there
  // is and made 0 by put: a selection here would wait for the loads.
  __device__ __forceinline__ void load(int left, T (&v)[H][8]) {
    const int past = max(0, k - (left - 1));
    if (left >= GSTEP && some == 8) {
#pragma unroll
      for (int h = 0; h < H; ++h) load8(p + off[h], v[h]);
    } else if (!km && some == 8) {
#pragma unroll
      for (int h = 0; h < H; ++h) load8(p + (off[h] - (uint32_t)past * (uint32_t)(step / GSTEP)), v[h]);
    } else {
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[h][j] = p[km ? off[h] - (uint32_t)k + (uint32_t)min(k + j, left - 1)
                         : off[h] - (uint32_t)past * (uint32_t)(step / GSTEP) + (uint32_t)min(j, some - 1)];
    }
    p += step;
  }
  __device__ __forceinline__ void put(T (*s)[gstage<T>::LD], int left, T (&v)[H][8]) const {
    if (left < GSTEP)
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[h][j] = (km ? k + j : k) < left ? v[h][j] : (T)0;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (km) {
        __builtin_memcpy(__builtin_assume_aligned(&s[row[h]][k], 16), v[h], sizeof(v[h]));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[row[h] + j][k] = v[h][j];
      }
    }
  }
};

// H: tiles of 64 H, waves of 32 H; DEPTH steps' loads are under way (four where the registers of four
// workgroups on a CU hold them: in fp32 three workgroups with four steps were no faster); CORNER: relu's
template <typename T, int H, bool CORNER = false>
__global__ __launch_bounds__(256, H == 2 ? 2 : 4) void k_linear_any(GeneralArgs<T> g) {
  constexpr int LD = gstage<T>::LD, TILE = 64 * H, DEPTH = H == 1 && sizeof(T) == 2 ? 4 : 2;
  __shared__ __attribute__((aligned(16))) T as[2][TILE][LD];   // [m][k]
  __shared__ __attribute__((aligned(16))) T bs[2][TILE][LD];   // [n][k]
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t m0 = (int64_t)blockIdx.x * TILE, n0 = (int64_t)blockIdx.y * TILE, k0 = blockIdx.z * g.ks;
  const int64_t k1 = min(g.K, k0 + g.ks);
  const int wm = (wv & 1) * 32 * H, wn = (wv >> 1) * 32 * H;
  GeneralLd<T, H> la, lb;
  la.setup(g.a, g.am, g.ak, m0, g.M, k0, tid);
  lb.setup(g.b, g.bn, g.bk, n0, g.N, k0, tid);
  f32x16 acc[H][H];
#pragma unroll
  for (int i = 0; i < H * H; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[i / H][i % H][j] = 0.f;
  T ra[DEPTH][H][8], rb[DEPTH][H][8];
  float qa = 0.f, qb = 0.f;   // CORNER: squares of a part of a row of each stage
  const int len = (int)(k1 - k0);
#pragma unroll
  for (int c = 0; c < DEPTH; ++c)
    if (c * GSTEP < len) {
      la.load(len - c * GSTEP, ra[c]);
      lb.load(len - c * GSTEP, rb[c]);
    }
  for (int k2 = 0; k2 < len; k2 += DEPTH * GSTEP)
#pragma unroll
    for (int c = 0; c < DEPTH; ++c) {
      const int k = k2 + c * GSTEP;
      if (k >= len) break;
      la.put(as[c & 1], len - k, ra[c]);
      lb.put(bs[c & 1], len - k, rb[c]);
      __syncthreads();   // the other stage's readers are past it: they have met this barrier since
      if (k + DEPTH * GSTEP < len) {
        la.load(len - k - DEPTH * GSTEP, ra[c]);
        lb.load(len - k - DEPTH * GSTEP, rb[c]);
      }
      const T* const pa = &as[c & 1][wm + (lane & 31)][0];
      const T* const pb = &bs[c & 1][wn + (lane & 31)][0];
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int kk = 0; kk < GSTEP; kk += 16) {
          bf16x8 va[H], vb[H];
#pragma unroll
          for (int h = 0; h < H; ++h) {
            va[h] = *reinterpret_cast<const bf16x8*>(pa + 32 * h * LD + kk + (lane >> 5) * 8);
            vb[h] = *reinterpret_cast<const bf16x8*>(pb + 32 * h * LD + kk + (lane >> 5) * 8);
          }
#pragma unroll
          for (int i = 0; i < H * H; ++i)
            acc[i / H][i % H] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va[i / H], vb[i % H], acc[i / H][i % H], 0, 0, 0);
        }
      } else {
        // the instruction sums k of its lower and of its upper lanes: here k and k + 4
#pragma unroll
        for (int kk = 0; kk < GSTEP; kk += 8) {
          f32x4 va[H], vb[H];
#pragma unroll
          for (int h = 0; h < H; ++h) {
            va[h] = *reinterpret_cast<const f32x4*>(pa + 32 * h * LD + kk + (lane >> 5) * 4);
            vb[h] = *reinterpret_cast<const f32x4*>(pb + 32 * h * LD + kk + (lane >> 5) * 4);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < H * H; ++i)
              acc[i / H][i % H] =
                  __builtin_amdgcn_mfma_f32_32x32x2f32(va[i / H][j], vb[i % H][j], acc[i / H][i % H], 0, 0, 0);
        }
      }
      if constexpr (CORNER) {
#pragma unroll
        for (int j = 0; j < 8 * H; j += 4) {
          const f32x4 u = *reinterpret_cast<const f32x4*>(&as[c & 1][tid % TILE][tid / TILE * 8 * H + j]);
          const f32x4 v = *reinterpret_cast<const f32x4*>(&bs[c & 1][tid % TILE][tid / TILE * 8 * H + j]);
          qa += fmaf(u[0], u[0], u[1] * u[1]) + fmaf(u[2], u[2], u[3] * u[3]);
          qb += fmaf(v[0], v[0], v[1] * v[1]) + fmaf(v[2], v[2], v[3] * v[3]);
        }
      }
    }
#pragma unroll
  for (int i = 0; i < H * H; ++i) {
    const int64_t n = n0 + wn + 32 * (i % H) + (lane & 31);
    if (n >= g.N) continue;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t m = m0 + wm + 32 * (i / H) + 8 * (j >> 2) + 4 * (lane >> 5) + (j & 3);
      if (m >= g.M) continue;
      const float v = acc[i / H][i % H][j];
      if (g.part) g.part[(blockIdx.z * g.M + m) * g.N + n] = v;
      else g.e.store(m, n, g.N, v);
    }
  }
  if constexpr (CORNER) {
    __shared__ float an[256], bn[256];
    an[tid] = qa;
    bn[tid] = qb;
    __syncthreads();
    if (tid < TILE) {
#pragma unroll
      for (int p = 1; p < 4 / H; ++p) {
        qa += an[tid + p * TILE];
        qb += bn[tid + p * TILE];
      }
      an[tid] = sqrtf(qa);
      bn[tid] = sqrtf(qb);
    }
    if (g.part) {   // rows by the first workgroup along N, columns by the first along M
      float* const to = g.squares + blockIdx.z * (g.M + g.N);
      if (tid < TILE && blockIdx.y == 0 && m0 + tid < g.M) to[m0 + tid] = qa;
      if (tid < TILE && blockIdx.x == 0 && n0 + tid < g.N) to[g.M + n0 + tid] = qb;
      return;
    }
    __syncthreads();
    const Corner c = corner_of(g);
    uint32_t near[H * H] = {};   // a bit for each of the lane's elements of a block of 32 x 32
#pragma unroll
    for (int i = 0; i < H * H; ++i) {
      const int nl = wn + 32 * (i % H) + (lane & 31);
      if (n0 + nl >= g.N) continue;
      const float b = c.bias ? c.bias[n0 + nl] : 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int ml = wm + 32 * (i / H) + 8 * (j >> 2) + 4 * (lane >> 5) + (j & 3);
        if (m0 + ml < g.M && corner_near(c, acc[i / H][i % H][j] + b, b, an[ml] * bn[nl])) near[i] |= 1u << j;
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // what is formed again is written over
#pragma unroll 1
    for (int i = 0; i < H * H; ++i) {
      uint32_t bits = near[0];
#pragma unroll
      for (int h = 1; h < H * H; ++h) bits = i == h ? near[h] : bits;
      uint64_t lanes = __ballot(bits != 0);
      if (lanes == 0) continue;
      const int64_t mb = m0 + wm + 32 * (i / H), nb = n0 + wn + 32 * (i % H);
      int count = __popc(bits);
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) count += __shfl_xor(count, off, 64);
      if (count > 12) {   // (a block takes about as long as 12 elements)
        settle_block(c, mb, nb);
        continue;
      }
      for (; lanes != 0; lanes &= lanes - 1) {
        const int src = __builtin_ctzll(lanes);
#pragma unroll 1
        for (uint32_t left = __shfl(bits, src, 64); left != 0; left &= left - 1) {
          const int j = __builtin_ctz(left);
          settle_one<4>(c, (int)mb + 8 * (j >> 2) + 4 * (src >> 5) + (j & 3), (int)nb + (src & 31), src);
        }
      }
    }
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

// The same with relu's corner; eight shares' numbers are loaded before they are added, in the same order
__global__ __launch_bounds__(256) void k_linear_corner_join(GeneralArgs<float> g, int splits) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, size = g.M * g.N;
  const bool in = i < size;
  const int64_t at = in ? i : size - 1;   // every lane stays
  const int m = (int)(at / g.N), n = (int)(at - m * g.N);
  const float *p = g.part + at, *pa = g.squares + m, *pb = g.squares + g.M + n;
  float s = 0.f, qa = 0.f, qb = 0.f;
  for (int sp = 0; sp < splits; sp += 8) {
    float u[8], a[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t k = min(sp + j, splits - 1);
      u[j] = p[k * size];
      a[j] = pa[k * (g.M + g.N)];
      b[j] = pb[k * (g.M + g.N)];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (sp + j < splits) {
        s += u[j];
        qa += a[j];
        qb += b[j];
      }
  }
  if (in) g.e.store(m, n, g.N, s);
  const Corner c = corner_of(g);
  const float b = c.bias ? c.bias[n] : 0.f, z = s + b;
  settle_wave(c, in && corner_near(c, z, b, sqrtf(qa) * sqrtf(qb)), m, n);
}

constexpr PlanCost kAny16[2] = {{128, 128, 2, 1.1, 0.6, 6.0, 5.0, 6.0}, {64, 64, 4, 0.8, 0.26, 3.0, 5.0, 6.0}};
constexpr PlanCost kAny32[2] = {{128, 128, 2, 2.8, 2.4, 7.0, 5.0, 6.0}, {64, 64, 4, 1.1, 0.66, 3.0, 5.0, 6.0}};
template <typename T>
Plan general_plan(int64_t M, int64_t N, int64_t K) {
  return plan_product(sizeof(T) == 2 ? kAny16 : kAny32, 2, GSTEP, gemm_cus(), M, N, K);
}
template <typename T>
size_t general_part_bytes(int64_t M, int64_t N, int64_t K, bool corner) {
  const int s = general_plan<T>(M, N, K).splits;
  return s == 1 ? 0 : (size_t)s * (M * N + (corner ? M + N : 0)) * 4;
}
// whether relu's slope is decided beside the product
template <typename T>
bool has_corner(const Epilogue<T>& e) { return sizeof(T) == 4 && e.act == MOE_ACT_RELU && e.z; }

template <typename T>
hipError_t general(const char* name, const T* a, const T* b, int64_t am, int64_t ak, int64_t bk, int64_t bn, int64_t M,
                   int64_t N, int64_t K, const Epilogue<T>& e, float* part, hipStream_t st) {
  if (M == 0 || N == 0) return hipSuccess;
  const Plan p = general_plan<T>(M, N, K);
  const GeneralArgs<T> g{a, b, am, ak, bk, bn, M, N, K, p.ks, p.splits > 1 ? part : nullptr, part + p.splits * M * N, e};
  const int tile = p.shape == 0 ? 128 : 64;
  const dim3 grid((unsigned)ceil_div(M, tile), (unsigned)ceil_div(N, tile), (unsigned)p.splits);
  const dim3 join((unsigned)ceil_div(M * N, 256));
  if constexpr (sizeof(T) == 4)
    if (has_corner(e)) {
      if (tile == 128) MOE_LAUNCH(name, (k_linear_any<T, 2, true>), grid, dim3(256), 0, st, g);
      else MOE_LAUNCH(name, (k_linear_any<T, 1, true>), grid, dim3(256), 0, st, g);
      if (p.splits > 1) MOE_LAUNCH("linear_join", k_linear_corner_join, join, dim3(256), 0, st, g, p.splits);
      return hipGetLastError();
    }
  if (tile == 128) MOE_LAUNCH(name, (k_linear_any<T, 2>), grid, dim3(256), 0, st, g);
  else MOE_LAUNCH(name, (k_linear_any<T, 1>), grid, dim3(256), 0, st, g);
  if (p.splits > 1)
    MOE_LAUNCH("linear_join", k_linear_any_join<T>, join, dim3(256), 0, st, g, p.splits);
  return hipGetLastError();
}

// ---------------- few rows ----------------
// Up to FEW rows (the tokens of a decode step) of 8 columns or more: W is read once, and that is what counts.  A
// workgroup takes 16 columns, two lanes of 8, and all of K, 256 of its rows at a time; its sums
// meet by lane exchanges and through LDS, so one launch does, without shares in memory.  What bounds
// it is latency: with all 16 rows of a lane requested before the first product 1 x 4096 x 1536 (12.6
// MB) takes 4.9 us, one after another 7.0; 4 x 4096 x 4096 (33.6 MB) 10.1 and 25.5.
constexpr int FEW = 4, FT = 512, FC = 16;

// U: rows of W under way; CORNER: relu's
template <typename T, int ROWS, bool CORNER = false, int U = (sizeof(T) == 2 ? 8 : 4) * (ROWS == 1 ? 2 : 1)>
__global__ __launch_bounds__(FT) void k_linear_few(const T* __restrict__ x, const T* __restrict__ w, int rows, int K, int N,
                                                   Epilogue<T> e) {
  constexpr int SUMS = ROWS + CORNER;   // the last: the squares of W's columns
  __shared__ float red[FT / 64][SUMS][FC], xred[FT / 64][ROWS];
  // neighbouring column blocks, which share lines of memory, on one XCD
  const int blocks = (N + FC - 1) / FC, xcd = blockIdx.x & 7;
  const int lo = (int)((int64_t)blocks * xcd >> 3), hi = (int)((int64_t)blocks * (xcd + 1) >> 3);
  const int block = lo + (int)(blockIdx.x >> 3);
  if (block >= hi) return;
  const int n0 = block * FC, n = n0 + (threadIdx.x & 1) * 8, kl = threadIdx.x >> 1;
  const int at = min(n, N - 8);   // the last columns: the last 8 there are, of which it keeps its own
  float acc[SUMS][8], xq[ROWS];   // xq: the squares of x's rows
#pragma unroll
  for (int t = 0; t < SUMS; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[t][j] = 0.f;
#pragma unroll
  for (int t = 0; t < ROWS; ++t) xq[t] = 0.f;
  const int64_t step = (int64_t)(FT / 2) * N;
  const T* wp = w + (int64_t)kl * N + at;
  // U rows of W: all loads before the first product; TAIL: past the end the first one again, for nothing
  auto rows_of_w = [&](auto tail, int k) {
    constexpr bool TAIL = decltype(tail)::value;
    raw8<T> v[U];
    T xv[U][ROWS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = !TAIL || k + u * (FT / 2) < K;
      v[u].load(in ? wp + u * step : wp);
      const T* const xp = x + (in ? k + u * (FT / 2) : k);
#pragma unroll
      for (int t = 0; t < ROWS; ++t) xv[u][t] = xp[(int64_t)min(t, rows - 1) * K];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8];
      v[u].get(f);
      const bool in = !TAIL || k + u * (FT / 2) < K;
#pragma unroll
      for (int t = 0; t < ROWS; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float s = fmaf(elem<T>::load(&xv[u][t]), f[j], acc[t][j]);
          acc[t][j] = in ? s : acc[t][j];
        }
      if constexpr (CORNER)
        if (in) {
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[ROWS][j] = fmaf(f[j], f[j], acc[ROWS][j]);
#pragma unroll
          for (int t = 0; t < ROWS; ++t) xq[t] = fmaf(xv[u][t], xv[u][t], xq[t]);
        }
    }
    wp += U * step;
  };
  int k = kl;
  for (; k + (U - 1) * (FT / 2) < K; k += U * (FT / 2)) rows_of_w(std::false_type{}, k);
  if (k < K) rows_of_w(std::true_type{}, k);
  // over the 32 lanes of a column block: half of the 8 values goes to the other lane of a pair,
  // then half of the 4 left, then of the 2
  const int lane = threadIdx.x & 63;
  const bool b1 = lane & 2, b2 = lane & 4, b3 = lane & 8;
  const int col = (b1 ? 4 : 0) + (b2 ? 2 : 0) + (b3 ? 1 : 0);
#pragma unroll
  for (int t = 0; t < SUMS; ++t) {
    float h[4], q[2], s;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = (b1 ? acc[t][4 + j] : acc[t][j]) + __shfl_xor(b1 ? acc[t][j] : acc[t][4 + j], 2, 64);
#pragma unroll
    for (int j = 0; j < 2; ++j) q[j] = (b2 ? h[2 + j] : h[j]) + __shfl_xor(b2 ? h[j] : h[2 + j], 4, 64);
    s = (b3 ? q[1] : q[0]) + __shfl_xor(b3 ? q[0] : q[1], 8, 64);
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if (lane < 16 && at + col >= n) red[threadIdx.x >> 6][t][at + col - n0] = s;
  }
  if constexpr (CORNER) {
#pragma unroll
    for (int t = 0; t < ROWS; ++t) {
#pragma unroll
      for (int off = 2; off < 64; off <<= 1) xq[t] += __shfl_xor(xq[t], off, 64);   // a pair of lanes has the same of x
      if (lane == 0) xred[threadIdx.x >> 6][t] = xq[t];
    }
  }
  __syncthreads();
  const int t = threadIdx.x / FC, m = n0 + (int)threadIdx.x % FC;
  const bool in = t < rows && t < ROWS && m < N;
  float s = 0.f;
  if (in) {
#pragma unroll
    for (int q = 0; q < FT / 64; ++q) s += red[q][t][threadIdx.x % FC];
    e.store(t, m, N, s);
  }
  if constexpr (CORNER)
    if (threadIdx.x < 64) {   // rows and columns of a block: one wave
      static_assert(FEW * FC <= 64, "one wave");
      float qa = 0.f, qb = 0.f;
#pragma unroll
      for (int q = 0; q < FT / 64; ++q) {
        qa += xred[q][min(t, ROWS - 1)];
        qb += red[q][ROWS][threadIdx.x % FC];
      }
      const Corner c{x, w, e.bias, e.z, K, 1, N, 1, rows, N, K};
      const float b = in && e.bias ? e.bias[m] : 0.f, z = s + b;
      settle_wave(c, in && corner_near(c, z, b, sqrtf(qa) * sqrtf(qb)), min(t, rows - 1), min(m, N - 1));
    }
}

template <typename T>
void launch_few(const T* x, const T* w, int rows, int K, int N, const Epilogue<T>& e, hipStream_t st) {
  const dim3 grid((unsigned)(ceil_div(ceil_div(N, FC), 8) * 8));
#define CALL(...) MOE_LAUNCH("linear_fwd", (k_linear_few<T, __VA_ARGS__>), grid, dim3(FT), 0, st, x, w, rows, K, N, e)
  if constexpr (sizeof(T) == 4)
    if (has_corner(e)) {
      if (rows == 1) CALL(1, true);
      else if (rows == 2) CALL(2, true);
      else CALL(4, true);
      return;
    }
  if (rows == 1) CALL(1);
  else if (rows == 2) CALL(2);
  else CALL(4);
#undef CALL
}

// ---------------- rows laid out for the tiles ----------------
// Two bf16 matrices copied with rows of whole 16-byte chunks, zeros behind: a row takes 2^sh
// lanes, a chunk each.  (8192 x 1001 and 1001 x 2049 in 9 us.)
struct Pad {
  const bf16_t* from;
  bf16_t* to;
  int64_t rows, wgs;
  int cols, sh;
};
__global__ __launch_bounds__(256) void k_linear_pad(Pad p0, Pad p1) {
  const bool second = blockIdx.x >= p0.wgs;
  const Pad p = second ? p1 : p0;
  const int64_t row = ((int64_t)blockIdx.x - (second ? p0.wgs : 0)) * (256 >> p.sh) + (threadIdx.x >> p.sh);
  if (row >= p.rows) return;
  const int chunks = (p.cols + 7) / 8;
  const bf16_t* const from = p.from + row * p.cols;
  i32x4* const to = reinterpret_cast<i32x4*>(p.to) + row * chunks;
  for (int c = threadIdx.x & ((1 << p.sh) - 1); c < chunks; c += 1 << p.sh) {
    i32x4 u;
    if (8 * c + 8 <= p.cols) {
      u = *reinterpret_cast<const i32x4_a2*>(from + 8 * c);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = 8 * c + 2 * j;
        u[j] = (int)((uint32_t)(n < p.cols ? from[n] : 0) | (uint32_t)(n + 1 < p.cols ? from[n + 1] : 0) << 16);
      }
    }
    to[c] = u;
  }
}

Pad pad_of(const bf16_t* from, bf16_t* to, int64_t rows, int cols) {
  int sh = 2;
  while (sh < 6 && (8 << sh) < cols) ++sh;
  return {from, to, rows, ceil_div(rows, 256 >> sh), cols, sh};
}

// ---------------- dz and db ----------------
// dz = dy act'(z) and the workgroup's share of db: 32 lanes of 8 columns by 8 rows at a time.  dz
// (or null) has rows of ldz, zeros past N; z may be null: no activation, dz a copy.  Bound by memory:
// 16384 x 4096 bf16 (403 MB) 84 us, 4.8 TB/s.
constexpr int ZC = 256;   // columns of a workgroup
template <typename T>
__global__ __launch_bounds__(256) void k_linear_dz(const T* __restrict__ dy, const T* __restrict__ z, int64_t rows,
                                                   int N, int act, int slab, T* __restrict__ dz, int ldz,
                                                   float* __restrict__ part) {
  __shared__ float red[8][ZC];
  const int64_t t0 = (int64_t)blockIdx.x * slab, t1 = min(rows, t0 + slab);
  const int c = (threadIdx.x & 31) * 8, r = threadIdx.x >> 5, n = blockIdx.y * ZC + c;
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = 0.f;
  if (n + 8 <= N) {
#pragma unroll 2
    for (int64_t t = t0 + r; t < t1; t += 8) {
      float d[8], v[8];
      load8(dy + t * N + n, d);
      if (dz) {
        if (z) {
          load8(z + t * N + n, v);
          slope8(d, v, act);
        }
        store8(dz + t * ldz + n, d);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += d[j];
    }
  } else if (n < N) {
    for (int64_t t = t0 + r; t < t1; t += 8) {
      float d[8], v[8];
      load_some(dy + t * N + n, N - n, d);
      if (dz) {
        if (z) {
          load_some(z + t * N + n, N - n, v);
          slope8(d, v, act);
        }
        store_some(dz + t * ldz + n, ldz - n, d);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += d[j];
    }
  }
  if (!part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) red[r][c + j] = s[j];
  __syncthreads();
  const int m = blockIdx.y * ZC + threadIdx.x;
  if (m < N) {
    float a = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) a += red[q][threadIdx.x];
    part[(size_t)blockIdx.x * N + m] = a;
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
// T K N from which odd widths are worth their copies: forward and backward of 300 x 777 x 1555 (3.6e8)
// take 43 us on the tiles and 52 on the general kernel, of 60 x 1001 x 2049 (1.2e8) 41 and 34
constexpr double kPadFrom = 2e8;
// the tiles take bf16 rows of whole 16-byte chunks, the general kernel the rest
template <typename T>
bool tiled(const moe_linear_shape& s) { return sizeof(T) == 2 && s.K % 8 == 0 && s.N % 8 == 0; }
// or, where that is worth the copies, the tiles after x and W were laid out anew
bool padded(const moe_linear_shape& s) {
  return s.dtype == MOE_BF16 && s.T > FEW && (s.K % 8 != 0 || s.N % 8 != 0) && (double)s.T * s.K * s.N >= kPadFrom;
}
inline int up8(int n) { return (n + 7) / 8 * 8; }

struct LinearLayout {
  // scratch: dz, x and W laid out anew, the shares of db, those of a product split along its sum
  size_t off_x, off_w, off_db, off_part;
};
// (the shares come last: their room takes the plans of all three products, which a call need not know.)  The
// forward's own has no dz and no db, and so lies within the backward's.
LinearLayout linear_layout(const moe_linear_shape& s, bool forward) {
  const size_t es = s.dtype == MOE_BF16 ? 2 : 4;
  LinearLayout L{};
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const bool pad = padded(s);
  L.off_x = forward || (s.act == MOE_ACT_NONE && !(pad && s.N % 8 != 0)) ? 0 : up((size_t)s.T * (pad ? up8(s.N) : s.N) * es);
  L.off_w = L.off_x + (pad && s.K % 8 != 0 ? up((size_t)s.T * up8(s.K) * es) : 0);
  L.off_db = L.off_w + (pad && s.N % 8 != 0 ? up((size_t)s.K * up8(s.N) * es) : 0);
  L.off_part = L.off_db + (forward ? 0 : up((size_t)ceil_div(s.T, dz_slab(s)) * s.N * 4));
  return L;
}

// the operands as the tiles take them; false: one is out of place
bool pad_operands(const moe_linear_shape& s, const LinearLayout& L, void* scratch, const bf16_t*& x, const bf16_t*& w,
                  hipStream_t st) {
  const bool px = s.K % 8 != 0, pw = s.N % 8 != 0;
  if ((!px && !at16(x)) || (!pw && !at16(w))) return false;
  Pad p[2];
  int n = 0;
  if (px) p[n++] = pad_of(x, (bf16_t*)((char*)scratch + L.off_x), s.T, s.K);
  if (pw) p[n++] = pad_of(w, (bf16_t*)((char*)scratch + L.off_w), s.K, s.N);
  if (n == 1) p[1] = Pad{};
  MOE_LAUNCH("linear_pad", k_linear_pad, dim3((unsigned)(p[0].wgs + p[1].wgs)), dim3(256), 0, st, p[0], p[1]);
  if (px) x = (const bf16_t*)((char*)scratch + L.off_x);
  if (pw) w = (const bf16_t*)((char*)scratch + L.off_w);
  return true;
}

template <typename T>
hipError_t fwd(const moe_linear_shape& s, const T* x, const T* w, const T* b, const T* res, T* z, T* y, void* scratch,
               hipStream_t st) {
  Epilogue<T> e{};
  e.out = y; e.z = z; e.bias = b; e.add = res; e.act = s.act;
  if (s.T <= FEW && s.N >= 8) {
    launch_few<T>(x, w, s.T, s.K, s.N, e, st);
    return hipGetLastError();
  }
  const LinearLayout L = linear_layout(s, true);
  float* const part = (float*)((char*)scratch + L.off_part);
  if constexpr (sizeof(T) == 2) {
    const bool wide = s.N % 8 == 0 && at16(b) && at16(res) && at16(z) && at16(y);
    if ((tiled<T>(s) && wide && at16(x) && at16(w)) || (padded(s) && pad_operands(s, L, scratch, x, w, st)))
      return launch_linear_tiles("linear_fwd", x, up8(s.K), true, w, up8(s.N), false, s.T, s.N, s.K,
                                 {y, z, b, res, s.act, wide}, part, st);
  }
  return general<T>("linear_fwd", x, w, s.K, 1, s.N, 1, s.T, s.N, s.K, e, part, st);
}

template <typename T>
hipError_t bwd(const moe_linear_shape& s, const T* dy, const T* x, const T* w, const T* z, const T* dx_in, T* dx,
               T* dw, T* db, void* scratch, hipStream_t st) {
  const LinearLayout L = linear_layout(s, false);
  bool tiles = tiled<T>(s) && at16(dy) && at16(x) && at16(w) && at16(dx_in) && at16(dx) && at16(dw);
  if constexpr (sizeof(T) == 2)
    if (padded(s) && (s.N % 8 != 0 || at16(dy))) tiles = pad_operands(s, L, scratch, x, w, st);
  const bool pad_dz = tiles && s.N % 8 != 0;
  const int ldz = pad_dz ? up8(s.N) : s.N;
  T* const dzbuf = s.act == MOE_ACT_NONE && !pad_dz ? nullptr : (T*)scratch;
  float* const dbp = (float*)((char*)scratch + L.off_db);
  float* const part = (float*)((char*)scratch + L.off_part);
  const T* dz = dzbuf ? dzbuf : dy;
  const int slab = dz_slab(s), W = (int)ceil_div(s.T, slab);
  if ((dzbuf || db) && s.T > 0) {
    const dim3 grid((unsigned)W, (unsigned)ceil_div(s.N, ZC));
    MOE_LAUNCH("linear_dz", k_linear_dz<T>, grid, dim3(256), 0, st, dy, z, (int64_t)s.T, s.N, s.act, slab, dzbuf, ldz,
               db ? dbp : nullptr);
  }
  if (db)
    MOE_LAUNCH("linear_db", k_linear_db<T>, dim3((unsigned)ceil_div(s.N, 64)), dim3(1024), 0, st, dbp, W, s.N, db);
  hipError_t err = hipGetLastError();
  if constexpr (sizeof(T) == 2)
    if (tiles) {
      const int ldx = up8(s.K), ldw = up8(s.N);
      if (err == hipSuccess && dx && s.T > 0)
        err = launch_linear_tiles("linear_dx", dz, ldw, true, w, ldw, true, s.T, s.K, s.N,
                                  {dx, nullptr, nullptr, dx_in, MOE_ACT_NONE, s.K % 8 == 0 && at16(dx) && at16(dx_in)}, part,
                                  st);
      if (err == hipSuccess)
        err = launch_linear_tiles("linear_dw", x, ldx, false, dz, ldw, false, s.K, s.N, s.T,
                                  {dw, nullptr, nullptr, nullptr, MOE_ACT_NONE, s.N % 8 == 0 && at16(dw)}, part, st);
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

size_t linear_scratch_bytes(const moe_linear_shape& s, bool forward) {
  if (forward && s.T <= FEW && s.N >= 8) return 0;
  size_t part = 0;   // of the largest of the products, on the tiles or on the general kernel
  const bool tiles = padded(s) || (s.dtype == MOE_BF16 && tiled<bf16_t>(s));
  const int64_t of[3][3] = {{s.T, s.N, s.K}, {s.T, s.K, s.N}, {s.K, s.N, s.T}};
  for (const auto& d : of) {
    if (forward && d != of[0]) break;
    const size_t a = tiles ? linear_part_bytes(d[0], d[1], d[2]) : 0;
    const size_t b = s.dtype == MOE_BF16 ? general_part_bytes<bf16_t>(d[0], d[1], d[2], false)
                                         : general_part_bytes<float>(d[0], d[1], d[2], s.act == MOE_ACT_RELU);
    part = a > part ? a : part;
    part = b > part ? b : part;
  }
  return linear_layout(s, forward).off_part + part;
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
