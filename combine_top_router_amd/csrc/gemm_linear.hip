// The matrix product with an epilogue on matrix-core tiles: bf16, rows of whole 16-byte chunks.
//
// Workgroups of four waves, several to a CU, so that one's barriers, first loads and epilogue hide
// behind the others' products (for the largest products eight waves alone).  K steps of 64 move
// global -> LDS by the direct loads into two stages, one barrier a step.  The operands keep their own
// layouts (an axis of K is read in 16-byte pieces, one of M or N by the transposing LDS reads), so
// nothing is transposed in memory.  Chunks past the end of K come from a zeroed area.  A product
// with few tiles is split along K: the shares of a tile, in the accumulators' own order, are added
// by a second launch in a fixed order, with the epilogue.
//
// The loads (127 to 170 us of 16384 x 1536 x 4096's 210) and the products (140 to 165) each come near
// the whole time: what is left is their overlap.  4096^3 takes 113 us, 1.22 PFLOP/s (a library's
// product of 8192^3: 1.27); 16384 x 1536 x 4096 forward 208 us with y alone, 264 with bias, silu,
// residual and z (the epilogue's 400 MB, unhidden with one workgroup on a CU), dx 211, dw
// about 230 with the sum of its shares.
#define MOE_GEMM_FW 256
#include "gemm_engine.h"
#include "linear.h"

namespace moe {

namespace {

__device__ __attribute__((aligned(16))) const uint32_t g_zero16[4] = {0, 0, 0, 0};

// A tile shape: TM x TN outputs, waves of 32 MI x 32 NI, K steps of BK in two stages, OCC
// workgroups on a CU
template <int TM_, int TN_, int MI_, int NI_, int OCC_>
struct Shape {
  static constexpr int TM = TM_, TN = TN_, MI = MI_, NI = NI_, OCC = OCC_;
  static constexpr int WMS = TM / (32 * MI), WNS = TN / (32 * NI);   // waves along M and N
  static constexpr int TW = WMS * WNS, THR = 64 * TW;
  static constexpr int A = TM * BK, STAGE = (TM + TN) * BK;
  static constexpr int LA = TM * BK * 2 / 1024 / TW, LB = TN * BK * 2 / 1024 / TW;   // loads of a wave a stage
  static constexpr int NB = NI;   // 32-column blocks of an epilogue band
  static constexpr int BAND = 32 * 32 * NB;
  static_assert(LA >= 1 && LB >= 1 && LA * TW * 512 == A, "whole loads");
  static_assert(OCC * 2 * STAGE * 2 <= 160 * 1024 && OCC * TW <= 16, "LDS");
  static_assert(TW * BAND <= STAGE, "the epilogue's bands fit in a stage");
};

// (K-major tiles as in gemm_engine.h.)  MN-major [BK][W]: the four k-rows that a transposing read
// takes lie 64 bytes apart in the 256 of the banks.
template <int W>
__device__ __forceinline__ int mn_chunk(int r, int c) {
  return W >= 128 ? c ^ ((r & 3) << 2) : c ^ ((r & 2) << 1);
}
template <int W>
__device__ __forceinline__ void mn_slot(int s, int& r, int& c) {
  r = s / (W / 8);
  c = mn_chunk<W>(r, s % (W / 8));
}
// (see frag_mnmaj)
template <int W>
__device__ __forceinline__ bf16x8 mn_frag(const bf16_t* s, int base, int kk, int lane) {
  const int g = lane >> 4, j = (lane >> 2) & 3, q = lane & 3;
  const int col = base + 16 * (g & 1) + 4 * q;
  s16x4 v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = kk * 16 + 8 * (g >> 1) + 4 * h + j;
    v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)(s + r * W + (mn_chunk<W>(r, col >> 3) << 3) + (col & 7)));
  }
  bf16x8 out;
  __builtin_memcpy(&out, v, 16);
  return out;
}

// LP loads into LDS, 16 bytes a lane: from the scalar base and the lane's 32-bit offsets into the
// consecutive 1 KB that start at `to` in the wave's part of a stage.  Neither takes an
// instruction of the vector ALU; each write of M0 and its load have a wait state between.
template <int LP>
__device__ __forceinline__ void dma_lds(const char* base, const uint32_t (&off)[LP], bf16_t* to) {
  static_assert(LP == 1 || LP == 2 || LP == 4, "loads of a wave");
  const uint32_t m = uni((uint32_t)(uintptr_t)((MOE_LDS void*)to));
  const uint64_t b = (uint64_t)(uintptr_t)base;
  const uint64_t sb = ((uint64_t)(uint32_t)uni((int)(b >> 32)) << 32) | (uint32_t)uni((int)b);
  uint32_t saved;   // M0 is the compiler's
#define LOAD1 "s_nop 0\n\tglobal_load_lds_dwordx4 "
#define NEXT "\n\ts_add_u32 m0, m0, 0x400\n\t"
#define FIRST "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\t"
#define LAST "\n\ts_mov_b32 m0, %0"
  if constexpr (LP == 1)
    asm volatile(FIRST LOAD1 "%3, %2" LAST : "=&s"(saved) : "s"(m), "s"(sb), "v"(off[0]) : "memory", "scc");
  else if constexpr (LP == 2)
    asm volatile(FIRST LOAD1 "%3, %2" NEXT LOAD1 "%4, %2" LAST
                 : "=&s"(saved) : "s"(m), "s"(sb), "v"(off[0]), "v"(off[1]) : "memory", "scc");
  else
    asm volatile(FIRST LOAD1 "%3, %2" NEXT LOAD1 "%4, %2" NEXT LOAD1 "%5, %2" NEXT LOAD1 "%6, %2" LAST
                 : "=&s"(saved) : "s"(m), "s"(sb), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]) : "memory", "scc");
#undef FIRST
#undef LAST
#undef LOAD1
#undef NEXT
}

// Where a lane's loads of one operand come from
template <bool KM, int W, int LP>
struct TileLd {
  const char* base;    // of the next step to load (uniform)
  int64_t step;        // bytes a step
  uint32_t off[LP];    // the lane's places
  __device__ __forceinline__ static void slot(int q, int wv, int lane, int& r, int& c) {
    const int s = (wv * LP + q) * 64 + lane;
    if constexpr (KM) kmaj_slot(s, r, c);
    else mn_slot<W>(s, r, c);
  }
  // rows (KM: of ld elements along K) or columns (of a [K, ld] matrix) x0 .. x0 + W - 1 of X
  __device__ __forceinline__ void setup(const bf16_t* m, int64_t ld, int64_t x0, int64_t X, int64_t k0, int wv, int lane) {
    base = (const char*)(m + (KM ? x0 * ld + k0 : k0 * ld + x0));
    step = 2 * (KM ? (int64_t)BK : BK * ld);
    const int most = (int)min(X - x0, (int64_t)W) - 1;   // the last row or column there is
#pragma unroll
    for (int q = 0; q < LP; ++q) {
      int r, c;
      slot(q, wv, lane, r, c);
      // rows and columns past the end: any valid address, their results are discarded
      off[q] = KM ? 2u * (uint32_t)(min(r, most) * (int)ld + c * 8) : 2u * (uint32_t)(r * (int)ld + (c * 8 <= most ? c * 8 : 0));
    }
  }
  // the step that has `left` elements of K to its end
  __device__ __forceinline__ void issue(int64_t left, bf16_t* dst, int wv, int lane) {
    dst += wv * LP * 512;
    if (left >= BK) {
      dma_lds<LP>(base, off, dst);
    } else {
#pragma unroll
      for (int q = 0; q < LP; ++q) {
        int r, c;
        slot(q, wv, lane, r, c);
        const bool in = (KM ? c * 8 : r) < left;
        dma16(in ? (const void*)(base + off[q]) : (const void*)g_zero16, dst + q * 512);
      }
    }
    base += step;
  }
};

struct TileArgs {
  const bf16_t* a;
  const bf16_t* b;
  int64_t lda, ldb;
  int64_t M, N, K;
  int tm, tn;        // tiles
  int splits;
  int64_t ks;        // elements of K a share, a multiple of 64
  float* part;       // shares, or null: one
  Epilogue<bf16_t> e;
};

// Work item of this workgroup: each XCD takes a contiguous range, in bands of 8 rows of tiles
// within which the row runs fastest, so that what runs together shares its operands in one L2
__device__ __forceinline__ bool tile_item(const TileArgs& g, int& mt, int& nt, int& sp) {
  const int V = g.tm * g.tn * g.splits, x = blockIdx.x & 7;
  const int lo = (int)(((int64_t)V * x) >> 3), hi = (int)(((int64_t)V * (x + 1)) >> 3);
  int v = lo + (int)(blockIdx.x >> 3);
  if (v >= hi) return false;
  sp = uni(v / (g.tm * g.tn));
  v -= sp * (g.tm * g.tn);
  const int band = v / (8 * g.tn), h = min(8, g.tm - band * 8);
  v -= band * 8 * g.tn;
  mt = uni(band * 8 + v % h);
  nt = uni(v / h);
  return true;
}

// 8 elements from column c of a row of N on; past its end any there are.  WIDE: the row is whole chunks
template <bool WIDE>
__device__ __forceinline__ i32x4 row_piece(const bf16_t* row, int64_t c, int64_t N) {
  if constexpr (WIDE) return *reinterpret_cast<const i32x4*>(row + min(c, N - 8));
  if (c + 8 <= N) return *reinterpret_cast<const i32x4_a2*>(row + c);
  i32x4 u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    u[j] = (int)((uint32_t)row[min(c + 2 * j, N - 1)] | (uint32_t)row[min(c + 2 * j + 1, N - 1)] << 16);
  return u;
}

// The added matrix's pieces of a band, as band_epilogue takes them; outside of it any valid one.
// Elements one by one take registers that the tile needs: they are loaded where they are added.
template <bool WIDE, int NB>
struct AddBand {
  const bf16_t* row;
  int64_t c, N;
  i32x4 u[WIDE ? NB : 1][2];
  __device__ __forceinline__ void load(const bf16_t* add, int64_t r0, int64_t c0, int64_t M, int64_t N_, int lane) {
    row = add + min(r0 + (lane & 31), M - 1) * N_;
    c = c0 + 8 * (lane >> 5);
    N = N_;
    if constexpr (WIDE)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int s = 0; s < 2; ++s) u[b][s] = row_piece<true>(row, c + 32 * b + 16 * s, N);
  }
  __device__ __forceinline__ i32x4 piece(int b, int s) const {
    if constexpr (WIDE) return u[b][s];
    else return row_piece<false>(row, c + 32 * b + 16 * s, N);
  }
};

// A band of 32 rows and 32 NB columns of C^T accumulators through the epilogue: lanes l and
// l + 32 trade halves so that each has 8 columns of its row in fp32, and the rounded results
// leave through the wave's LDS region as whole row segments.  add: loaded, if e.add is there;
// after(): what to issue ahead of the stores.  FULL: with bias, activation and z.
template <bool FULL, bool WIDE, int NB, class F>
__device__ __forceinline__ void band_epilogue(const Epilogue<bf16_t>& e, const f32x16* acc, const AddBand<WIDE, NB>& add,
                                              int64_t r0, int64_t c0, int64_t M, int64_t N, bf16_t* wreg, int lane,
                                              F&& after) {
  i32x4 chz[NB][2], chy[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[b][8 * s + i]),
                                                        __float_as_uint(acc[b][8 * s + 4 + i]), false, false);
        v[i] = __uint_as_float(r[0]);
        v[4 + i] = __uint_as_float(r[1]);
      }
      float u[8];
      if constexpr (FULL) {
        if (e.bias) {
          const int64_t col = c0 + 32 * b + 16 * s + 8 * (lane >> 5);
          unpack8(row_piece<WIDE>(e.bias, col, N), u);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += u[i];
        }
        if (e.z) chz[b][s] = pack8(v);
        act8(v, e.act);
      }
      if (e.add) {
        unpack8(add.piece(b, s), u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += u[i];
      }
      chy[b][s] = pack8(v);
    }
  after();
  auto put = [&](bf16_t* to, const i32x4 (&ch)[NB][2]) {
    band_store(wreg, ch, [&](int rr, int cb, i32x4 v) {
      const int64_t r = r0 + rr, c = c0 + cb;
      if constexpr (WIDE) {
        if (r < M && c < N) *reinterpret_cast<i32x4*>(to + r * N + c) = v;
      } else if (r < M && c + 8 <= N) {
        *reinterpret_cast<i32x4_a2*>(to + r * N + c) = v;
      } else if (r < M) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < N) to[r * N + c + j] = (bf16_t)((uint32_t)v[j / 2] >> (16 * (j & 1)));
      }
    });
  };
  if constexpr (FULL)
    if (e.z) put(e.z, chz);
  put(e.out, chy);
}

// The products of the stage at st
template <class S, bool AK, bool BKM>
__device__ __forceinline__ void stage_products(const bf16_t* st, f32x16 (&acc)[S::MI][S::NI], int wm, int wn, int lane) {
#pragma unroll
  for (int kk = 0; kk < BK / 16; ++kk) {
    bf16x8 af[S::MI], bf[S::NI];
#pragma unroll
    for (int i = 0; i < S::MI; ++i)
      af[i] = AK ? frag_kmaj(st, wm + i * 32, kk, lane) : mn_frag<S::TM>(st, wm + i * 32, kk, lane);
#pragma unroll
    for (int j = 0; j < S::NI; ++j)
      bf[j] = BKM ? frag_kmaj(st + S::A, wn + j * 32, kk, lane) : mn_frag<S::TN>(st + S::A, wn + j * 32, kk, lane);
#pragma unroll
    for (int i = 0; i < S::MI; ++i)
#pragma unroll
      for (int j = 0; j < S::NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
  }
}

// WIDE: the epilogue's rows are whole 16-byte chunks at multiples of 16
template <class S, bool AK, bool BKM, bool WIDE>
__global__ __launch_bounds__(S::THR, (S::OCC * S::TW + 3) / 4) void k_linear_tile(TileArgs g) {
  constexpr int TW = S::TW;
  __shared__ __attribute__((aligned(16))) bf16_t lds[2 * S::STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wv = uni(tid >> 6);
  int mt, nt, sp;
  if (!tile_item(g, mt, nt, sp)) return;
  const int64_t m0 = (int64_t)mt * S::TM, n0 = (int64_t)nt * S::TN, k0 = sp * g.ks;
  const int64_t kn = min(g.ks, g.K - k0);   // this share's part of K
  const int nk = (int)ceil_div(kn, BK);
  const int wm = wv % S::WMS * (32 * S::MI), wn = wv / S::WMS * (32 * S::NI);
  TileLd<AK, S::TM, S::LA> la;
  TileLd<BKM, S::TN, S::LB> lb;
  la.setup(g.a, g.lda, m0, g.M, k0, wv, lane);
  lb.setup(g.b, g.ldb, n0, g.N, k0, wv, lane);
  f32x16 acc[S::MI][S::NI];
#pragma unroll
  for (int i = 0; i < S::MI; ++i)
#pragma unroll
    for (int j = 0; j < S::NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  auto issue = [&](int kt) {
    bf16_t* const st = lds + (kt & 1) * S::STAGE;
    la.issue(kn - (int64_t)kt * BK, st, wv, lane);
    lb.issue(kn - (int64_t)kt * BK, st + S::A, wv, lane);
  };
  if (nk > 0) issue(0);
  // a copy of the step for each stage, whose addresses are constants of the code
  for (int k = 0; k < nk; k += 2)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int kt = k + c;
      if (kt < nk) {
        // this step's loads have landed, and every wave is done with the stage that the next fill
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (kt + 1 < nk) issue(kt + 1);
        stage_products<S, AK, BKM>(lds + c * S::STAGE, acc, wm, wn, lane);
      }
    }
  if (g.part) {   // the accumulators in their own order
    const size_t item = ((size_t)sp * g.tm + mt) * g.tn + nt;
#pragma unroll
    for (int i = 0; i < S::MI; ++i)
#pragma unroll
      for (int j = 0; j < S::NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float* const to = g.part + ((((item * S::MI + i) * TW + wv) * S::NI + j) * 4 + q) * 256 + lane * 4;
          *reinterpret_cast<f32x4*>(to) = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                               acc[i][j][4 * q + 3]};
        }
    return;
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // every wave is done with the stages
  bf16_t* const wreg = lds + wv * S::BAND;
  AddBand<WIDE, S::NB> add[2];   // of a band and the next
  auto fetch = [&](int i) {
    if (g.e.add) add[i & 1].load(g.e.add, m0 + wm + i * 32, n0 + wn, g.M, g.N, lane);
  };
  fetch(0);
#pragma unroll
  for (int i = 0; i < S::MI; ++i)
    band_epilogue<AK && !BKM, WIDE, S::NB>(g.e, acc[i], add[i & 1], m0 + wm + i * 32, n0 + wn, g.M, g.N, wreg, lane, [&] {
      if (i + 1 < S::MI) fetch(i + 1);
    });
}

// The shares of a tile's bands added in order, and the epilogue: a workgroup for a band of each wave
template <class S, bool FULL, bool WIDE>
__global__ __launch_bounds__(S::THR) void k_linear_join(TileArgs g) {
  constexpr int TW = S::TW;
  __shared__ __attribute__((aligned(16))) bf16_t lds[TW * S::BAND];
  const int tid = threadIdx.x, lane = tid & 63, wv = uni(tid >> 6);
  const int i = blockIdx.x % S::MI, tile = blockIdx.x / S::MI;
  const int mt = tile / g.tn, nt = tile % g.tn;
  const int wm = wv % S::WMS * (32 * S::MI), wn = wv / S::WMS * (32 * S::NI);
  const int64_t r0 = (int64_t)mt * S::TM + wm + i * 32, c0 = (int64_t)nt * S::TN + wn;
  AddBand<WIDE, S::NB> add;
  if (g.e.add) add.load(g.e.add, r0, c0, g.M, g.N, lane);
  f32x16 acc[S::NB];
#pragma unroll
  for (int j = 0; j < S::NB; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[j][r] = 0.f;
  const size_t share = (size_t)g.tm * g.tn * S::MI * TW * S::NI * 1024;
  const float* p = g.part + ((((size_t)tile * S::MI + i) * TW + wv) * S::NI) * 1024 + lane * 4;
#pragma unroll S::NB == 1 ? 8 : 4
  for (int sp = 0; sp < g.splits; ++sp, p += share) {
    f32x4 v[S::NB][4];
#pragma unroll
    for (int j = 0; j < S::NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[j][q] = *reinterpret_cast<const f32x4*>(p + (j * 4 + q) * 256);
#pragma unroll
    for (int j = 0; j < S::NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][4 * q + r] += v[j][q][r];
  }
  band_epilogue<FULL, WIDE, S::NB>(g.e, acc, add, r0, c0, g.M, g.N, lds + wv * S::BAND, lane, [] {});
}

typedef Shape<256, 256, 4, 2, 1> Big;     // 8 waves of 128 x 64
typedef Shape<128, 128, 2, 2, 2> Mid;     // waves of 64 x 64
typedef Shape<64, 64, 1, 1, 4> Small;     // waves of 32 x 32

constexpr PlanCost kCost[3] = {{256, 256, 1, 1.35, 1.6, 7.0, 5.0, 4.0}, {128, 128, 2, 0.65, 0.5, 6.0, 5.0, 4.0},
                                {64, 64, 4, 0.45, 0.182, 4.0, 5.0, 4.0}};
// wide: the largest tiles have no registers for an epilogue element by element.  arrays: 1 and how
// many more the epilogue reads or writes; alone on its CU, a largest tile hides none of them.
Plan plan_of(int64_t M, int64_t N, int64_t K, bool wide, int arrays) {
  PlanCost c[3] = {kCost[0], kCost[1], kCost[2]};
  c[0].over += 4.0 * (arrays - 1);
  const int first = wide ? 0 : 1;
  Plan p = plan_product(c + first, 3 - first, BK, num_cus(), M, N, K);
  p.shape += first;
  return p;
}

template <class S, bool WIDE>
hipError_t run(const char* name, bool a_k, bool b_k, const TileArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)(ceil_div((int64_t)g.tm * g.tn * g.splits, 8) * 8));
  if (a_k && !b_k) MOE_LAUNCH(name, (k_linear_tile<S, true, false, WIDE>), grid, dim3(S::THR), 0, st, g);
  else if (a_k) MOE_LAUNCH(name, (k_linear_tile<S, true, true, WIDE>), grid, dim3(S::THR), 0, st, g);
  else MOE_LAUNCH(name, (k_linear_tile<S, false, false, WIDE>), grid, dim3(S::THR), 0, st, g);
  const dim3 bands((unsigned)(g.tm * g.tn * S::MI));
  if (g.part && a_k && !b_k) MOE_LAUNCH("linear_join", (k_linear_join<S, true, WIDE>), bands, dim3(S::THR), 0, st, g);
  else if (g.part) MOE_LAUNCH("linear_join", (k_linear_join<S, false, WIDE>), bands, dim3(S::THR), 0, st, g);
  return hipGetLastError();
}

}  // namespace

size_t linear_part_bytes(int64_t M, int64_t N, int64_t K) {
  size_t most = 0;
  for (int i = 0; i < 4; ++i) {   // element by element, or wide with 1, 2 or 3 arrays
    const Plan p = plan_of(M, N, K, i > 0, i);
    const PlanCost& c = kCost[p.shape];
    const size_t b = p.splits == 1 ? 0 : (size_t)p.splits * ceil_div(M, c.tm) * ceil_div(N, c.tn) * c.tm * c.tn * 4;
    most = b > most ? b : most;
  }
  return most;
}

hipError_t launch_linear_tiles(const char* name, const bf16_t* a, int64_t lda, bool a_k, const bf16_t* b, int64_t ldb,
                               bool b_k, int64_t M, int64_t N, int64_t K, const LinearOut& o, float* part,
                               hipStream_t st) {
  const Plan p = plan_of(M, N, K, o.wide, 1 + (o.z ? 1 : 0) + (o.add ? 1 : 0));
  TileArgs g{};
  g.a = a; g.b = b; g.lda = lda; g.ldb = ldb; g.M = M; g.N = N; g.K = K;
  g.tm = (int)ceil_div(M, kCost[p.shape].tm); g.tn = (int)ceil_div(N, kCost[p.shape].tn);
  g.splits = p.splits; g.ks = p.ks;
  g.part = p.splits > 1 ? part : nullptr;
  g.e.out = o.out; g.e.z = o.z; g.e.bias = o.bias; g.e.add = o.add; g.e.act = o.act;
  switch (p.shape) {
    case 0: return run<Big, true>(name, a_k, b_k, g, st);
    case 1: return o.wide ? run<Mid, true>(name, a_k, b_k, g, st) : run<Mid, false>(name, a_k, b_k, g, st);
    default: return o.wide ? run<Small, true>(name, a_k, b_k, g, st) : run<Small, false>(name, a_k, b_k, g, st);
  }
}

}  // namespace moe
