// Routing by scores: softmax or sigmoid scores, a balance bias, groups of experts, top-k and
// renormalised weights, with its backward, the experts' counts and the step of the bias.
//
//   s = softmax(l) or sigmoid(l);  c_e = s_e + b_e  (no bias: c_e = l_e, which orders alike)
//   a group's score: the sum of its group_top largest c (of s where there is no bias)
//   the topk_groups best groups, in them the k largest c, ties to the lower id
//   q_j = s_j / sum_i s_i over the chosen (renorm), or s_j;  w_j = scale q_j
//
// A choice is decided where two c differ in their last bits, so c is compared in fp64.  That
// takes longer than fp32 (16384 x 256 in 8 groups: 56 us against 21), so a token is
// routed in fp32 first, with a bound on what fp32 has got wrong; only where two neighbours of the
// order, or the last open group and the first closed one, lie within it is the token routed
// again in fp64 (one in some hundreds, on ordinary logits).
//
// A token takes 16 lanes (up to 256 experts) or 64, its row in their registers: one read of the
// logits, no barrier.  The k + 2 rounds of the selection, each a maximum over the lanes by
// rotations, bound it, not memory: 16384 x 256 (16.8 MB) 21 us, 4096 x 128 without groups 9.  The
// counts go through LDS and are joined by a second launch (3 to 4 us); fewer workgroups than 1024 would
// shorten that and lengthen the forward (30 us at 512).  The backward writes its row once:
// 16384 x 256 in 7 us, 2.7 TB/s.
#include "row_lanes.h"

namespace moe {

namespace {

constexpr int GT = 256;          // threads of a workgroup
constexpr int kMaxGroups = 64;
constexpr int kPadId = 0x7fffffff;

struct GateArgs {
  const float* logits;
  const float* bias;
  const uint8_t* mask;
  int32_t* idx;
  float* w;
  int32_t* part_c;   // [gridDim.x, E], or null
  int T, E, k, score, groups, topk_groups, group_top, renorm;
  float scale;
};

__device__ __forceinline__ bool better(double av, int aid, double bv, int bid) {
  return av > bv || (av == bv && aid < bid);
}

template <int LPR>
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
template <int LPR>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}

// 1 / n!, n = 13 .. 2, then log2 e and ln 2 in two parts: read as scalars, so that they take no
// vector registers from the code around
__constant__ double kExp[15] = {1.0 / 6227020800.0, 1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0,
                                1.0 / 40320.0, 1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5,
                                1.44269504088896340736, 0x1.62e42fefap-1, 0x1.cf79abc9e3b3ap-40};
// exp(d), d <= 0 or NaN, to about 1 unit in the last place: d = n ln 2 + r, |r| <= 0.35, and the
// series of exp(r) to r^13 / 13! (the next term is below 2^-57)
__device__ __forceinline__ double exp_d(double d) {
  const double n = rint(d * kExp[12]);
  const double r = fma(-n, kExp[14], fma(-n, kExp[13], d));
  double p = kExp[0];
#pragma unroll
  for (int i = 1; i < 12; ++i) p = fma(p, r, kExp[i]);
  p = fma(fma(p, r, 1.0), r, 1.0);
  return d < -746.0 ? 0.0 : ldexp(p, (int)n);
}

// exp_neg down to the smallest numbers: the hardware's exponential makes 0 of what lies below
// 2^-126, so the lower half is taken 2^64 higher (h + 64 is exact) and brought back
__device__ __forceinline__ float exp_low(float d) {
  constexpr float L2E = 1.44269502f, L2E_LO = 1.92596302e-8f, LN2 = 0.693147182f;
  const float h = d * L2E;
  const float r = fmaf(d, L2E_LO, fmaf(d, L2E, -h));
  const bool low = h < -64.f;
  const float p = __builtin_amdgcn_exp2f(low ? h + 64.f : h);
  const float q = fmaf(p, r * LN2, p);
  return d < -104.f ? 0.f : low ? q * 0x1p-64f : q;
}

// sigmoid(l) and 1 - sigmoid(l), each to its own last bits; NaN gives NaN
__device__ __forceinline__ void sigmoid2(float l, float& s, float& r) {
  const float e = exp_low(-fabsf(l)), d = 1.f / (1.f + e);
  s = l >= 0.f ? d : e * d;
  r = l >= 0.f ? e * d : d;
}

// Over the 16 lanes of a row by rotations (vector ALU alone), beyond them by exchanges; every
// lane gets the same bits, as each step adds the same two values on both sides
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, false);
}
template <int LPR, class F>
__device__ __forceinline__ float fold(float v, F&& f) {
  v = f(v, __uint_as_float(row_ror<8>(__float_as_uint(v))));
  v = f(v, __uint_as_float(row_ror<4>(__float_as_uint(v))));
  v = f(v, __uint_as_float(row_ror<2>(__float_as_uint(v))));
  v = f(v, __uint_as_float(row_ror<1>(__float_as_uint(v))));
  if constexpr (LPR == 64) {
    v = f(v, __shfl_xor(v, 16, 64));
    v = f(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int LPR>
__device__ __forceinline__ uint32_t fold_max(uint32_t v) {
  v = max(v, row_ror<8>(v));
  v = max(v, row_ror<4>(v));
  v = max(v, row_ror<2>(v));
  v = max(v, row_ror<1>(v));
  if constexpr (LPR == 64) {
    v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    v = max(v, (uint32_t)__shfl_xor((int)v, 32, 64));
  }
  return v;
}
// the bits of a ballot that the lane's token has
template <int LPR>
__device__ __forceinline__ uint64_t token_bits(bool p) {
  const uint64_t b = __ballot(p);
  return LPR == 64 ? b : (b >> (threadIdx.x & 48)) & 0xffffull;
}

// The chosen experts' shares q of lanes sub < k (others 0) from their logits l: sigmoids over
// their sum, scaled by exp(-min(max l, 0)) so that none of the largest underflows, or exp(l)
// over its sum.  All of -inf: 0.
template <int LPR>
__device__ __forceinline__ float shares(float l, bool on, bool sigm) {
  const float m = fold<LPR>(on ? l : -__builtin_inff(), [](float x, float y) { return fmaxf(x, y); });
  float z = 0.f;
  if (on && m != -__builtin_inff()) {
    if (sigm) {
      const float e = exp_low(-fabsf(l));
      z = (l >= 0.f ? 1.f : exp_low(l - fminf(m, 0.f))) / (1.f + e);
    } else {
      z = exp_low(l - m);
    }
  }
  if (on && l != l) z = l;   // also where the row holds nothing but NaN
  const float sum = fold<LPR>(z, [](float x, float y) { return x + y; });
  return sum == 0.f ? 0.f : z / sum;
}

// One token routed in fp64 by a whole wave (c and gscore: LDS of the wave); lane slot0 + j gets
// the id of slot j.  Loops, not copies: it runs seldom, and its registers are everyone's.
__device__ __forceinline__ void route_exact(const GateArgs& a, const float* row, int slot0, double* c, double* gscore,
                                            int& my_id) {
  const int lane = threadIdx.x & 63, E = a.E, per = E / a.groups;
  const bool sigm = a.score == MOE_SCORE_SIGMOID, groups2 = a.groups > 1 && a.group_top > 1;
  const bool scored = a.bias || groups2;
  const double ninf = -__builtin_inf();
  float m = 0.f;
  double inv = 0.0;
  if (scored && !sigm) {
    m = -__builtin_inff();
#pragma unroll 1
    for (int e = lane; e < E; e += 64) m = fmaxf(m, row[e]);
    m = lanes_max<64>(m);
    if (m == -__builtin_inff()) m = 0.f;
    double sum = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 64) sum += exp_d((double)row[e] - (double)m);
    sum = lanes_sum<64>(sum);
    inv = sum > 0.0 ? 1.0 / sum : sum;   // NaN stays
  }
#pragma unroll 1
  for (int e = lane; e < E; e += 64) {
    const float l = row[e];
    double s = l;
    if (scored) {
      const double x = exp_d(sigm ? -fabs((double)l) : (double)l - (double)m);
      s = sigm ? (l >= 0.f ? 1.0 : x) / (1.0 + x) : x * inv;
      if (a.bias) s += (double)a.bias[e];
    }
    c[e] = l > -__builtin_inff() && s == s ? s : ninf;   // masked or not a number: behind every other
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  uint64_t open = ~0ull;
  if (a.groups > 1) {
    double s = ninf;
    if (lane < a.groups) {
      double b1 = ninf, b2 = ninf;
#pragma unroll 1
      for (int e = lane * per; e < (lane + 1) * per; ++e) {
        b2 = fmax(b2, fmin(b1, c[e]));
        b1 = fmax(b1, c[e]);
      }
      s = groups2 ? b1 + b2 : b1;
      if (s != s) s = ninf;
      gscore[lane] = s;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    int rank = 0;   // a group is open if fewer than topk_groups are better
#pragma unroll 1
    for (int o = 0; o < a.groups; ++o) rank += better(gscore[o], o, s, lane);
    open = __ballot(lane < a.groups && rank < a.topk_groups);
    if (!a.bias && groups2) {   // in the groups the logits order the experts
#pragma unroll 1
      for (int e = lane; e < E; e += 64) c[e] = row[e] == row[e] ? (double)row[e] : ninf;
    }
  }
  uint32_t left = 0;   // which of the lane's experts can be chosen
#pragma unroll 1
  for (int e = lane, i = 0; e < E; e += 64, ++i)
    if (a.groups == 1 || (open >> (e / per) & 1)) left |= 1u << i;
#pragma unroll 1
  for (int n = 0; n < a.k; ++n) {
    double bv = ninf;
    int bid = kPadId;
#pragma unroll 1
    for (int e = lane, i = 0; e < E; e += 64, ++i)
      if ((left >> i & 1) && better(c[e], e, bv, bid)) {
        bv = c[e];
        bid = e;
      }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const double ov = __shfl_xor(bv, off, 64);
      const int oid = __shfl_xor(bid, off, 64);
      if (better(ov, oid, bv, bid)) {
        bv = ov;
        bid = oid;
      }
    }
    if ((bid & 63) == lane) left &= ~(1u << (bid >> 6));
    if (lane == slot0 + n) my_id = bid;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// fp32 numbers as whole ones in the same order, above 0; the low bits give way to a slot's place
__device__ __forceinline__ uint32_t sortable(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unsorted(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// What orders an expert, in fp64; NaN and masked ones as -inf
struct Exact {
  const float* row;
  const float* bias;   // or null
  bool scored, sigm;
  float m;             // softmax: the row's largest, and 1 / sum exp(l - m)
  double inv;
  __device__ __forceinline__ double operator()(int e) const {
    const float l = row[e];
    double s = l;
    if (scored) {
      const double x = exp_d(sigm ? -fabs((double)l) : (double)l - (double)m);
      s = sigm ? (l >= 0.f ? 1.0 : x) / (1.0 + x) : x * inv;
      if (bias) s += (double)bias[e];
    }
    return l > -__builtin_inff() && s == s ? s : -__builtin_inf();
  }
};

// A lane's 4 NV columns are kept as keys: the sortable c with its low 4 bits replaced by the
// column's place in the lane, 0 for what cannot be chosen.  A maximum of keys then needs no
// ids: the place is in the key, the lane from a ballot.  What the cut costs (16 units in the last
// place) is counted with fp32's own errors, u = 2^-24:
//   sigmoid: 4 u;  softmax: s (|l - m| + 12) u with s |l - m| <= 0.37 and s at most the row's largest,
//   taken as 2^-19 of that (|l - m| < 20: what is smaller is below any of it);  the sum with b: u |c|
// Two c that differ by more than the two bounds together are in order.  k + 2 rounds give the
// order of the first k + 2: where the k-th and the next, or that one and the next, are apart, the
// first k or k + 1 are the right set, and they are put in order in fp64, a lane each.  Else (ties)
// the whole token is routed again.
template <int LPR, int NV, bool GROUPS>
__global__ __launch_bounds__(GT, 4) void k_gate_fwd(GateArgs a) {
  constexpr int TOK = GT / LPR, COLS = 4 * LPR * NV;
  __shared__ int hist[1024];
  __shared__ float cs[GROUPS ? TOK : 1][GROUPS ? COLS + 4 : 1];     // the c of a token's experts
  __shared__ double gscore[GROUPS ? TOK : 1][GROUPS ? kMaxGroups : 1];
  __shared__ double ce[GT / 64][COLS], ge[GT / 64][GROUPS ? kMaxGroups : 1];
  __shared__ int order[TOK][17];
  const int group = threadIdx.x / LPR;
  const int E = a.E, k = a.k;
  const bool sigm = a.score == MOE_SCORE_SIGMOID, count = a.part_c != nullptr;
  const float inf = __builtin_inff();
  const bool groups2 = GROUPS && a.group_top > 1, scored = a.bias || groups2;
  const int per = GROUPS ? E / a.groups : E;
  if (count) {
    for (int e = threadIdx.x; e < E; e += GT) hist[e] = 0;
    __syncthreads();
  }
  for (int64_t t0 = (int64_t)blockIdx.x * TOK; t0 < a.T; t0 += (int64_t)gridDim.x * TOK) {
    // what follows from the lane's place is worked out anew, not kept in registers over the loop
    int sub = threadIdx.x % LPR;
    asm volatile("" : "+v"(sub));
    const int64_t t = t0 + group < a.T ? t0 + group : a.T - 1;   // all lanes stay
    const bool there = t0 + group < a.T, live = there && (!a.mask || a.mask[t] != 0);
    const float* row = a.logits + (size_t)t * E;
    float c[NV][4];
    float m = -inf, sum = 0.f, err = 0.f;
    load_row<LPR, NV>(row, sub, E, -inf, c);
    if (!sigm && (scored || !a.renorm)) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = fmaxf(m, c[i][j]);
      m = fold<LPR>(m, [](float x, float y) { return fmaxf(x, y); });
      if (m == -inf) m = 0.f;
    }
    const float m0 = m;
    // the scores; bit p of `out`: the lane's p-th expert is masked or not a number
    uint32_t out = 0;
    float p[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float l = c[i][j];
        if (!(l > -inf)) out |= 1u << (4 * i + j);
        if (sigm) {
          const float e = exp_neg(-fabsf(l)), d = 1.f / (1.f + e);
          p[i][j] = l >= 0.f ? d : e * d;
        } else {
          p[i][j] = exp_neg(l - m0);
          sum += p[i][j];
        }
      }
      __builtin_amdgcn_sched_barrier(0);   // a few at a time: registers
    }
    if (!sigm && (scored || !a.renorm)) sum = fold<LPR>(sum, [](float x, float y) { return x + y; });
    const bool by_logit = !a.bias;   // in the groups, too
    const float inv = sigm ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
    if (scored) err = sigm ? 0x1p-22f : 0x1p-19f * inv;   // (the row's largest score is inv)
#pragma unroll
    for (int i = 0; i < NV; ++i) {   // c: what orders the experts; what the groups go by to LDS
      f32x4 u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool no = out >> (4 * i + j) & 1;
        float s = 0.f;
        if (scored) {
          s = fmaf(p[i][j], inv, a.bias ? a.bias[min(4 * (sub + LPR * i) + j, E - 1)] : 0.f);
          s = no || s != s ? -inf : s;
        }
        if (by_logit) c[i][j] = no ? -inf : c[i][j] + 0.f;   // -0 as 0: keys tell them apart
        else c[i][j] = s;
        u[j] = scored ? s : c[i][j];
      }
      if constexpr (GROUPS) *reinterpret_cast<f32x4*>(&cs[group][4 * (sub + LPR * i)]) = u;
    }
    const Exact exact0{row, a.bias, scored, sigm, m0, 0.0};
    // 1 / sum exp(l - m) of the lanes' tokens in fp64 (softmax alone has one)
    auto exact_of = [&]() {
      Exact x = exact0;
      if (scored && !sigm) {
        double z = 0.0;
#pragma unroll 1
        for (int e = sub; e < E; e += LPR) z += exp_d((double)row[e] - (double)m0);
        z = lanes_sum<LPR>(z);
        x.inv = z > 0.0 ? 1.0 / z : z;   // NaN stays
      }
      return x;
    };
    bool whole = false;   // the token has to be routed again as a whole
    uint64_t open = ~0ull;
    if constexpr (GROUPS) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // 2^h lanes to a group, so many groups at a time; low, high: the lowest open score and the
      // highest closed one; size: the largest sum of the sizes of a score's terms, that are not infinite
      int h = 0;
      while ((a.groups << (h + 1)) <= LPR) ++h;
      const int gl = 1 << h;
      uint64_t mine = 0;
      double low = 0.0, high = 0.0;
      float size = 0.f;
      auto score_groups = [&](auto&& value) {
        for (int g0 = 0; g0 < a.groups; g0 += LPR >> h) {
          const int g = g0 + (sub >> h);
          double b1 = -inf, b2 = -inf;
          value(g, sub & (gl - 1), gl, b1, b2);
#pragma unroll 1
          for (int off = 1; off < gl; off <<= 1) {
            const double o1 = __shfl_xor(b1, off, 64), o2 = __shfl_xor(b2, off, 64);
            b2 = fmax(fmin(b1, o1), fmax(b2, o2));
            b1 = fmax(b1, o1);
          }
          if (g < a.groups && (sub & (gl - 1)) == 0) {
            const double s = groups2 ? b1 + b2 : b1;
            gscore[group][g] = s == s ? s : -inf;
            const float z1 = fabsf((float)b1), z2 = groups2 ? fabsf((float)b2) : 0.f;
            size = fmaxf(size, (z1 < inf ? z1 : 0.f) + (z2 < inf ? z2 : 0.f));
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        mine = 0;
        low = inf, high = -inf;
        for (int g = sub; g < a.groups; g += LPR) {   // open if fewer than topk_groups are better
          const double s = gscore[group][g];
          int rank = 0;
#pragma unroll 4
          for (int o = 0; o < a.groups; ++o) rank += better(gscore[group][o], o, s, g);
          if (rank < a.topk_groups) {
            mine |= 1ull << g;
            low = fmin(low, s);
          } else {
            high = fmax(high, s);
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int off = LPR / 2; off >= 1; off >>= 1) mine |= (uint64_t)__shfl_xor((unsigned long long)mine, off, 64);
      };
      score_groups([&](int g, int e0, int step, double& b1, double& b2) {
        float x1 = -inf, x2 = -inf;
        if (g < a.groups)
#pragma unroll 4
          for (int e = e0; e < per; e += step) {
            const float x = cs[group][g * per + e];
            x2 = fmaxf(x2, fminf(x1, x));
            x1 = fmaxf(x1, x);
          }
        b1 = x1, b2 = x2;
      });
      open = mine;
      if (scored && a.topk_groups < a.groups) {   // logits alone have no error
        const float lo = fold<LPR>((float)low, [](float x, float y) { return fminf(x, y); });
        const float hi = fold<LPR>((float)high, [](float x, float y) { return fmaxf(x, y); });
        const float sz = fold<LPR>(size, [](float x, float y) { return fmaxf(x, y); });
        // two scores of two c each: their errors, and the roundings of c = s + b, u of each (a sum may be far
        // smaller than its terms), of the scores to fp32 and of this difference: 8 u of the terms in all
        const bool unsure = !(lo - hi > 4.f * err + sz * 0x1p-21f);
        if (__ballot(unsure && live) != 0) {
          const Exact x = exact_of();
          score_groups([&](int g, int e0, int step, double& b1, double& b2) {
            if (g < a.groups)
#pragma unroll 1
              for (int e = e0; e < per; e += step) {
                const double y = x(g * per + e);
                b2 = fmax(b2, fmin(b1, y));
                b1 = fmax(b1, y);
              }
          });
          if (unsure) open = mine;
        }
      }
    }
    if (by_logit) err = 0.f;
    uint32_t key[NV][4];
    const float inv_per = 1.f / (float)per;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 4 * (sub + LPR * i) + j;
        bool in = e < E;
        // e / per: (e + 1/2) / per lies 1 / (2 per) >= 2^-11 from a whole number, past its rounding
        if constexpr (GROUPS) in = in && (open >> (int)(((float)e + 0.5f) * inv_per) & 1);
        key[i][j] = in ? (sortable(c[i][j]) & ~15u) | (uint32_t)(4 * i + j) : 0u;
      }
    int my_id = 0;
    float last = 0.f;
    bool near = false, at_k = false;   // neighbours among the first k, and the k-th and the next
    for (int n = 0; n < k + 2; ++n) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) best = max(best, max(max(key[i][0], key[i][1]), max(key[i][2], key[i][3])));
      const uint32_t all = fold_max<LPR>(best);
      const float f = unsorted(all & ~15u);
      // the cut takes at most 15 units of 2^-23 off, downwards as the order goes
      if (n > 0 && all != 0) {
        const bool close = !(last - f > 2.f * err + fmaxf(fabsf(last), fabsf(f)) * 0x1p-18f);
        if (n < k) near |= close;
        else if (n == k) at_k = close;
        else whole |= at_k && close;
      }
      last = f;
      if (n == k + 1) break;
      const uint64_t who = token_bits<LPR>(best == all);
      if (n < k) near |= (who & (who - 1)) != 0;   // two lanes' keys alike
      else at_k |= all != 0 && (who & (who - 1)) != 0;
      whole |= all != 0 && (who & (who - 1)) != 0;
      const int lane = LPR == 64 ? __builtin_ctzll(who) : __builtin_ctz((uint32_t)who);
      const int place = (int)(all & 15u);
      if (sub == n) my_id = all != 0 ? 4 * (lane + LPR * (place >> 2)) + (place & 3) : kPadId;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) key[i][j] = key[i][j] == all ? 0u : key[i][j];
    }
    if (LPR == 16 && k == 16) whole |= at_k;   // no lane for the seventeenth
    if (__ballot((near || at_k) && !whole && live) != 0) {
      // without a bias by the logits, as the keys: their scores may be equal
      Exact x = exact0;
      if (!by_logit) x = exact_of();
      x.scored = !by_logit;
      const int most = at_k && k < LPR ? k + 1 : k;   // the right set
      const bool cand = sub < most && my_id != kPadId;
      const double y = cand ? x(my_id) : 0.0;
      int rank = 0;
#pragma unroll 1
      for (int n = 0; n <= k && n < LPR; ++n) {
        const int src = (threadIdx.x & 63) - sub + n;
        const double o = __shfl(y, src, 64);
        const int oid = __shfl(cand ? my_id : kPadId, src, 64);
        rank += oid != kPadId && better(o, oid, y, my_id);
      }
      if (cand) order[group][rank] = my_id;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if ((near || at_k) && sub < k) my_id = order[group][sub];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    for (uint64_t todo = __ballot(whole && live); todo != 0;) {   // token by token
      const int slot0 = __builtin_ctzll(todo) / LPR * LPR;
      todo &= LPR == 64 ? 0 : ~(0xffffull << slot0);
      route_exact(a, a.logits + (size_t)__shfl(t, slot0, 64) * E, slot0, ce[threadIdx.x >> 6], ge[threadIdx.x >> 6],
                  my_id);
    }
    // what is not live has not been routed again: its ids may be none
    const bool on = sub < k && live;
    const float l = on ? row[my_id] : 0.f;
    float q;
    if (a.renorm) {
      q = shares<LPR>(l, on, sigm);
    } else if (sigm) {
      float r;
      sigmoid2(l, q, r);
    } else {
      q = sum == 0.f ? 0.f : exp_low(l - m0) / sum;
    }
    if (sub < k && there) {
      a.idx[t * k + sub] = live ? my_id : -1;
      a.w[t * k + sub] = live ? a.scale * q : 0.f;
      if (count && live) atomicAdd(&hist[my_id], 1);
    }
  }
  if (count) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += GT) a.part_c[(size_t)blockIdx.x * E + e] = hist[e];
  }
}

// counts[e] = the workgroups' shares added up: 64 experts a workgroup, 16 slices of the shares
constexpr int CT = 1024;
__global__ __launch_bounds__(CT) void k_gate_counts(const int32_t* __restrict__ part_c, int W, int E,
                                                    int32_t* __restrict__ counts) {
  __shared__ int red[CT];
  const int e = blockIdx.x * 64 + (threadIdx.x & 63);
  int c = 0;
  if (e < E)
    #pragma unroll 8
    for (int w = threadIdx.x >> 6; w < W; w += CT / 64) c += part_c[(size_t)w * E + e];
  red[threadIdx.x] = c;
  __syncthreads();
  if (threadIdx.x < 64 && e < E) {
    for (int s = 1; s < CT / 64; ++s) c += red[threadIdx.x + 64 * s];
    counts[e] = c;
  }
}

// b_e + rate sign(sum c / E - c_e), the mean compared in whole numbers
__global__ __launch_bounds__(CT) void k_gate_bias(const int32_t* __restrict__ counts, const float* bias, int E,
                                                  float rate, float* out) {
  __shared__ long long red[CT / 64];
  const int e = threadIdx.x;
  const long long c = e < E ? counts[e] : 0;
  long long n = c;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off, 64);
  if ((e & 63) == 0) red[e >> 6] = n;
  __syncthreads();
  n = 0;
  for (int w = 0; w < CT / 64; ++w) n += red[w];
  if (e < E) {
    const long long d = n - c * E;
    out[e] = bias[e] + (d > 0 ? rate : d < 0 ? -rate : 0.f);
  }
}

template <int LPR, int NV>
__global__ __launch_bounds__(GT) void k_gate_bwd(GateArgs a, const int32_t* __restrict__ idx,
                                                 const float* __restrict__ dw, float* __restrict__ d_logits) {
  constexpr int TOK = GT / LPR;
  const int sub = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int E = a.E, k = a.k;
  const int64_t t = (int64_t)blockIdx.x * TOK + group;
  if (t >= a.T) return;
  const bool sigm = a.score == MOE_SCORE_SIGMOID;
  const float* row = a.logits + (size_t)t * E;
  const int id = sub < k ? idx[t * k + sub] : -1;
  const bool on = id >= 0 && id < E;
  const float l = on ? row[id] : -__builtin_inff();
  const float d = on ? dw[t * k + sub] : 0.f;
  const bool any = group_sum<LPR>(on ? 1.f : 0.f) > 0.f;
  const bool whole = any && !sigm && !a.renorm;   // every expert's probability has a gradient
  float o[NV][4], p[NV][4];
  float g = 0.f, inv = 0.f, dot = 0.f;
  if (whole) {
    load_row<LPR, NV>(row, sub, E, -__builtin_inff(), p);
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, p[i][j]);
    m = lanes_max<LPR>(m);
    if (m == -__builtin_inff()) m = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[i][j] = exp_low(p[i][j] - m);
        sum += p[i][j];
      }
    sum = group_sum<LPR>(sum);
    inv = sum == 0.f ? 0.f : 1.f / sum;
    dot = group_sum<LPR>(on ? exp_low(l - m) * inv * d : 0.f);
    g = d;
  } else if (a.renorm) {
    const float q = shares<LPR>(l, on, sigm);
    dot = group_sum<LPR>(q * d);
    g = a.scale * q * (d - dot);
    if (sigm) {
      float s, r;
      sigmoid2(l, s, r);
      g *= r;
    }
  } else {
    float s, r;
    sigmoid2(l, s, r);
    g = a.scale * s * r * d;
  }
  if (!on) g = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  for (int n = 0; n < k; ++n) {
    const int src = (threadIdx.x & 63) - sub + n;
    const int id_n = __shfl(on ? id : -1, src, 64);
    const float g_n = __shfl(g, src, 64);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (4 * (sub + LPR * i) + j == id_n) o[i][j] += g_n;
  }
  if (whole) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = a.scale * (p[i][j] * inv) * (o[i][j] - dot);
  }
  float* out = d_logits + (size_t)t * E;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 4 * (sub + LPR * i);
    if (e + 4 <= E) {
      f32x4 u;
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = o[i][j];
      *reinterpret_cast<f32x4_a4*>(out + e) = u;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e + j < E) out[e + j] = o[i][j];
    }
  }
}

// lanes of a row (16 at least: a lane for each chosen expert) and vectors of four columns a lane
#define GATE_DISPATCH(E, CALL)             \
  do {                                     \
    if ((E) <= 64) { CALL(16, 1); }        \
    else if ((E) <= 128) { CALL(16, 2); }  \
    else if ((E) <= 256) { CALL(16, 4); }  \
    else if ((E) <= 512) { CALL(64, 2); }  \
    else { CALL(64, 4); }                  \
  } while (0)

inline int tokens_of(int E) { return GT / (E <= 256 ? 16 : 64); }
// workgroups of a launch, far below what a launch takes (2^32 threads: beyond, the runtime cuts it off in silence)
constexpr int64_t kMostGroups = 1 << 22;

GateArgs gate_args(const moe_gate_shape& s, const float* logits) {
  GateArgs a{};
  a.logits = logits;
  a.T = s.T; a.E = s.E; a.k = s.k; a.score = s.score; a.groups = s.groups; a.topk_groups = s.topk_groups;
  a.group_top = s.group_top; a.renorm = s.renorm; a.scale = s.scale;
  return a;
}

}  // namespace

// Workgroups of a counting forward, each with a share of the counts
int gate_parts(int T, int E) {
  const int64_t w = ceil_div(T, tokens_of(E));
  return (int)(w < 1 ? 1 : w > 1024 ? 1024 : w);
}

hipError_t launch_gate_fwd(const moe_gate_shape& s, const float* logits, const float* bias, const uint8_t* mask,
                           int32_t* idx, float* w, int32_t* counts, int32_t* part_c, hipStream_t st) {
  GateArgs a = gate_args(s, logits);
  a.bias = bias; a.mask = mask; a.idx = idx; a.w = w;
  a.part_c = counts ? part_c : nullptr;
  const int64_t all = ceil_div(s.T, tokens_of(s.E));
  const unsigned W = counts ? (unsigned)gate_parts(s.T, s.E) : (unsigned)(all < kMostGroups ? all : kMostGroups);
  if (W > 0) {
#define CALL(LPR, NV)                                                                              \
  if (s.groups > 1) MOE_LAUNCH("gate_fwd", (k_gate_fwd<LPR, NV, true>), dim3(W), dim3(GT), 0, st, a); \
  else MOE_LAUNCH("gate_fwd", (k_gate_fwd<LPR, NV, false>), dim3(W), dim3(GT), 0, st, a)
    GATE_DISPATCH(s.E, CALL);
#undef CALL
  }
  if (counts)
    MOE_LAUNCH("gate_counts", k_gate_counts, dim3((unsigned)ceil_div(s.E, 64)), dim3(CT), 0, st, part_c, (int)W, s.E,
               counts);
  return hipGetLastError();
}

hipError_t launch_gate_bwd(const moe_gate_shape& s, const float* logits, const int32_t* idx, const float* dw,
                           float* d_logits, hipStream_t st) {
  GateArgs a = gate_args(s, logits);
  const int64_t most = kMostGroups * tokens_of(s.E);   // tokens of a launch
  for (int64_t t = 0; t < s.T; t += most) {
    a.T = (int)(s.T - t < most ? s.T - t : most);
    a.logits = logits + t * s.E;
    const dim3 grid((unsigned)ceil_div(a.T, tokens_of(s.E)));
#define CALL(LPR, NV) \
  MOE_LAUNCH("gate_bwd", (k_gate_bwd<LPR, NV>), grid, dim3(GT), 0, st, a, idx + t * s.k, dw + t * s.k, d_logits + t * s.E)
    GATE_DISPATCH(s.E, CALL);
#undef CALL
  }
  return hipGetLastError();
}

hipError_t launch_gate_bias(const moe_gate_shape& s, const int32_t* counts, const float* bias, float rate, float* out,
                            hipStream_t st) {
  MOE_LAUNCH("gate_bias", k_gate_bias, dim3(1), dim3(CT), 0, st, counts, bias, s.E, rate, out);
  return hipGetLastError();
}

}  // namespace moe
