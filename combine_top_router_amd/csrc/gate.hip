// Routing by scores: softmax or sigmoid scores, a balance bias, groups of experts, top-k and
// renormalised weights, with its backward, the experts' counts and the step of the bias.
//
//   s = softmax(l) or sigmoid(l);  c_e = s_e + b_e  (no bias: c_e = l_e, which orders alike)
//   a group's score: the sum of its group_top largest c (of s where there is no bias)
//   the topk_groups best groups, in them the k largest c, ties to the lower id
//   q_j = s_j / sum_i s_i over the chosen (renorm), or s_j;  w_j = scale q_j
// A choice is decided where two c differ in their last bits, so c is compared in fp64; the
// weights and gradients are fp32.
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

__device__ __forceinline__ double sigmoid_d(double l) {
  const double e = exp(-fabs(l));
  return (l >= 0.0 ? 1.0 : e) / (1.0 + e);
}
// sigmoid(l) and 1 - sigmoid(l), each to its own last bits; NaN gives NaN
__device__ __forceinline__ void sigmoid2(float l, float& s, float& r) {
  const float e = exp_low(-fabsf(l)), d = 1.f / (1.f + e);
  s = l >= 0.f ? d : e * d;
  r = l >= 0.f ? e * d : d;
}

// The chosen experts' shares q of lanes sub < k (others 0) from their logits l: sigmoids over
// their sum, scaled by exp(-min(max l, 0)) so that none of the largest underflows, or exp(l)
// over its sum.  All of -inf: 0.
template <int LPR>
__device__ __forceinline__ float shares(float l, bool on, bool sigm) {
  const float m = lanes_max<LPR>(on ? l : -__builtin_inff());
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
  const float sum = group_sum<LPR>(z);
  return sum == 0.f ? 0.f : z / sum;
}

template <int LPR, int NV>
__global__ __launch_bounds__(GT) void k_gate_fwd(GateArgs a) {
  constexpr int TOK = GT / LPR;
  __shared__ int hist[1024];
  __shared__ double gscore[TOK][kMaxGroups];
  const int sub = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int E = a.E, k = a.k;
  const bool sigm = a.score == MOE_SCORE_SIGMOID, count = a.part_c != nullptr;
  const double ninf = -__builtin_inf();
  if (count) {
    for (int e = threadIdx.x; e < E; e += GT) hist[e] = 0;
    __syncthreads();
  }
  for (int64_t t = (int64_t)blockIdx.x * TOK + group; t < a.T; t += (int64_t)gridDim.x * TOK) {
    if (a.mask && a.mask[t] == 0) {
      if (sub < k) {
        a.idx[t * k + sub] = -1;
        a.w[t * k + sub] = 0.f;
      }
      continue;
    }
    const float* row = a.logits + (size_t)t * E;
    float v[NV][4];
    load_row<LPR, NV>(row, sub, E, -__builtin_inff(), v);
    double c[NV][4];
    float m = -__builtin_inff();
    double sum = 0.0;
    const bool scored = a.bias || (a.groups > 1 && a.group_top > 1);
    if (!sigm && (scored || !a.renorm)) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = fmaxf(m, v[i][j]);
      m = lanes_max<LPR>(m);
      if (m == -__builtin_inff()) m = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[i][j] = exp((double)v[i][j] - (double)m);
          sum += c[i][j];
        }
      sum = lanes_sum<LPR>(sum);
    }
    if (scored) {
      const double inv = sum > 0.0 ? 1.0 / sum : sum;   // NaN stays
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * (sub + LPR * i) + j;
          double s = sigm ? sigmoid_d((double)v[i][j]) : c[i][j] * inv;
          if (a.bias && e < E) s += (double)a.bias[e];
          // masked or not a number: behind every other
          c[i][j] = v[i][j] > -__builtin_inff() && s == s ? s : ninf;
        }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = v[i][j] == v[i][j] ? (double)v[i][j] : ninf;
    }
    uint64_t open = ~0ull;
    if (a.groups > 1) {
      const int per = E / a.groups;
      for (int g = 0; g < a.groups; ++g) {
        double b1 = ninf, b2 = ninf;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 4 * (sub + LPR * i) + j;
            if (e >= g * per && e < (g + 1) * per) {
              b2 = fmax(b2, fmin(b1, c[i][j]));
              b1 = fmax(b1, c[i][j]);
            }
          }
#pragma unroll
        for (int off = LPR / 2; off >= 1; off >>= 1) {
          const double o1 = __shfl_xor(b1, off, 64), o2 = __shfl_xor(b2, off, 64);
          b2 = fmax(fmin(b1, o1), fmax(b2, o2));
          b1 = fmax(b1, o1);
        }
        double s = a.group_top > 1 ? b1 + b2 : b1;
        if (s != s) s = ninf;
        if (sub == 0) gscore[group][g] = s;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // a group is open if fewer than topk_groups are better
      uint64_t mine = 0;
      for (int g = sub; g < a.groups; g += LPR) {
        const double s = gscore[group][g];
        int rank = 0;
        for (int o = 0; o < a.groups; ++o) rank += better(gscore[group][o], o, s, g);
        if (rank < a.topk_groups) mine |= 1ull << g;
      }
#pragma unroll
      for (int off = LPR / 2; off >= 1; off >>= 1) mine |= (uint64_t)__shfl_xor((unsigned long long)mine, off, 64);
      open = mine;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (!a.bias && a.group_top > 1) {   // in the groups the logits order the experts
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) c[i][j] = v[i][j] == v[i][j] ? (double)v[i][j] : ninf;
      }
    }
    bool taken[NV][4];
    const int per = E / a.groups;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 4 * (sub + LPR * i) + j;
        taken[i][j] = e >= E || (a.groups > 1 && !(open >> (e / per) & 1));
      }
    int my_id = 0;
    for (int n = 0; n < k; ++n) {
      double bv = ninf;
      int bid = kPadId;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 4 * (sub + LPR * i) + j;
          if (!taken[i][j] && better(c[i][j], e, bv, bid)) { bv = c[i][j]; bid = e; }
        }
#pragma unroll
      for (int off = LPR / 2; off >= 1; off >>= 1) {
        const double ov = __shfl_xor(bv, off, 64);
        const int oid = __shfl_xor(bid, off, 64);
        if (better(ov, oid, bv, bid)) { bv = ov; bid = oid; }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * (sub + LPR * i) + j == bid) taken[i][j] = true;
      if (sub == n) my_id = bid;
    }
    const bool on = sub < k;
    const float l = on ? row[my_id] : 0.f;
    float q;
    if (a.renorm) {
      q = shares<LPR>(l, on, sigm);
    } else if (sigm) {
      float r;
      sigmoid2(l, q, r);
    } else {
      q = (float)(exp((double)l - (double)m) / sum);
      if (sum == 0.0) q = 0.f;
    }
    if (on) {
      a.idx[t * k + sub] = my_id;
      a.w[t * k + sub] = a.scale * q;
      if (count) atomicAdd(&hist[my_id], 1);
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
  return (int)(w < 1 ? 1 : w > 512 ? 512 : w);
}

hipError_t launch_gate_fwd(const moe_gate_shape& s, const float* logits, const float* bias, const uint8_t* mask,
                           int32_t* idx, float* w, int32_t* counts, int32_t* part_c, hipStream_t st) {
  GateArgs a = gate_args(s, logits);
  a.bias = bias; a.mask = mask; a.idx = idx; a.w = w;
  a.part_c = counts ? part_c : nullptr;
  const unsigned W = counts ? (unsigned)gate_parts(s.T, s.E) : (unsigned)ceil_div(s.T, tokens_of(s.E));
  if (W > 0) {
#define CALL(LPR, NV) MOE_LAUNCH("gate_fwd", (k_gate_fwd<LPR, NV>), dim3(W), dim3(GT), 0, st, a)
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
  const GateArgs a = gate_args(s, logits);
  const dim3 grid((unsigned)ceil_div(s.T, tokens_of(s.E)));
#define CALL(LPR, NV) MOE_LAUNCH("gate_bwd", (k_gate_bwd<LPR, NV>), grid, dim3(GT), 0, st, a, idx, dw, d_logits)
  GATE_DISPATCH(s.E, CALL);
#undef CALL
  return hipGetLastError();
}

hipError_t launch_gate_bias(const moe_gate_shape& s, const int32_t* counts, const float* bias, float rate, float* out,
                            hipStream_t st) {
  MOE_LAUNCH("gate_bias", k_gate_bias, dim3(1), dim3(CT), 0, st, counts, bias, s.E, rate, out);
  return hipGetLastError();
}

}  // namespace moe
