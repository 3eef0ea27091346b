// One AdamW step over many tensors in one launch (per 40 tensors), moments in fp32 or 8 bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
// in fp32, from the new m and v before they are rounded.
//
// 8 bits: m and sqrt(v) as E4M3 codes, 32 consecutive elements sharing a power of two (the
// scale rule of mx_scale_exp).  sqrt(v) has half v's range in exponents, and its relative
// step of 1/8 at most is what the update sees.  Rounded to nearest, a moment whose step
// changes it by less than half a code stands still (at b2 = 0.95 every decay of v); rounded
// stochastically it moves on average as it should.  A v above 0 keeps the smallest code at
// least: as 0 it would leave m / eps.
// Random bits: 32 per element, h = mix(lo(i) ^ mix(hi(i) + k)) with i the element's place
// (moe_adamw_tensor::at), k = mix(t + mix(lo(seed) + mix(hi(seed)))) and mix the output
// permutation of PCG (O'Neill 2014): m takes the low half, sqrt(v) the high one, and a
// stochastically rounded bf16 parameter the low half of mix(h).
//
// Every tensor's pieces of 2048 elements are workgroups of one grid, found by a search in a table
// that travels with the arguments (no memory to fill ahead of a launch): 24 small tensors take 7 us.
// Large ones are bound by memory: bf16 parameters with fp32 states and copies (28 bytes an element,
// 100 M elements) 517 us, 5.4 TB/s; 8-bit states, stochastic (10 bytes, 201 M) 506, 4.0 TB/s, where
// the random bits, codes and roots, about 70 instructions an element, run nearly as long (481 with the
// hardware's root, which is off by 1 ulp at most and so takes another code for some in a million).
#include "common.h"

namespace moe {

namespace {

constexpr int AT = 256;       // threads of a workgroup
constexpr int VEC = 8;        // elements a thread takes at a time
constexpr int CHUNK = AT * VEC;
constexpr int kTensors = 40;  // tensors of a launch: their table travels with its arguments
// workgroups of a launch: 2^31 threads (from 2^32 on the runtime cuts a launch off in silence)
constexpr int64_t kMostGroups = (1LL << 31) / AT;

struct AdamwTable {
  moe_adamw_tensor t[kTensors];
  uint32_t first[kTensors];   // a tensor's first workgroup
  int n;
};
static_assert(sizeof(AdamwTable) <= 3600, "the arguments of a launch hold 4 KB");

struct AdamwHyper {
  float b1, b1c, b2, b2c;     // beta and 1 - beta
  float decay, rate, root;    // 1 - lr wd; lr / (1 - b1^t); 1 / sqrt(1 - b2^t)
  float eps, wd;
  float to_m;                 // 1 / (1 - b1^t)
  uint32_t key;               // the step's random key
  int stochastic;
  const float* lr;            // device, or null
  const float* grad_scale;    // device, or null
  const AdamwClock* clock;    // device, or null
};

__host__ __device__ inline uint32_t mix(uint32_t v) {
  const uint32_t s = v * 747796405u + 2891336453u;
  const uint32_t w = ((s >> ((s >> 28) + 4)) ^ s) * 277803737u;
  return (w >> 22) ^ w;
}
__host__ __device__ inline uint32_t step_key(uint64_t seed, int64_t t) {
  return mix((uint32_t)t + mix((uint32_t)seed + mix((uint32_t)(seed >> 32))));
}

// The E4M3 code of y >= 0 (at most 448), up with r16 / 2^16 below the part that is cut off.  From
// 2^-6 on the code is the fp32 number's exponent and upper 3 bits, less 960 for the bias; 20
// bits are cut.  Below, the grid is that of 2^-9: y 2^29 cuts the same 20 bits (rounded up to
// a whole number, which leaves every comparison with 16 r16 as it is).  Adding 2^20 - 1 - 16 r16
// carries where the cut part is above 16 r16.
__device__ __forceinline__ uint32_t e4m3_stochastic(float y, uint32_t room) {   // room = 2^20 - 1 - 16 r16
  const uint32_t norm = __float_as_uint(y) - (960u << 20), sub = (uint32_t)ceilf(y * 0x1p29f);
  return ((y < 0x1p-6f ? sub : norm) + room) >> 20;
}

// 2^X, X in -127 .. 127; 128 (a scale of 255, that no code written here has) as 127: its zeros stay zeros
__device__ __forceinline__ float power(int X) {
  return __uint_as_float(X > -127 ? (uint32_t)(min(X, 127) + 127) << 23 : 0x400000u);
}

// The 8 values of a thread, 4 threads to a block of 32, as codes and the block's scale.
// What is not finite becomes NaN and does not move the scale; FINITE: nothing is.
template <bool ROOT, bool FINITE>
__device__ __forceinline__ void encode(const float (&x)[VEC], const uint32_t (&h)[VEC], bool stochastic, uint2& codes,
                                       int& X) {
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float a = fabsf(x[i]);
    am = fmaxf(am, FINITE || a < __builtin_inff() ? a : 0.f);
  }
  am = fmaxf(am, __shfl_xor(am, 1, 64));
  am = fmaxf(am, __shfl_xor(am, 2, 64));
  X = mx_scale_exp(am);
  const float inv = power(-X);
  uint32_t c[VEC];
  if (stochastic) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const uint32_t r = ROOT ? h[i] >> 16 : h[i] & 0xffffu;
      float a = fabsf(x[i]);
      if (!FINITE) a = a < __builtin_inff() ? a : 0.f;
      c[i] = e4m3_stochastic(a * inv, ((r ^ 0xffffu) << 4) | 15u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      const float a = FINITE || fabsf(x[i]) < __builtin_inff() ? fabsf(x[i]) : 0.f;
      const float b = FINITE || fabsf(x[i + 1]) < __builtin_inff() ? fabsf(x[i + 1]) : 0.f;
      const uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
      c[i] = w & 0xffu;
      c[i + 1] = w >> 8 & 0xffu;
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    if (ROOT) c[i] = max(c[i], min(__float_as_uint(x[i]), 1u));   // what is above 0 stays above 0
    else c[i] |= __float_as_uint(x[i]) >> 24 & 0x80u;
    if (!FINITE && !(fabsf(x[i]) < __builtin_inff())) c[i] = 0x7fu;
  }
  codes.x = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
  codes.y = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
}

__device__ __forceinline__ void decode(uint2 c, int X, float (&x)[VEC]) {
  const float f = power(X);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = (int)(h ? c.y : c.x);
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    x[4 * h] = lo[0] * f; x[4 * h + 1] = lo[1] * f;
    x[4 * h + 2] = hi[0] * f; x[4 * h + 3] = hi[1] * f;
  }
}

// a x + b y, each product and the sum rounded by itself: with gradients of few bits b1 m + (1 - b1) g
// often lies halfway between two codes in fp32, and a fused product would take the other one
__device__ __forceinline__ float blend(float a, float x, float b, float y) {
#pragma clang fp contract(off)
  return a * x + b * y;
}

// elements i .. i + 7 of a tensor of n; whole: all inside and the address at a multiple of 16
__device__ __forceinline__ void load8(const void* p, int dtype, int64_t i, int64_t n, bool whole, float (&x)[VEC]) {
  if (dtype == MOE_BF16) {
    const bf16_t* q = (const bf16_t*)p + i;
    if (whole) {
      const i32x4 u = *reinterpret_cast<const i32x4*>(q);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float((uint32_t)u[j] << 16);
        x[2 * j + 1] = __uint_as_float((uint32_t)u[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[j] = i + j < n ? bf2f(q[j]) : 0.f;
    }
  } else {
    const float* q = (const float*)p + i;
    if (whole) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(q), b = *reinterpret_cast<const f32x4*>(q + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = a[j];
        x[4 + j] = b[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[j] = i + j < n ? q[j] : 0.f;
    }
  }
}
__device__ __forceinline__ void store8_f32(float* q, int64_t left, bool whole, const float (&x)[VEC]) {
  if (whole) {
    *reinterpret_cast<f32x4*>(q) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4*>(q + 4) = f32x4{x[4], x[5], x[6], x[7]};
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) q[j] = x[j];
  }
}
__device__ __forceinline__ void store8_bf16(bf16_t* q, int64_t left, bool whole, const uint32_t (&w)[VEC / 2]) {
  if (whole) {
    *reinterpret_cast<i32x4*>(q) = i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j < left) q[j] = (bf16_t)(w[j / 2] >> (16 * (j & 1)));
  }
}

// bf16 bits of x: towards 0 after 16 random bits were added below; NaN stays, and what could
// round past the largest number does not
__device__ __forceinline__ uint32_t bf16_stochastic(float x, uint32_t r) {
  const uint32_t u = __float_as_uint(x);
  const bool top = (u & 0x7fffffffu) >= 0x7f7f0001u;
  if (top && x != x) return u >> 16 | 0x40u;
  return (top ? u : u + r) >> 16;
}

template <bool S8>
__global__ __launch_bounds__(AT) void k_adamw(AdamwTable tab, AdamwHyper h) {
  // the workgroup's tensor
  int lo = 0, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const moe_adamw_tensor& T = tab.t[lo];
  const int64_t n = T.n, i = (int64_t)(blockIdx.x - tab.first[lo]) * CHUNK + (int64_t)threadIdx.x * VEC;
  float rate = h.rate, unbias = h.root, decay = h.decay;
  uint32_t key = h.key;
  if (h.clock) {
    rate = h.rate * h.clock->to_m;   // h.rate: the rate itself
    unbias = h.clock->root;
    key = h.clock->key;
  }
  if (h.lr) {
    decay = 1.f - h.lr[0] * h.wd;
    rate = h.lr[0] * (h.clock ? h.clock->to_m : h.to_m);
  }
  const float gs = h.grad_scale ? h.grad_scale[0] : 1.f;
  const int64_t left = n - i;
  const bool full = left >= VEC;
  if ((i & ~(int64_t)31) >= n) return;   // a block of 32, four lanes, stays together
  const bool p16 = ((uintptr_t)T.p & 15) == 0, g16 = ((uintptr_t)T.g & 15) == 0;
  const void* pin = T.master ? (const void*)T.master : T.p;
  const int pdt = T.master ? MOE_F32 : T.p_dtype;
  const bool in16 = ((uintptr_t)pin & 15) == 0;
  float p[VEC], g[VEC], m[VEC], v[VEC];
  load8(T.g, T.g_dtype, i, n, full && g16, g);
  load8(pin, pdt, i, n, full && in16, p);
  if constexpr (S8) {
    if (left > 0) {   // the states' room ends with a block
      float s[VEC];
      decode(*reinterpret_cast<const uint2*>((const uint8_t*)T.m + i), (int)T.m_scale[i >> 5] - 127, m);
      decode(*reinterpret_cast<const uint2*>((const uint8_t*)T.v + i), (int)T.v_scale[i >> 5] - 127, s);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = s[j] * s[j];
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j >= left) m[j] = v[j] = 0.f;
  } else {
    load8(T.m, MOE_F32, i, n, full, m);
    load8(T.v, MOE_F32, i, n, full, v);
  }
  float s[VEC];
  float probe = 0.f;   // 8 bits: stays 0 where every root and every m is finite, which encode's FINITE form asks for
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const float gj = g[j] * gs;
    m[j] = blend(h.b1, m[j], h.b1c, gj);
    v[j] = blend(h.b2, v[j], h.b2c, gj * gj);
    s[j] = sqrtf(v[j]);   // rounded to nearest: with 8 bits its last bits decide a code (the hardware's is off by 1 ulp)
    p[j] = p[j] * decay - rate * m[j] * __builtin_amdgcn_rcpf(fmaf(s[j], unbias, h.eps));
    if constexpr (S8) probe = fmaf(s[j], 0.f, fmaf(m[j], 0.f, probe));
  }
  uint32_t r[VEC];
  if (h.stochastic) {
    // the upper half of the place changes once in the thread's 8 at most
    const uint64_t at = (uint64_t)T.at + (uint64_t)i;
    const uint32_t lo = (uint32_t)at, k0 = mix((uint32_t)(at >> 32) + key), k1 = mix((uint32_t)(at >> 32) + 1u + key);
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[j] = mix((lo + j) ^ (lo + j >= lo ? k0 : k1));
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) r[j] = 0;
  }
  if constexpr (S8) {
    uint2 cm, cv;
    int Xm, Xv;
    if (__ballot(probe != 0.f) == 0) {
      encode<false, true>(m, r, h.stochastic != 0, cm, Xm);
      encode<true, true>(s, r, h.stochastic != 0, cv, Xv);
    } else {
      encode<false, false>(m, r, h.stochastic != 0, cm, Xm);
      encode<true, false>(s, r, h.stochastic != 0, cv, Xv);
    }
    if (left > 0) {
      *reinterpret_cast<uint2*>((uint8_t*)T.m + i) = cm;
      *reinterpret_cast<uint2*>((uint8_t*)T.v + i) = cv;
      if ((i & 31) == 0) {
        T.m_scale[i >> 5] = (uint8_t)(Xm + 127);
        T.v_scale[i >> 5] = (uint8_t)(Xv + 127);
      }
    }
  } else {
    store8_f32((float*)T.m + i, left, full, m);
    store8_f32((float*)T.v + i, left, full, v);
  }
  if (T.master) store8_f32(T.master + i, left, full && in16, p);
  if (T.p_dtype == MOE_F32) {
    store8_f32((float*)T.p + i, left, full && p16, p);
  } else {
    uint32_t w[VEC / 2];
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      if (h.stochastic && !T.master)
        w[j] = bf16_stochastic(p[2 * j], mix(r[2 * j]) & 0xffffu) |
               bf16_stochastic(p[2 * j + 1], mix(r[2 * j + 1]) & 0xffffu) << 16;
      else
        w[j] = pk_bf16(p[2 * j], p[2 * j + 1]);
    }
    store8_bf16((bf16_t*)T.p + i, left, full && p16, w);
  }
}

// t + 1 and what follows from it
__global__ void k_adamw_clock(AdamwClock* c, double b1, double b2, uint64_t seed) {
  const int64_t t = c->t + 1;
  c->t = t;
  c->to_m = (float)(1.0 / (1.0 - pow(b1, (double)t)));
  c->root = (float)(1.0 / sqrt(1.0 - pow(b2, (double)t)));
  c->key = step_key(seed, t);
}

}  // namespace

hipError_t launch_adamw(const moe_adamw_params& s, const moe_adamw_tensor* tensors, int count, const float* lr,
                        const float* grad_scale, void* clock, hipStream_t st) {
  if (clock)
    MOE_LAUNCH("adamw_clock", k_adamw_clock, dim3(1), dim3(1), 0, st, (AdamwClock*)clock, s.beta1, s.beta2, s.seed);
  AdamwHyper h{};
  h.b1 = (float)s.beta1; h.b1c = (float)(1.0 - s.beta1);
  h.b2 = (float)s.beta2; h.b2c = (float)(1.0 - s.beta2);
  h.decay = (float)(1.0 - s.lr * s.weight_decay);
  h.eps = (float)s.eps; h.wd = (float)s.weight_decay;
  if (clock) {
    h.rate = (float)s.lr;
  } else {
    const double to_m = 1.0 / (1.0 - pow(s.beta1, (double)s.step));
    h.to_m = (float)to_m;
    h.rate = (float)(s.lr * to_m);
    h.root = (float)(1.0 / sqrt(1.0 - pow(s.beta2, (double)s.step)));
    h.key = step_key(s.seed, s.step);
  }
  h.stochastic = s.stochastic;
  h.lr = lr; h.grad_scale = grad_scale; h.clock = (const AdamwClock*)clock;
  const bool eight = s.state == MOE_STATE_8BIT;
  AdamwTable tab{};
  int64_t wgs = 0;
  auto go = [&]() -> hipError_t {
    if (tab.n == 0) return hipSuccess;
    if (eight)
      MOE_LAUNCH("adamw_8bit", k_adamw<true>, dim3((unsigned)wgs), dim3(AT), 0, st, tab, h);
    else
      MOE_LAUNCH("adamw", k_adamw<false>, dim3((unsigned)wgs), dim3(AT), 0, st, tab, h);
    tab.n = 0;
    wgs = 0;
    return hipGetLastError();
  };
  for (int i = 0; i < count; ++i) {
    moe_adamw_tensor t = tensors[i];   // what is left of it
    if (!t.g) continue;
    while (t.n > 0) {
      if (tab.n == kTensors || wgs == kMostGroups) {
        const hipError_t e = go();
        if (e != hipSuccess) return e;
      }
      const int64_t need = ceil_div(t.n, CHUNK), take = need < kMostGroups - wgs ? need : kMostGroups - wgs;
      const int64_t n = take < need ? take * CHUNK : t.n;
      tab.t[tab.n] = t;
      tab.t[tab.n].n = n;
      tab.first[tab.n] = (uint32_t)wgs;
      ++tab.n;
      wgs += take;
      t.n -= n;
      if (t.n == 0) break;
      // whole chunks are whole blocks of 32: the rest is a tensor of its own
      t.p = (char*)t.p + n * (t.p_dtype == MOE_BF16 ? 2 : 4);
      t.g = (const char*)t.g + n * (t.g_dtype == MOE_BF16 ? 2 : 4);
      if (t.master) t.master += n;
      t.m = (char*)t.m + n * (eight ? 1 : 4);
      t.v = (char*)t.v + n * (eight ? 1 : 4);
      if (eight) {
        t.m_scale += n / 32;
        t.v_scale += n / 32;
      }
      t.at += n;
    }
  }
  return go();
}

}  // namespace moe
