// Device-side pieces shared by the layer kernels: element access by dtype, activations and
// their derivatives, and warp sums.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "muon_b200.h"

namespace muon {

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_elem(void* p, int64_t i, int bf16, float v) {
  if (bf16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}

// Two fp32 values in one register pair: sm_100 adds, multiplies and fuses both in one
// instruction.
using F2 = unsigned long long;

__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 pair(float a) { return pair(a, a); }
__device__ __forceinline__ float2 split(F2 p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 2^x and 1 / x by the special function unit (a unit or two of the last place; 1 / inf = 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// z clamped to [-128, 128], a NaN kept: there every derivative is at its limit in fp32, so that
// infinity times zero does not come up.
__device__ __forceinline__ float clamp128(float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(-128.f));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(128.f));
  return r;
}

// 1 / (1 + 2^t) for both of t.
__device__ __forceinline__ F2 sigmoid2(F2 t) {
  const float2 v = split(t);
  const F2 d = add2(pair(fast_exp2(v.x), fast_exp2(v.y)), pair(1.f));
  const float2 w = split(d);
  return pair(fast_rcp(w.x), fast_rcp(w.y));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// The exponent of 2 in (1 + tanh u) / 2 = sigmoid(2 u) = 1 / (1 + 2^t), for
// 2 u = kTanhScale (z + 0.044715 z^3); this form keeps its relative accuracy where
// 1 + tanh u cancels.
__device__ __forceinline__ F2 tanh_exponent(F2 z, F2 zz) {
  return mul2(z, fma2(zz, pair(-kLog2e * kTanhScale * 0.044715f), pair(-kLog2e * kTanhScale)));
}

// Phi(-|z|) and exp(-z^2 / 2), for the exact GELU.  With x = |z| / sqrt 2 and t = 1 / (1 + 0.3 x),
// erfc(x) exp(x^2) / t is smooth on (0, 1]; the polynomial is its minimax fit (relative error)
// of degree 8 for x <= 10, found by iteratively reweighted least squares on Chebyshev points:
// with these constants 4.5e-8 in exact arithmetic, 4.4e-7 as evaluated in fp32.  The exponent of
// the bell is rounded to fp32 first, which weighs up to z^2 2^-24 relative: the tail is off by
// 4.6e-7 up to |z| = 2, 1.9e-6 up to 6, 5.2e-6 up to 10 and 7.5e-6 at 13, where it is 1e-38.
__device__ __forceinline__ F2 normal_tail2(F2 z, F2& bell) {
  const float2 e = split(mul2(mul2(z, z), pair(-0.5f * kLog2e)));
  bell = pair(fast_exp2(e.x), fast_exp2(e.y));
  const float2 v = split(z);
  const float2 d = split(fma2(pair(fabsf(v.x), fabsf(v.y)), pair(0.3f * 0.70710678118654752f), pair(1.f)));
  const F2 t = pair(fast_rcp(d.x), fast_rcp(d.y));
  F2 q = pair(-0.06476138532161713f);
  q = fma2(q, t, pair(0.24278128147125244f));
  q = fma2(q, t, pair(-0.2561383843421936f));
  q = fma2(q, t, pair(0.27385929226875305f));
  q = fma2(q, t, pair(-0.04732486978173256f));
  q = fma2(q, t, pair(0.1074628233909607f));
  q = fma2(q, t, pair(0.07416963577270508f));
  q = fma2(q, t, pair(0.08535760641098022f));
  q = fma2(q, t, pair(0.0845940038561821f));
  return mul2(mul2(q, t), bell);
}

// Phi(z) from Phi(-|z|).
__device__ __forceinline__ F2 normal_cdf2(F2 z, F2 tail) {
  const float2 v = split(z), w = split(tail);
  return pair(v.x < 0.f ? w.x : 1.f - w.x, v.y < 0.f ? w.y : 1.f - w.y);
}

__device__ __forceinline__ F2 relu2_of(F2 z) {  // max(z, 0); a NaN stays one
  const float2 v = split(z);
  return pair(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y);
}

// act(z) in fp32, two at a time: epilogues are paced by their instructions.
template <int ACT>
__device__ __forceinline__ F2 act_value2(F2 z) {
  if constexpr (ACT == MUON_ACT_RELU) {
    return relu2_of(z);
  } else if constexpr (ACT == MUON_ACT_RELU2) {
    const F2 r = relu2_of(z);
    return mul2(r, r);
  } else if constexpr (ACT == MUON_ACT_GELU) {
    F2 bell;
    const F2 tail = normal_tail2(z, bell);
    return mul2(z, normal_cdf2(z, tail));
  } else if constexpr (ACT == MUON_ACT_GELU_TANH) {
    return mul2(z, sigmoid2(tanh_exponent(z, mul2(z, z))));
  } else {
    static_assert(ACT == MUON_ACT_SILU, "an activation");
    return mul2(z, sigmoid2(mul2(z, pair(-kLog2e))));
  }
}

// act'(z) in fp32.
template <int ACT>
__device__ __forceinline__ F2 act_slope2(F2 z) {
  if constexpr (ACT == MUON_ACT_RELU) {
    const float2 v = split(z);
    return pair(v.x > 0.f ? 1.f : 0.f, v.y > 0.f ? 1.f : 0.f);
  } else if constexpr (ACT == MUON_ACT_RELU2) {
    return mul2(relu2_of(z), pair(2.f));
  } else {
    const float2 v = split(z);
    z = pair(clamp128(v.x), clamp128(v.y));
    if constexpr (ACT == MUON_ACT_GELU) {
      F2 bell;
      const F2 tail = normal_tail2(z, bell);
      return fma2(mul2(z, pair(0.39894228040143268f)), bell, normal_cdf2(z, tail));
    } else if constexpr (ACT == MUON_ACT_GELU_TANH) {
      // p + z p (1 - p) kTanhScale (1 + 3 0.044715 z^2)
      const F2 zz = mul2(z, z), p = sigmoid2(tanh_exponent(z, zz));
      const F2 g = mul2(z, fma2(zz, pair(kTanhScale * 0.134145f), pair(kTanhScale)));
      return mul2(p, fma2(g, fma2(p, pair(-1.f), pair(1.f)), pair(1.f)));
    } else {
      static_assert(ACT == MUON_ACT_SILU, "an activation");
      const F2 p = sigmoid2(mul2(z, pair(-kLog2e)));
      return mul2(p, fma2(z, fma2(p, pair(-1.f), pair(1.f)), pair(1.f)));
    }
  }
}

// v = act(v) and v *= act'(t), the choice made once for N pairs.
template <int N>
__device__ __forceinline__ void apply_act(int act, F2 (&v)[N]) {
#define MUON_EACH(A)                                                        \
  case A:                                                                   \
    _Pragma("unroll") for (int j = 0; j < N; ++j) v[j] = act_value2<A>(v[j]); \
    break
  switch (act) {
    MUON_EACH(MUON_ACT_RELU);
    MUON_EACH(MUON_ACT_RELU2);
    MUON_EACH(MUON_ACT_GELU);
    MUON_EACH(MUON_ACT_GELU_TANH);
    MUON_EACH(MUON_ACT_SILU);
    default: break;
  }
#undef MUON_EACH
}

template <int N>
__device__ __forceinline__ void apply_slope(int act, const F2 (&t)[N], F2 (&v)[N]) {
#define MUON_EACH(A)                                                                        \
  case A:                                                                                   \
    _Pragma("unroll") for (int j = 0; j < N; ++j) v[j] = mul2(v[j], act_slope2<A>(t[j])); \
    break
  switch (act) {
    MUON_EACH(MUON_ACT_RELU);
    MUON_EACH(MUON_ACT_RELU2);
    MUON_EACH(MUON_ACT_GELU);
    MUON_EACH(MUON_ACT_GELU_TANH);
    MUON_EACH(MUON_ACT_SILU);
    default: break;
  }
#undef MUON_EACH
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace muon
