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

__device__ __forceinline__ float sigmoid(float t) { return __fdividef(1.f, 1.f + __expf(-t)); }

// Phi(-|z|) and exp(-z^2 / 2), for the exact GELU.  With x = |z| / sqrt 2 and t = 1 / (1 + 0.3 x),
// erfc(x) exp(x^2) / t is smooth on (0, 1]; the polynomial is its minimax fit (relative error)
// of degree 8 for x <= 10, found by iteratively reweighted least squares on Chebyshev points:
// 2e-8 in exact arithmetic, 5e-7 as evaluated in fp32, in the far tail too.
__device__ __forceinline__ float normal_tail(float z, float& bell) {
  bell = __expf(-0.5f * z * z);
  const float t = __fdividef(1.f, fmaf(0.3f * 0.70710678118654752f, fabsf(z), 1.f));
  float q = -0.06476138532161713f;
  q = fmaf(q, t, 0.24278128147125244f);
  q = fmaf(q, t, -0.2561383843421936f);
  q = fmaf(q, t, 0.27385929226875305f);
  q = fmaf(q, t, -0.04732486978173256f);
  q = fmaf(q, t, 0.1074628233909607f);
  q = fmaf(q, t, 0.07416963577270508f);
  q = fmaf(q, t, 0.08535760641098022f);
  q = fmaf(q, t, 0.0845940038561821f);
  return q * t * bell;
}

// act(z) in fp32.  The tanh form is z sigmoid(2 u): (1 + tanh u) / 2 = sigmoid(2 u), which
// keeps its relative accuracy where 1 + tanh u cancels.  Comparisons are written so that a
// NaN comes out as a NaN.
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case MUON_ACT_RELU: return z < 0.f ? 0.f : z;
    case MUON_ACT_RELU2: {
      const float r = z < 0.f ? 0.f : z;
      return r * r;
    }
    case MUON_ACT_GELU: {
      float bell;
      const float tail = normal_tail(z, bell);
      return z * (z < 0.f ? tail : 1.f - tail);
    }
    case MUON_ACT_GELU_TANH: return z * sigmoid(1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.f));
    case MUON_ACT_SILU: return z * sigmoid(z);
    default: return z;
  }
}

// act'(z) in fp32.  The second terms vanish long before |z| = 64; clamping z there keeps
// infinity times zero out of them.
__device__ __forceinline__ float act_slope(int act, float z) {
  const float c = fminf(fmaxf(z, -64.f), 64.f);
  switch (act) {
    case MUON_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case MUON_ACT_RELU2: return z < 0.f ? 0.f : 2.f * z;
    case MUON_ACT_GELU: {
      float bell;
      const float tail = normal_tail(z, bell);
      return fmaf(c * 0.39894228040143268f, bell, z < 0.f ? tail : 1.f - tail);
    }
    case MUON_ACT_GELU_TANH: {
      const float p = sigmoid(1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.f));
      return fmaf(c * p * (1.f - p), 1.5957691216057308f * fmaf(0.134145f * c, c, 1.f), p);
    }
    case MUON_ACT_SILU: {
      const float p = sigmoid(z);
      return p * fmaf(c, 1.f - p, 1.f);
    }
    default: return 1.f;
  }
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace muon
