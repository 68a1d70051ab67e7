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
    case MUON_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
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
    case MUON_ACT_GELU:
      return fmaf(c, 0.39894228040143268f * __expf(-0.5f * c * c), 0.5f * erfcf(-0.70710678118654752f * z));
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace muon
