// Layer norm and its gradients.
//
//   y = (x - mean) rstd gain + bias,  mean = sum(x) / D,  rstd = 1 / sqrt(sum((x - mean)^2) / D + eps)
//   h = (x - mean) rstd,  q = dy gain
//   dx = rstd (q - avg(q) - h avg(q h)) + skip,  dgain = sum_rows dy h,  dbias = sum_rows dy
//
// The variance is summed from the centred values, never as E[x^2] - mean^2, which cancels
// where the mean is large.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "muon_layers.cuh"
#include "muon_layers_host.h"

namespace muon {

struct NormParams {
  const void* x;
  const void* gain;
  const void* bias;
  void* y;
  float* mean;
  float* rstd;
  int64_t rows, ld_x, ld_y;
  int32_t cols, x_bf16, gain_bf16, bias_bf16;
  float eps;
};

struct NormGradParams {
  const void* dy;
  const void* x;
  const void* gain;
  const void* skip;
  void* dx;
  const float* mean;
  const float* rstd;
  float* dgain;
  float* dbias;
  float* partial;  // [slices][2][cols]
  int64_t rows, ld_dy, ld_x, ld_skip, ld_dx;
  int32_t cols, x_bf16, gain_bf16, skip_bf16;
  int32_t accumulate, slices;
};

constexpr int kNormThreads = 256;

// Sum over the block; every thread gets it.  `red` holds 33 floats.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    const float w = warp_sum(threadIdx.x < blockDim.x / 32 ? red[threadIdx.x] : 0.f);
    if (threadIdx.x == 0) red[32] = w;
  }
  __syncthreads();
  return red[32];
}

// One row per block, the row read three times (from L2 after the first).
__global__ void __launch_bounds__(kNormThreads) layer_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[33];
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const int64_t xo = r * p.ld_x, yo = r * p.ld_y;
    float s = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += kNormThreads) s += load_elem(p.x, xo + c, p.x_bf16);
    const float mean = block_sum(s, red) / static_cast<float>(p.cols);
    s = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += kNormThreads) {
      const float d = load_elem(p.x, xo + c, p.x_bf16) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = 1.f / sqrtf(block_sum(s, red) / static_cast<float>(p.cols) + p.eps);
    for (int c = threadIdx.x; c < p.cols; c += kNormThreads) {
      float v = (load_elem(p.x, xo + c, p.x_bf16) - mean) * rstd;
      if (p.gain != nullptr) v *= load_elem(p.gain, c, p.gain_bf16);
      if (p.bias != nullptr) v += load_elem(p.bias, c, p.bias_bf16);
      store_elem(p.y, yo + c, p.x_bf16, v);
    }
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[r] = mean;
      if (p.rstd != nullptr) p.rstd[r] = rstd;
    }
  }
}

__global__ void __launch_bounds__(kNormThreads) layer_norm_dx_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ float red[33];
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const float mean = p.mean[r], rstd = p.rstd[r];
    float sq = 0.f, sqh = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += kNormThreads) {
      float q = load_elem(p.dy, r * p.ld_dy + c, p.x_bf16);
      if (p.gain != nullptr) q *= load_elem(p.gain, c, p.gain_bf16);
      sq += q;
      sqh = fmaf(q, (load_elem(p.x, r * p.ld_x + c, p.x_bf16) - mean) * rstd, sqh);
    }
    const float aq = block_sum(sq, red) / static_cast<float>(p.cols);
    const float aqh = block_sum(sqh, red) / static_cast<float>(p.cols);
    for (int c = threadIdx.x; c < p.cols; c += kNormThreads) {
      float q = load_elem(p.dy, r * p.ld_dy + c, p.x_bf16);
      if (p.gain != nullptr) q *= load_elem(p.gain, c, p.gain_bf16);
      const float h = (load_elem(p.x, r * p.ld_x + c, p.x_bf16) - mean) * rstd;
      float v = rstd * (q - aq - h * aqh);
      if (p.skip != nullptr) v += load_elem(p.skip, r * p.ld_skip + c, p.skip_bf16);
      store_elem(p.dx, r * p.ld_dx + c, p.x_bf16, v);
    }
  }
}

// Partial column sums: block (b, s) takes 32 columns and every slices-th group of 8 rows.
__global__ void __launch_bounds__(256) layer_norm_columns_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ float sg[8][33], sb[8][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float dg = 0.f, db = 0.f;
  if (c < p.cols)
    for (int64_t r = blockIdx.y * 8 + w; r < p.rows; r += int64_t(8) * gridDim.y) {
      const float dy = load_elem(p.dy, r * p.ld_dy + c, p.x_bf16);
      const float h = (load_elem(p.x, r * p.ld_x + c, p.x_bf16) - p.mean[r]) * p.rstd[r];
      dg = fmaf(dy, h, dg);
      db += dy;
    }
  sg[w][lane] = dg;
  sb[w][lane] = db;
  __syncthreads();
  if (w == 0 && c < p.cols) {
    for (int k = 1; k < 8; ++k) {
      dg += sg[k][lane];
      db += sb[k][lane];
    }
    float* o = p.partial + static_cast<int64_t>(blockIdx.y) * 2 * p.cols;
    o[c] = dg;
    o[p.cols + c] = db;
  }
}

__global__ void __launch_bounds__(256) layer_norm_finish_kernel(const __grid_constant__ NormGradParams p) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float dg = 0.f, db = 0.f;
  for (int s = 0; s < p.slices; ++s) {
    dg += p.partial[static_cast<int64_t>(s) * 2 * p.cols + c];
    db += p.partial[static_cast<int64_t>(s) * 2 * p.cols + p.cols + c];
  }
  if (p.dgain != nullptr) p.dgain[c] = p.accumulate ? p.dgain[c] + dg : dg;
  if (p.dbias != nullptr) p.dbias[c] = p.accumulate ? p.dbias[c] + db : db;
}

}  // namespace muon

namespace {
using namespace muon;

bool sizes_ok(int64_t rows, int64_t cols) { return rows >= 0 && rows <= kMaxRows && cols >= 1 && cols <= kMaxSide; }

int slices_for(const muon_layer_norm_grad_t* d) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, ceil_div(d->rows, 64))));
}

size_t norm_grad_bytes(const muon_layer_norm_grad_t* d) {
  if (d->dgain == nullptr && d->dbias == nullptr) return 0;
  return static_cast<size_t>(slices_for(d)) * 2 * static_cast<size_t>(d->cols) * sizeof(float);
}

}  // namespace

extern "C" muon_status_t muon_layer_norm(const muon_layer_norm_t* d, void* stream) {
  if (d == nullptr || !std::isfinite(d->eps) || d->eps < 0.f) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->cols)) return MUON_ERR_UNSUPPORTED_SHAPE;
  Operands ops;
  ops.add(d->x, d->rows, d->cols, true, false);
  ops.add(d->gain, 1, d->cols, false, false);
  ops.add(d->bias, 1, d->cols, false, false);
  ops.add(d->y, d->rows, d->cols, true, true);
  ops.add_f32(d->mean, d->rows, false, true);
  ops.add_f32(d->rstd, d->rows, false, true);
  if (d->rows > 0 && d->x.dtype != d->y.dtype) ops.fail(MUON_ERR_UNSUPPORTED_DTYPE);
  muon_status_t st = ops.check();
  if (st != MUON_OK) return st;
  int sms = 0;
  if ((st = layers_device(&sms)) != MUON_OK) return st;
  if (d->rows == 0) return MUON_OK;
  NormParams p{};
  p.x = d->x.data;
  p.gain = d->gain.data;
  p.bias = d->bias.data;
  p.y = d->y.data;
  p.mean = d->mean;
  p.rstd = d->rstd;
  p.rows = d->rows;
  p.ld_x = row_stride(d->x, d->rows, d->cols);
  p.ld_y = row_stride(d->y, d->rows, d->cols);
  p.cols = static_cast<int32_t>(d->cols);
  p.x_bf16 = d->x.dtype == MUON_BF16;
  p.gain_bf16 = d->gain.dtype == MUON_BF16;
  p.bias_bf16 = d->bias.dtype == MUON_BF16;
  p.eps = d->eps;
  layer_norm_kernel<<<static_cast<unsigned>(std::min<int64_t>(d->rows, 1 << 20)), kNormThreads, 0,
                      static_cast<cudaStream_t>(stream)>>>(p);
  return launched();
}

extern "C" muon_status_t muon_layer_norm_backward_workspace(const muon_layer_norm_grad_t* d, size_t* bytes) {
  if (d == nullptr || bytes == nullptr) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->cols)) return MUON_ERR_UNSUPPORTED_SHAPE;
  *bytes = norm_grad_bytes(d);
  return MUON_OK;
}

extern "C" muon_status_t muon_layer_norm_backward(const muon_layer_norm_grad_t* d, void* workspace,
                                                  size_t workspace_bytes, void* stream) {
  if (d == nullptr || (d->accumulate != 0 && d->accumulate != 1)) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->cols)) return MUON_ERR_UNSUPPORTED_SHAPE;
  const bool grads = d->dgain != nullptr || d->dbias != nullptr;
  const bool alias = d->dx.data != nullptr && same_view(d->dx, d->skip, d->rows);
  Operands ops;
  ops.add(d->dy, d->rows, d->cols, true, false);
  ops.add(d->x, d->rows, d->cols, true, false);
  ops.add(d->gain, 1, d->cols, false, false);
  if (!alias) ops.add(d->skip, d->rows, d->cols, false, false);
  ops.add(d->dx, d->rows, d->cols, false, true);
  ops.add_f32(d->mean, d->rows, true, false);
  ops.add_f32(d->rstd, d->rows, true, false);
  ops.add_f32(d->dgain, d->cols, false, true);
  ops.add_f32(d->dbias, d->cols, false, true);
  if (d->dx.data == nullptr && !grads) ops.fail(MUON_ERR_INVALID_ARG);
  if (d->rows > 0 && (d->x.dtype != d->dy.dtype || (d->dx.data != nullptr && d->dx.dtype != d->x.dtype)))
    ops.fail(MUON_ERR_UNSUPPORTED_DTYPE);
  const size_t need = norm_grad_bytes(d);
  if (ops.status == MUON_OK && need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned_bytes(workspace, 256)) return MUON_ERR_ALIGNMENT;
    ops.add_bytes(workspace, need);
  }
  muon_status_t st = ops.check();
  if (st != MUON_OK) return st;
  int sms = 0;
  if ((st = layers_device(&sms)) != MUON_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NormGradParams p{};
  p.dy = d->dy.data;
  p.x = d->x.data;
  p.gain = d->gain.data;
  p.skip = d->skip.data;
  p.dx = d->dx.data;
  p.mean = d->mean;
  p.rstd = d->rstd;
  p.dgain = d->dgain;
  p.dbias = d->dbias;
  p.partial = static_cast<float*>(workspace);
  p.rows = d->rows;
  p.ld_dy = row_stride(d->dy, d->rows, d->cols);
  p.ld_x = row_stride(d->x, d->rows, d->cols);
  p.ld_skip = row_stride(d->skip, d->rows, d->cols);
  p.ld_dx = row_stride(d->dx, d->rows, d->cols);
  p.cols = static_cast<int32_t>(d->cols);
  p.x_bf16 = d->x.dtype == MUON_BF16;
  p.gain_bf16 = d->gain.dtype == MUON_BF16;
  p.skip_bf16 = d->skip.dtype == MUON_BF16;
  p.accumulate = d->accumulate;
  p.slices = slices_for(d);
  if (d->dx.data != nullptr && d->rows > 0) {
    layer_norm_dx_kernel<<<static_cast<unsigned>(std::min<int64_t>(d->rows, 1 << 20)), kNormThreads, 0, s>>>(p);
    if ((st = launched()) != MUON_OK) return st;
  }
  if (grads) {
    const dim3 g(static_cast<unsigned>(ceil_div(d->cols, 32)), static_cast<unsigned>(p.slices));
    layer_norm_columns_kernel<<<g, 256, 0, s>>>(p);
    if ((st = launched()) != MUON_OK) return st;
    layer_norm_finish_kernel<<<static_cast<unsigned>(ceil_div(d->cols, 256)), 256, 0, s>>>(p);
    return launched();
  }
  return MUON_OK;
}
