// Linear layers and their gradients: the C ABI entry points, and the elementwise kernels.
//
//   muon_linear            z = x W^T + bias,  y = act(z) + residual
//   muon_linear_backward   dx = (dy W) act'(z_in) + skip,  dW (+)= dy^T x,  db (+)= sum of dy
//   muon_activation_backward  dz = dy act'(z)
//
// All three products are D[M x N] = sum_k A(m, k) B(n, k) with operands that are contiguous
// along k or along their own side, and one epilogue:
//   v = sum + bias[n];  preact[m, n] = v;  v = act(v);  v *= act'(slope[m, n]);  v += add[m, n]
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "muon_layers.cuh"
#include "muon_layers_host.h"

namespace muon {

struct ProductParams {
  const void* a;
  const void* b;
  int64_t a_side, a_k, b_side, b_k;  // element strides
  int64_t m, n, k;
  int32_t a_bf16, b_bf16;
  const void* bias;
  void* preact;
  const void* slope;
  const void* add;
  void* out;
  int64_t ld_preact, ld_slope, ld_add, ld_out;
  int32_t bias_bf16, preact_bf16, slope_bf16, add_bf16, out_bf16;
  int32_t act, slope_act;
};

__global__ void __launch_bounds__(256) product_kernel(const __grid_constant__ ProductParams p) {
  __shared__ float sa[16][65], sb[16][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 64, n0 = static_cast<int64_t>(blockIdx.x) * 64;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.k; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int ka = p.a_k == 1 ? (i & 15) : (i >> 6), ma = p.a_k == 1 ? (i >> 4) : (i & 63);
      sa[ka][ma] = (m0 + ma < p.m && k0 + ka < p.k)
                       ? load_elem(p.a, (m0 + ma) * p.a_side + (k0 + ka) * p.a_k, p.a_bf16) : 0.f;
      const int kb = p.b_k == 1 ? (i & 15) : (i >> 6), nb = p.b_k == 1 ? (i >> 4) : (i & 63);
      sb[kb][nb] = (n0 + nb < p.n && k0 + kb < p.k)
                       ? load_elem(p.b, (n0 + nb) * p.b_side + (k0 + kb) * p.b_k, p.b_bf16) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[kk][ty + 16 * i], sb[kk][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= p.m || n >= p.n) continue;
      float v = acc[i][j];
      if (p.bias != nullptr) v += load_elem(p.bias, n, p.bias_bf16);
      if (p.preact != nullptr) store_elem(p.preact, m * p.ld_preact + n, p.preact_bf16, v);
      v = act_value(p.act, v);
      if (p.slope != nullptr) v *= act_slope(p.slope_act, load_elem(p.slope, m * p.ld_slope + n, p.slope_bf16));
      if (p.add != nullptr) v += load_elem(p.add, m * p.ld_add + n, p.add_bf16);
      store_elem(p.out, m * p.ld_out + n, p.out_bf16, v);
    }
}

struct ColumnSumParams {
  const void* dy;
  float* db;
  int64_t rows, ld;
  int32_t cols, bf16, accumulate;
};

// One warp-wide column group per block, all rows.
__global__ void __launch_bounds__(256) column_sum_kernel(const __grid_constant__ ColumnSumParams p) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < p.cols)
    for (int64_t r = w; r < p.rows; r += 8) s += load_elem(p.dy, r * p.ld + c, p.bf16);
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < p.cols) {
    for (int k = 1; k < 8; ++k) s += red[k][lane];
    p.db[c] = p.accumulate ? p.db[c] + s : s;
  }
}

struct ActGradParams {
  const void* dy;
  const void* z;
  void* dz;
  int64_t rows, cols, ld_dy, ld_z, ld_dz;
  int32_t dy_bf16, z_bf16, act;
};

__global__ void __launch_bounds__(256) activation_backward_kernel(const __grid_constant__ ActGradParams p) {
  const int64_t per_row = (p.cols + 255) / 256;
  for (int64_t b = blockIdx.x; b < p.rows * per_row; b += gridDim.x) {
    const int64_t r = b / per_row, c = (b - r * per_row) * 256 + threadIdx.x;
    if (c >= p.cols) continue;
    const float g = load_elem(p.dy, r * p.ld_dy + c, p.dy_bf16);
    store_elem(p.dz, r * p.ld_dz + c, p.dy_bf16, g * act_slope(p.act, load_elem(p.z, r * p.ld_z + c, p.z_bf16)));
  }
}

__device__ int32_t g_layers_status[2];  // code, wait site

}  // namespace muon

namespace {
using namespace muon;

bool sizes_ok(int64_t rows, int64_t in, int64_t out) {
  return rows >= 0 && rows <= kMaxRows && in >= 1 && in <= kMaxSide && out >= 1 && out <= kMaxSide;
}

bool act_ok(int act) { return act >= MUON_ACT_NONE && act <= MUON_ACT_SILU; }

muon_status_t run_product(const ProductParams& p, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>(ceil_div(p.n, 64)), static_cast<unsigned>(ceil_div(p.m, 64)));
  product_kernel<<<g, 256, 0, s>>>(p);
  return launched();
}

}  // namespace

extern "C" {

muon_status_t muon_linear_workspace(const muon_linear_t* d, size_t* bytes) {
  if (d == nullptr || bytes == nullptr) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->in, d->out)) return MUON_ERR_UNSUPPORTED_SHAPE;
  *bytes = 0;
  return MUON_OK;
}

muon_status_t muon_linear(const muon_linear_t* d, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  if (d == nullptr || !act_ok(d->act)) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->in, d->out)) return MUON_ERR_UNSUPPORTED_SHAPE;
  Operands ops;
  ops.add(d->x, d->rows, d->in, true, false);
  ops.add(d->w, d->out, d->in, true, false);
  ops.add(d->bias, 1, d->out, false, false);
  if (!same_view(d->y, d->residual, d->rows)) ops.add(d->residual, d->rows, d->out, false, false);
  ops.add(d->y, d->rows, d->out, true, true);
  ops.add(d->preact, d->rows, d->out, false, true);
  muon_status_t st = ops.check();
  if (st != MUON_OK) return st;
  int sms = 0;
  if ((st = layers_device(&sms)) != MUON_OK) return st;
  if (d->rows == 0) return MUON_OK;
  ProductParams p{};
  p.a = d->x.data;
  p.a_side = row_stride(d->x, d->rows, d->in);
  p.a_k = 1;
  p.a_bf16 = d->x.dtype == MUON_BF16;
  p.b = d->w.data;
  p.b_side = row_stride(d->w, d->out, d->in);
  p.b_k = 1;
  p.b_bf16 = d->w.dtype == MUON_BF16;
  p.m = d->rows;
  p.n = d->out;
  p.k = d->in;
  p.bias = d->bias.data;
  p.bias_bf16 = d->bias.dtype == MUON_BF16;
  p.preact = d->preact.data;
  p.ld_preact = row_stride(d->preact, d->rows, d->out);
  p.preact_bf16 = d->preact.dtype == MUON_BF16;
  p.act = d->act;
  p.add = d->residual.data;
  p.ld_add = row_stride(d->residual, d->rows, d->out);
  p.add_bf16 = d->residual.dtype == MUON_BF16;
  p.out = d->y.data;
  p.ld_out = row_stride(d->y, d->rows, d->out);
  p.out_bf16 = d->y.dtype == MUON_BF16;
  return run_product(p, static_cast<cudaStream_t>(stream));
}

muon_status_t muon_linear_backward_workspace(const muon_linear_grad_t* d, size_t* bytes) {
  if (d == nullptr || bytes == nullptr) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->in, d->out)) return MUON_ERR_UNSUPPORTED_SHAPE;
  *bytes = 0;
  return MUON_OK;
}

muon_status_t muon_linear_backward(const muon_linear_grad_t* d, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  if (d == nullptr || !act_ok(d->in_act) || (d->accumulate != 0 && d->accumulate != 1)) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->in, d->out)) return MUON_ERR_UNSUPPORTED_SHAPE;
  const bool dx = d->dx.data != nullptr, dw = d->dw.data != nullptr, slope = dx && d->in_act != MUON_ACT_NONE;
  Operands ops;
  ops.add(d->dy, d->rows, d->out, true, false);
  ops.add(d->x, d->rows, d->in, dw, false);
  ops.add(d->w, d->out, d->in, dx, false);
  ops.add(d->preact, d->rows, d->in, slope, false);
  if (!(dx && same_view(d->dx, d->skip, d->rows))) ops.add(d->skip, d->rows, d->in, false, false);
  ops.add(d->dx, d->rows, d->in, false, true);
  ops.add(d->dw, d->out, d->in, false, true);
  ops.add_f32(d->db, d->out, false, true);
  if (dw && d->dw.dtype != MUON_F32) ops.fail(MUON_ERR_UNSUPPORTED_DTYPE);
  if (!dx && !dw && d->db == nullptr && d->rows > 0) ops.fail(MUON_ERR_INVALID_ARG);
  muon_status_t st = ops.check();
  if (st != MUON_OK) return st;
  int sms = 0;
  if ((st = layers_device(&sms)) != MUON_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dx && d->rows > 0) {
    ProductParams p{};
    p.a = d->dy.data;
    p.a_side = row_stride(d->dy, d->rows, d->out);
    p.a_k = 1;
    p.a_bf16 = d->dy.dtype == MUON_BF16;
    p.b = d->w.data;
    p.b_side = 1;
    p.b_k = row_stride(d->w, d->out, d->in);
    p.b_bf16 = d->w.dtype == MUON_BF16;
    p.m = d->rows;
    p.n = d->in;
    p.k = d->out;
    p.slope = slope ? d->preact.data : nullptr;
    p.ld_slope = row_stride(d->preact, d->rows, d->in);
    p.slope_bf16 = d->preact.dtype == MUON_BF16;
    p.slope_act = d->in_act;
    p.add = d->skip.data;
    p.ld_add = row_stride(d->skip, d->rows, d->in);
    p.add_bf16 = d->skip.dtype == MUON_BF16;
    p.out = d->dx.data;
    p.ld_out = row_stride(d->dx, d->rows, d->in);
    p.out_bf16 = d->dx.dtype == MUON_BF16;
    if ((st = run_product(p, s)) != MUON_OK) return st;
  }
  if (dw && !(d->rows == 0 && d->accumulate)) {
    ProductParams p{};
    p.a = d->dy.data;
    p.a_side = 1;
    p.a_k = row_stride(d->dy, d->rows, d->out);
    p.a_bf16 = d->dy.dtype == MUON_BF16;
    p.b = d->x.data;
    p.b_side = 1;
    p.b_k = row_stride(d->x, d->rows, d->in);
    p.b_bf16 = d->x.dtype == MUON_BF16;
    p.m = d->out;
    p.n = d->in;
    p.k = d->rows;
    p.out = d->dw.data;
    p.ld_out = row_stride(d->dw, d->out, d->in);
    p.add = d->accumulate ? d->dw.data : nullptr;
    p.ld_add = p.ld_out;
    if ((st = run_product(p, s)) != MUON_OK) return st;
  }
  if (d->db != nullptr && !(d->rows == 0 && d->accumulate)) {
    ColumnSumParams c{};
    c.dy = d->dy.data;
    c.db = d->db;
    c.rows = d->rows;
    c.ld = row_stride(d->dy, d->rows, d->out);
    c.cols = static_cast<int32_t>(d->out);
    c.bf16 = d->dy.dtype == MUON_BF16;
    c.accumulate = d->accumulate;
    column_sum_kernel<<<static_cast<unsigned>(ceil_div(d->out, 32)), 256, 0, s>>>(c);
    return launched();
  }
  return MUON_OK;
}

muon_status_t muon_activation_backward(const muon_activation_grad_t* d, void* stream) {
  if (d == nullptr || !act_ok(d->act) || d->act == MUON_ACT_NONE) return MUON_ERR_INVALID_ARG;
  if (!sizes_ok(d->rows, d->cols, 1)) return MUON_ERR_UNSUPPORTED_SHAPE;
  Operands ops;
  ops.add(d->dy, d->rows, d->cols, true, false);
  ops.add(d->z, d->rows, d->cols, true, false);
  ops.add(d->dz, d->rows, d->cols, true, true);
  if (d->rows > 0 && d->dz.dtype != d->dy.dtype) ops.fail(MUON_ERR_UNSUPPORTED_DTYPE);
  muon_status_t st = ops.check();
  if (st != MUON_OK) return st;
  int sms = 0;
  if ((st = layers_device(&sms)) != MUON_OK) return st;
  if (d->rows == 0) return MUON_OK;
  ActGradParams p{};
  p.dy = d->dy.data;
  p.z = d->z.data;
  p.dz = d->dz.data;
  p.rows = d->rows;
  p.cols = d->cols;
  p.ld_dy = row_stride(d->dy, d->rows, d->cols);
  p.ld_z = row_stride(d->z, d->rows, d->cols);
  p.ld_dz = row_stride(d->dz, d->rows, d->cols);
  p.dy_bf16 = d->dy.dtype == MUON_BF16;
  p.z_bf16 = d->z.dtype == MUON_BF16;
  p.act = d->act;
  const int64_t blocks = std::min<int64_t>(d->rows * ceil_div(d->cols, 256), sms * 64);
  activation_backward_kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return launched();
}

muon_status_t muon_layers_status(void* stream, int clear, int32_t* device_status, int32_t* where) {
  if (device_status == nullptr) return MUON_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t h[2] = {0, 0};
  const int32_t zero[2] = {0, 0};
  if (cudaMemcpyFromSymbolAsync(h, g_layers_status, sizeof(h), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MUON_ERR_CUDA;
  if (clear && (cudaMemcpyToSymbolAsync(g_layers_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) !=
                    cudaSuccess ||
                cudaStreamSynchronize(s) != cudaSuccess))
    return MUON_ERR_CUDA;
  *device_status = h[0];
  if (where != nullptr) *where = h[1];
  return MUON_OK;
}

}  // extern "C"
