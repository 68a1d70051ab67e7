// The epilogue of the layer products: loads and stores of row segments, and the arithmetic.
#pragma once

#include "muon_device.cuh"
#include "muon_layers.cuh"
#include "muon_product.h"

namespace muon {

// NC (a multiple of 8) consecutive elements of a row, the first `valid` of them; the rest
// are left at zero.  `off` is the element offset of the segment.
template <int NC>
__device__ __forceinline__ void load_segment(const EpiView& v, int64_t off, int valid, float (&x)[NC]) {
  if (valid >= NC && v.vec) {
    if (v.bf16) {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(v.p) + off;
      uint4 w[NC / 8];
      if (NC % 16 == 0 && v.vec == 2) {
#pragma unroll
        for (int i = 0; i < NC / 16; ++i) ld_global_v8(p + 16 * i, w[2 * i], w[(2 * i + 1) % (NC / 8)]);
      } else {
#pragma unroll
        for (int i = 0; i < NC / 8; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
      }
#pragma unroll
      for (int i = 0; i < NC / 8; ++i) {
        const uint32_t q[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[8 * i + 2 * j] = __uint_as_float(q[j] << 16);
          x[8 * i + 2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
        }
      }
    } else {
      const float* p = static_cast<const float*>(v.p) + off;
      uint4 w[NC / 4];
      if (v.vec == 2) {
#pragma unroll
        for (int i = 0; i < NC / 8; ++i) ld_global_v8(p + 8 * i, w[2 * i], w[2 * i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < NC / 4; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
      }
#pragma unroll
      for (int i = 0; i < NC / 4; ++i) {
        x[4 * i] = __uint_as_float(w[i].x);
        x[4 * i + 1] = __uint_as_float(w[i].y);
        x[4 * i + 2] = __uint_as_float(w[i].z);
        x[4 * i + 3] = __uint_as_float(w[i].w);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j) x[j] = j < valid ? load_elem(v.p, off + j, v.bf16) : 0.f;
  }
}

template <int NC>
__device__ __forceinline__ void store_segment(const EpiView& v, int64_t off, int valid, const float (&x)[NC]) {
  if (valid >= NC && v.vec) {
    if (v.bf16) {
      __nv_bfloat16* p = static_cast<__nv_bfloat16*>(v.p) + off;
      uint4 w[NC / 8];
#pragma unroll
      for (int i = 0; i < NC / 8; ++i) {
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
          q[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        w[i] = make_uint4(q[0], q[1], q[2], q[3]);
      }
      if (NC % 16 == 0 && v.vec == 2) {
#pragma unroll
        for (int i = 0; i < NC / 16; ++i) st_global_v8(p + 16 * i, w[2 * i], w[(2 * i + 1) % (NC / 8)]);
      } else {
#pragma unroll
        for (int i = 0; i < NC / 8; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
      }
    } else {
      float* p = static_cast<float*>(v.p) + off;
      uint4 w[NC / 4];
#pragma unroll
      for (int i = 0; i < NC / 4; ++i)
        w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                          __float_as_uint(x[4 * i + 3]));
      if (v.vec == 2) {
#pragma unroll
        for (int i = 0; i < NC / 8; ++i) st_global_v8(p + 8 * i, w[2 * i], w[2 * i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < NC / 4; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (j < valid) store_elem(v.p, off + j, v.bf16, x[j]);
  }
}

// v = act(v) and v *= act'(t), the choice made once for the segment.
template <int NC>
__device__ __forceinline__ void apply_act(int act, float (&v)[NC]) {
#define MUON_EACH(A)                                        \
  case A:                                                   \
    _Pragma("unroll") for (int j = 0; j < NC; ++j) v[j] = act_value(A, v[j]); \
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

template <int NC>
__device__ __forceinline__ void apply_slope(int act, const float (&t)[NC], float (&v)[NC]) {
#define MUON_EACH(A)                                        \
  case A:                                                   \
    _Pragma("unroll") for (int j = 0; j < NC; ++j) v[j] *= act_slope(A, t[j]); \
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

// ------------------------------------------------------------------ the common epilogue
//
// When everything but the bias is bf16 in rows of whole 32-byte units, 32 columns of a row
// are 64 bytes of each operand.  With two epilogue warps per scheduler, the epilogue's pace
// is its number of instructions times their latency, so this path has no choices inside:
// addresses are carried per row, and the inputs are fetched a step ahead (16 words each).
struct EpiRow {
  const uint8_t* slope;
  const uint8_t* add;
  uint8_t* preact;
  uint8_t* out;
  uint32_t slope_w[16], add_w[16];

  __device__ __forceinline__ void start(const Epilogue& e, int64_t m, int64_t n) {
    slope = e.slope.p == nullptr ? nullptr : static_cast<const uint8_t*>(e.slope.p) + 2 * (m * e.slope.ld + n);
    add = e.add.p == nullptr ? nullptr : static_cast<const uint8_t*>(e.add.p) + 2 * (m * e.add.ld + n);
    preact = e.preact.p == nullptr ? nullptr : static_cast<uint8_t*>(e.preact.p) + 2 * (m * e.preact.ld + n);
    out = static_cast<uint8_t*>(e.out.p) + 2 * (m * e.out.ld + n);
  }

  static __device__ __forceinline__ void words(const uint8_t* p, uint32_t (&w)[16]) {
    uint4 a, b, c, d;
    ld_global_v8(p, a, b);
    ld_global_v8(p + 32, c, d);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    w[8] = c.x, w[9] = c.y, w[10] = c.z, w[11] = c.w, w[12] = d.x, w[13] = d.y, w[14] = d.z, w[15] = d.w;
  }

  __device__ __forceinline__ void fetch(int col) {
    if (slope != nullptr) words(slope + 2 * col, slope_w);
    if (add != nullptr) words(add + 2 * col, add_w);
  }

  static __device__ __forceinline__ void store(uint8_t* p, const F2 (&v)[16]) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 f = split(v[j]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    st_global_v8(p, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
    st_global_v8(p + 32, make_uint4(w[8], w[9], w[10], w[11]), make_uint4(w[12], w[13], w[14], w[15]));
  }

  // Columns [col, col + 32) of the row (from column n of the output), from the sums in v;
  // `more`: the next 32 follow.
  __device__ __forceinline__ void finish(const Epilogue& e, int64_t n, int col, bool more, F2 (&v)[16]) {
    if (e.bias.p != nullptr) {
      if (e.bias.bf16) {
        uint32_t w[16];
        words(static_cast<const uint8_t*>(e.bias.p) + 2 * n, w);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          v[j] = add2(v[j], pair(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)));
      } else {
        const float* b = static_cast<const float*>(e.bias.p) + n;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 x, y;
          ld_global_v8(b + 8 * j, x, y);
          v[4 * j] = add2(v[4 * j], pair(__uint_as_float(x.x), __uint_as_float(x.y)));
          v[4 * j + 1] = add2(v[4 * j + 1], pair(__uint_as_float(x.z), __uint_as_float(x.w)));
          v[4 * j + 2] = add2(v[4 * j + 2], pair(__uint_as_float(y.x), __uint_as_float(y.y)));
          v[4 * j + 3] = add2(v[4 * j + 3], pair(__uint_as_float(y.z), __uint_as_float(y.w)));
        }
      }
    }
    if (preact != nullptr) store(preact + 2 * col, v);
    if (e.act != MUON_ACT_NONE) {
      float x[32];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 f = split(v[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
      }
      apply_act<32>(e.act, x);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = pair(x[2 * j], x[2 * j + 1]);
    }
    if (slope != nullptr) {
      float t[32], x[32];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 f = split(v[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
        t[2 * j] = __uint_as_float(slope_w[j] << 16);
        t[2 * j + 1] = __uint_as_float(slope_w[j] & 0xFFFF0000u);
      }
      apply_slope<32>(e.slope_act, t, x);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = pair(x[2 * j], x[2 * j + 1]);
    }
    if (add != nullptr) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        v[j] = add2(v[j], pair(__uint_as_float(add_w[j] << 16), __uint_as_float(add_w[j] & 0xFFFF0000u)));
    }
    if (more) fetch(col + 32);
    store(out + 2 * col, v);
  }
};

// Brings `cols` columns of row m from column n on into L2.
__device__ __forceinline__ void prefetch_row(const EpiView& v, int64_t m, int64_t n, int cols) {
  if (v.p == nullptr) return;
  const int step = v.bf16 ? 64 : 32;  // 128 bytes
  const char* p = static_cast<const char*>(v.p) + (m * v.ld + n) * (v.bf16 ? 2 : 4);
  for (int c = 0; c < cols; c += step) prefetch_l2(p + c * (v.bf16 ? 2 : 4));
}

// Row m, columns [n, n + NC) (n a multiple of 8) without a fetch ahead: the join kernel's.
template <int NC>
__device__ __forceinline__ void finish_segment(const Epilogue& e, int64_t m, int64_t n, float (&v)[NC]) {
  const int64_t left = e.cols - n;
  if (m >= e.rows || left <= 0) return;
  const int valid = left < NC ? static_cast<int>(left) : NC;
  float t[NC];
  if (e.bias.p != nullptr) {
    load_segment<NC>(e.bias, n, valid, t);
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] += t[j];
  }
  if (e.preact.p != nullptr) store_segment<NC>(e.preact, m * e.preact.ld + n, valid, v);
  apply_act<NC>(e.act, v);
  if (e.slope.p != nullptr) {
    load_segment<NC>(e.slope, m * e.slope.ld + n, valid, t);
    apply_slope<NC>(e.slope_act, t, v);
  }
  if (e.add.p != nullptr) {
    load_segment<NC>(e.add, m * e.add.ld + n, valid, t);
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] += t[j];
  }
  store_segment<NC>(e.out, m * e.out.ld + n, valid, v);
}

// Column n of rows [m, m + NC): neighbouring threads hold neighbouring columns.
template <int NC>
__device__ __forceinline__ void finish_column(const Epilogue& e, int64_t m, int64_t n, float (&v)[NC]) {
  if (n >= e.cols) return;
  const int64_t left = e.rows - m;
  const int valid = left < NC ? static_cast<int>(left) : NC;
  if (e.bias.p != nullptr) {
    const float b = load_elem(e.bias.p, n, e.bias.bf16);
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] += b;
  }
  if (e.preact.p != nullptr) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (j < valid) store_elem(e.preact.p, (m + j) * e.preact.ld + n, e.preact.bf16, v[j]);
  }
  apply_act<NC>(e.act, v);
  float t[NC];
  if (e.slope.p != nullptr) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      t[j] = j < valid ? load_elem(e.slope.p, (m + j) * e.slope.ld + n, e.slope.bf16) : 0.f;
    apply_slope<NC>(e.slope_act, t, v);
  }
  if (e.add.p != nullptr) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      t[j] = j < valid ? load_elem(e.add.p, (m + j) * e.add.ld + n, e.add.bf16) : 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] += t[j];
  }
#pragma unroll
  for (int j = 0; j < NC; ++j)
    if (j < valid) store_elem(e.out.p, (m + j) * e.out.ld + n, e.out.bf16, v[j]);
}

}  // namespace muon
