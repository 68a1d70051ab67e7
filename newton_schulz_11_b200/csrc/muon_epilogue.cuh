// The epilogue of the layer products: loads and stores of row segments, and the arithmetic.
#pragma once

#include "muon_device.cuh"
#include "muon_layers.cuh"
#include "muon_product.h"

namespace muon {

// N 32-bit words from byte address `a`, which need not be aligned to 16: the 16-byte units
// that hold them, shifted into place.  Units from `end` on (the end of the row) are not
// touched; their words are zero.  HALVES: `a` is a multiple of 2, else of 4.
template <int N, bool HALVES>
__device__ __forceinline__ void load_shifted(uintptr_t a, uintptr_t end, uint32_t (&x)[N]) {
  const uint32_t o = static_cast<uint32_t>(a & 15u);
  const uintptr_t u = a - o;
  uint32_t w[N + 4];
#pragma unroll
  for (int i = 0; i < N / 4 + 1; ++i) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if ((i < N / 4 || o != 0) && u + 16 * i < end) v = *reinterpret_cast<const uint4*>(u + 16 * i);
    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
  }
  if (o & 8u) {
#pragma unroll
    for (int i = 0; i < N + 2; ++i) w[i] = w[i + 2];
  }
  if (o & 4u) {
#pragma unroll
    for (int i = 0; i < N + 1; ++i) w[i] = w[i + 1];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = HALVES && (o & 2u) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
}

// NC (a multiple of 8) consecutive elements of a row, the first `valid` of them; the rest
// are left at zero.  `off` is the element offset of the segment.
template <int NC>
__device__ __forceinline__ void load_segment(const EpiView& v, int64_t off, int valid, float (&x)[NC]) {
  const bool whole = valid >= NC && v.vec != 0;
  if (v.bf16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(v.p) + off;
#pragma unroll
    for (int h = 0; h < NC / 8; ++h) {
      uint32_t q[4];
      if (whole) {
        const uint4 w = reinterpret_cast<const uint4*>(p)[h];
        q[0] = w.x, q[1] = w.y, q[2] = w.z, q[3] = w.w;
      } else {
        load_shifted<4, true>(reinterpret_cast<uintptr_t>(p + 8 * h), reinterpret_cast<uintptr_t>(p + valid), q);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * h + 2 * j] = __uint_as_float(q[j] << 16);
        x[8 * h + 2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
      }
    }
  } else {
    const float* p = static_cast<const float*>(v.p) + off;
#pragma unroll
    for (int h = 0; h < NC / 8; ++h) {
      uint32_t q[8];
      if (whole && v.vec == 2) {
        uint4 a, b;
        ld_global_v8(p + 8 * h, a, b);
        q[0] = a.x, q[1] = a.y, q[2] = a.z, q[3] = a.w, q[4] = b.x, q[5] = b.y, q[6] = b.z, q[7] = b.w;
      } else {
        load_shifted<8, false>(reinterpret_cast<uintptr_t>(p + 8 * h), reinterpret_cast<uintptr_t>(p + valid), q);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) x[8 * h + j] = __uint_as_float(q[j]);
    }
  }
  if (valid < NC) {  // what shares a unit with the row's end
#pragma unroll
    for (int j = 0; j < NC; ++j) x[j] = j < valid ? x[j] : 0.f;
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

template <int NC>
__device__ __forceinline__ void load_pairs(const EpiView& v, int64_t off, int valid, F2 (&x)[NC / 2]) {
  float e[NC];
  load_segment<NC>(v, off, valid, e);
#pragma unroll
  for (int j = 0; j < NC / 2; ++j) x[j] = pair(e[2 * j], e[2 * j + 1]);
}

template <int NC>
__device__ __forceinline__ void store_pairs(const EpiView& v, int64_t off, int valid, const F2 (&x)[NC / 2]) {
  float e[NC];
#pragma unroll
  for (int j = 0; j < NC / 2; ++j) {
    const float2 f = split(x[j]);
    e[2 * j] = f.x;
    e[2 * j + 1] = f.y;
  }
  store_segment<NC>(v, off, valid, e);
}

// ------------------------------------------------------------------ the common epilogue
//
// When everything but the bias is bf16 in rows of whole 32-byte units, NC = 16 or 32 columns
// of a row are one or two 32-byte accesses of each operand.  The epilogue's pace is its
// number of instructions times their latency over the few warps that run it, so this path
// has no choices inside: addresses are carried per row, and the inputs are fetched a step
// ahead.
template <int NC>
struct EpiRow {
  static constexpr int W = NC / 2;  // 32-bit words of NC bf16 values
  const uint8_t* slope;
  const uint8_t* add;
  uint8_t* preact;
  uint8_t* out;
  uint32_t slope_w[W], add_w[W];

  __device__ __forceinline__ void start(const Epilogue& e, int64_t m, int64_t n) {
    slope = e.slope.p == nullptr ? nullptr : static_cast<const uint8_t*>(e.slope.p) + 2 * (m * e.slope.ld + n);
    add = e.add.p == nullptr ? nullptr : static_cast<const uint8_t*>(e.add.p) + 2 * (m * e.add.ld + n);
    preact = e.preact.p == nullptr ? nullptr : static_cast<uint8_t*>(e.preact.p) + 2 * (m * e.preact.ld + n);
    out = static_cast<uint8_t*>(e.out.p) + 2 * (m * e.out.ld + n);
  }

  static __device__ __forceinline__ void words(const uint8_t* p, uint32_t (&w)[W]) {
#pragma unroll
    for (int i = 0; i < W / 8; ++i) {
      uint4 a, b;
      ld_global_v8(p + 32 * i, a, b);
      w[8 * i] = a.x, w[8 * i + 1] = a.y, w[8 * i + 2] = a.z, w[8 * i + 3] = a.w;
      w[8 * i + 4] = b.x, w[8 * i + 5] = b.y, w[8 * i + 6] = b.z, w[8 * i + 7] = b.w;
    }
  }

  static __device__ __forceinline__ F2 value(uint32_t w) {
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }

  __device__ __forceinline__ void fetch(int col) {
    if (slope != nullptr) words(slope + 2 * col, slope_w);
    if (add != nullptr) words(add + 2 * col, add_w);
  }

  static __device__ __forceinline__ void store(uint8_t* p, const F2 (&v)[W]) {
    uint32_t w[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float2 f = split(v[j]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
#pragma unroll
    for (int i = 0; i < W / 8; ++i)
      st_global_v8(p + 32 * i, make_uint4(w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3]),
                   make_uint4(w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]));
  }

  // Columns [col, col + NC) of the row (from column n of the output), from the sums in v;
  // `more`: the next NC follow.
  __device__ __forceinline__ void finish(const Epilogue& e, int64_t n, int col, bool more, F2 (&v)[W]) {
    if (e.bias.p != nullptr) {
      if (e.bias.bf16) {
        uint32_t w[W];
        words(static_cast<const uint8_t*>(e.bias.p) + 2 * n, w);
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = add2(v[j], value(w[j]));
      } else {
        const float* b = static_cast<const float*>(e.bias.p) + n;
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
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
    apply_act<W>(e.act, v);
    if (slope != nullptr) {
      F2 t[W];
#pragma unroll
      for (int j = 0; j < W; ++j) t[j] = value(slope_w[j]);
      apply_slope<W>(e.slope_act, t, v);
    }
    if (add != nullptr) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = add2(v[j], value(add_w[j]));
    }
    if (more) fetch(col + NC);
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

// Row m, columns [n, n + NC) of the output (n a multiple of 8), whatever its operands are.
template <int NC>
__device__ __forceinline__ void finish_segment(const Epilogue& e, int64_t m, int64_t n, F2 (&v)[NC / 2]) {
  const int64_t left = e.cols - n;
  if (m >= e.rows || left <= 0) return;
  const int valid = left < NC ? static_cast<int>(left) : NC;
  F2 t[NC / 2];
  if (e.bias.p != nullptr) {
    load_pairs<NC>(e.bias, n, valid, t);
#pragma unroll
    for (int j = 0; j < NC / 2; ++j) v[j] = add2(v[j], t[j]);
  }
  if (e.preact.p != nullptr) store_pairs<NC>(e.preact, m * e.preact.ld + n, valid, v);
  apply_act<NC / 2>(e.act, v);
  if (e.slope.p != nullptr) {
    load_pairs<NC>(e.slope, m * e.slope.ld + n, valid, t);
    apply_slope<NC / 2>(e.slope_act, t, v);
  }
  if (e.add.p != nullptr) {
    load_pairs<NC>(e.add, m * e.add.ld + n, valid, t);
#pragma unroll
    for (int j = 0; j < NC / 2; ++j) v[j] = add2(v[j], t[j]);
  }
  store_pairs<NC>(e.out, m * e.out.ld + n, valid, v);
}

// Column n of rows [m, m + NC): neighbouring threads hold neighbouring columns.
template <int NC>
__device__ __forceinline__ void load_column(const EpiView& v, int64_t m, int64_t n, int valid, F2 (&x)[NC / 2]) {
  float e[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) e[j] = j < valid ? load_elem(v.p, (m + j) * v.ld + n, v.bf16) : 0.f;
#pragma unroll
  for (int j = 0; j < NC / 2; ++j) x[j] = pair(e[2 * j], e[2 * j + 1]);
}

template <int NC>
__device__ __forceinline__ void store_column(const EpiView& v, int64_t m, int64_t n, int valid,
                                             const F2 (&x)[NC / 2]) {
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const float2 f = split(x[j / 2]);
    if (j < valid) store_elem(v.p, (m + j) * v.ld + n, v.bf16, (j & 1) ? f.y : f.x);
  }
}

template <int NC>
__device__ __forceinline__ void finish_column(const Epilogue& e, int64_t m, int64_t n, F2 (&v)[NC / 2]) {
  const int64_t left = e.rows - m;
  if (n >= e.cols || left <= 0) return;
  const int valid = left < NC ? static_cast<int>(left) : NC;
  F2 t[NC / 2];
  if (e.bias.p != nullptr) {
    const F2 b = pair(load_elem(e.bias.p, n, e.bias.bf16));
#pragma unroll
    for (int j = 0; j < NC / 2; ++j) v[j] = add2(v[j], b);
  }
  if (e.preact.p != nullptr) store_column<NC>(e.preact, m, n, valid, v);
  apply_act<NC / 2>(e.act, v);
  if (e.slope.p != nullptr) {
    load_column<NC>(e.slope, m, n, valid, t);
    apply_slope<NC / 2>(e.slope_act, t, v);
  }
  if (e.add.p != nullptr) {
    load_column<NC>(e.add, m, n, valid, t);
#pragma unroll
    for (int j = 0; j < NC / 2; ++j) v[j] = add2(v[j], t[j]);
  }
  store_column<NC>(e.out, m, n, valid, v);
}

}  // namespace muon
