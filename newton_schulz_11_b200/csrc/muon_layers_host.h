// Host-side checks shared by the layer entry points.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "muon_b200.h"
#include "muon_product.h"

namespace muon {

inline bool aligned_bytes(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline size_t elem_bytes(int32_t dtype) { return dtype == MUON_BF16 ? 2 : 4; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The bytes of one strided operand, for the overlap check.
struct Span {
  uintptr_t lo, hi, pitch, width;
  int64_t rows;
  bool written;
};

// Collects a call's operands, checking each; `status` keeps the first error.  (An array of the
// most a call has: nothing here can throw through the C ABI.)
struct Operands {
  static constexpr int kMost = 10;
  Span spans[kMost];
  int count = 0;
  muon_status_t status = MUON_OK;

  void fail(muon_status_t s) {
    if (status == MUON_OK) status = s;
  }

  void put(const Span& s) {
    if (count < kMost)
      spans[count++] = s;
    else
      fail(MUON_ERR_INVALID_ARG);
  }

  // `required` views must have data; an absent optional one is skipped.
  void add(const muon_view_t& v, int64_t rows, int64_t cols, bool required, bool written) {
    if (v.data == nullptr) {
      if (required && rows > 0) fail(MUON_ERR_INVALID_ARG);
      return;
    }
    if (v.dtype != MUON_F32 && v.dtype != MUON_BF16) return fail(MUON_ERR_UNSUPPORTED_DTYPE);
    const int64_t ld = rows == 1 ? cols : v.ld;
    if (ld < cols || ld > (int64_t(1) << 40)) return fail(MUON_ERR_UNSUPPORTED_SHAPE);
    const size_t e = elem_bytes(v.dtype);
    if (!aligned_bytes(v.data, e)) return fail(MUON_ERR_ALIGNMENT);
    if (rows == 0) return;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(v.data);
    const uintptr_t bytes = static_cast<uintptr_t>(((rows - 1) * ld + cols) * static_cast<int64_t>(e));
    put({lo, lo + bytes, static_cast<uintptr_t>(ld) * e, static_cast<uintptr_t>(cols) * e, rows, written});
  }

  void add_f32(const float* p, int64_t n, bool required, bool written) {
    if (n == 0) return;
    muon_view_t v{const_cast<float*>(p), n, MUON_F32, 0};
    add(v, 1, n, required, written);
  }

  void add_bytes(const void* p, size_t n) {
    if (n > 0) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
      put({lo, lo + n, n, n, 1, true});
    }
  }

  // Whether two operands share a byte.  Views of one buffer (the same pitch) are compared
  // row by row; otherwise overlapping extents count as sharing.
  static bool meet(const Span& a, const Span& b) {
    if (a.hi <= b.lo || b.hi <= a.lo) return false;
    const Span& x = a.lo <= b.lo ? a : b;
    const Span& y = a.lo <= b.lo ? b : a;
    if (x.pitch != y.pitch) return true;
    const uintptr_t d = y.lo - x.lo;
    const int64_t row = static_cast<int64_t>(d / x.pitch);
    const uintptr_t off = d % x.pitch;
    if (row < x.rows && off < x.width) return true;
    return row + 1 < x.rows && off + y.width > x.pitch;
  }

  // No written operand may share bytes with another.
  muon_status_t check() const {
    if (status != MUON_OK) return status;
    for (int i = 0; i < count; ++i)
      for (int j = i + 1; j < count; ++j)
        if ((spans[i].written || spans[j].written) && meet(spans[i], spans[j])) return MUON_ERR_INVALID_ARG;
    return MUON_OK;
  }
};

// y may be the residual itself: the same elements, each read before it is written.
inline bool same_view(const muon_view_t& a, const muon_view_t& b, int64_t rows) {
  return a.data == b.data && a.dtype == b.dtype && (a.ld == b.ld || rows <= 1);
}

// Row stride in elements: one row has none of its own.
inline int64_t row_stride(const muon_view_t& v, int64_t rows, int64_t cols) { return rows <= 1 ? cols : v.ld; }

// A view as the kernels take it, with the widest access its address and row stride allow.
inline EpiView epi_view(const muon_view_t& v, int64_t rows, int64_t cols) {
  EpiView e{v.data, row_stride(v, rows, cols), v.dtype == MUON_BF16 ? 1 : 0, 0};
  const size_t pitch = static_cast<size_t>(e.ld) * elem_bytes(v.dtype);
  const bool one = rows <= 1;
  for (int k = 1; k <= 2; ++k)
    if (aligned_bytes(v.data, 16 * k) && (one || pitch % (16 * k) == 0)) e.vec = k;
  return e;
}

// MUON_OK and the SM count when the current device is an sm_100 GPU.
muon_status_t layers_device(int* sms);

// Device status word of the layer kernels, and the budget of their waits.
unsigned long long layers_wait_ns();

// Reads (or clears) the status word of the norm kernels, queued on `s`.
cudaError_t norm_status(int32_t (&out)[2], bool clear, cudaStream_t s);

inline muon_status_t queued(cudaError_t e) { return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA; }

// The start of a workspace: the step's status word and counts (muon_workspace_init).  The
// layers leave it alone, so that one region can serve both.
constexpr size_t kHeaderBytes = 256;

constexpr int64_t kMaxSide = int64_t(1) << 24;  // columns, features (as for muon_matrix_t)
constexpr int64_t kMaxRows = int64_t(1) << 30;  // tokens

}  // namespace muon
