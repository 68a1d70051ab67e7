// Layer norm and its gradients.
//
//   y = (x - mean) rstd gain + bias,  mean = sum(x) / D,  rstd = 1 / sqrt(sum((x - mean)^2) / D + eps)
//   h = (x - mean) rstd,  q = dy gain
//   dx = rstd (q - avg(q) - h avg(q h)) + skip,  dgain = sum_rows dy h,  dbias = sum_rows dy
//
// The variance is summed from the centred values, never as E[x^2] - mean^2, and h is formed
// from the difference, never as x rstd - mean rstd: both cancel where the mean is large.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "muon_epilogue.cuh"
#include "muon_layers_host.h"

namespace muon {

struct NormParams {
  EpiView x, gain, bias, y;
  float* mean;
  float* rstd;
  int64_t rows;
  int32_t cols, stages;
  float eps;
  unsigned long long timeout_ns;
};

constexpr int kMaxStages = 4;

// Shared memory of a row of `bytes`: its 16-byte units, wherever it starts.
__host__ __device__ __forceinline__ uint32_t slot_bytes(uint32_t bytes) { return (bytes + 15u + 15u) & ~15u; }

struct NormGradParams {
  EpiView dy, x, gain, skip, dx;
  const float* mean;
  const float* rstd;
  float* dgain;
  float* dbias;
  float* partial;  // [slices][2][cols], or nullptr: no parameter gradients
  int64_t rows;
  int32_t cols, accumulate, slices, stages;
  unsigned long long timeout_ns;
};

// ------------------------------------------------------------------ a row and its threads
//
// A row is shared by TPR threads, NV groups of 8 elements each; a row group (a warp, or a
// block for wide rows) takes every gridDim-th row.  VEC: a group is 8 neighbouring elements;
// otherwise (odd widths, unaligned rows) its elements are TPR apart, so that a warp's
// accesses are contiguous all the same.  The arithmetic is in fp32 pairs: on bf16 rows the
// kernels are bound by instruction issue before memory (in scalar form the backward pass
// took 37 instructions an element, and 209 us instead of 149 us at 32768 x 4096, which rows
// without column checks brought to 129).

enum Form : int { kLoose = 0, kGroups8 = 1, kFull = 2 };  // not VEC; VEC; VEC and no thread without columns

template <int TPR_, int NV_, bool BF16_, int FORM_>
struct Rows {
  static constexpr int TPR = TPR_, NV = NV_;
  static constexpr bool BF16 = BF16_, VEC = FORM_ != kLoose, FULL = FORM_ == kFull;
  static constexpr int kThreads = TPR == 32 ? 128 : TPR;
  static constexpr int kGroups = kThreads / TPR;  // rows in flight per block
  static constexpr int kWarps = TPR / 32;         // warps per row
  // blocks per SM: what the registers allow, so that the persistent grid is one wave
  static constexpr int kForward = TPR == 32 ? (NV == 1 ? 8 : NV == 2 ? 6 : 4) : TPR == 128 ? 6 : TPR == 256 && NV == 2 ? 3
                                  : TPR == 256 ? 2 : 1;
  static constexpr int kBackward = TPR == 32 ? (NV == 1 ? 6 : NV <= 3 ? 4 : 3) : TPR == 128 ? 4
                                   : TPR == 256 && NV == 2 ? 2 : 1;
};

// Column of element j of group v of thread t.
template <class L>
__device__ __forceinline__ int column(int v, int j, int t) {
  return L::VEC ? (v * L::TPR + t) * 8 + j : (v * 8 + j) * L::TPR + t;
}

// Whether column c of this thread exists.
template <class L>
__device__ __forceinline__ bool exists(int c, int cols) {
  return L::FULL || c < cols;
}

// Group k of a vector (a gain, a bias), zero past the last column.
template <class L>
__device__ __forceinline__ void load_group(const EpiView& v, int k, int t, int cols, F2 (&x)[4]) {
  float e[8];
  if constexpr (L::VEC) {
    const int c = column<L>(k, 0, t);
    load_segment<8>(v, c, cols - c, e);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<L>(k, j, t);
      e[j] = c < cols ? load_elem(v.p, c, v.bf16) : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = pair(e[2 * j], e[2 * j + 1]);
}

// BF16: the dtype of `v`.
template <class L, bool BF16>
__device__ __forceinline__ void store_group(const EpiView& v, int64_t off, int k, int t, int cols, const F2 (&x)[4]) {
  if constexpr (L::VEC) {
    const int c = column<L>(k, 0, t);
    if (!exists<L>(c, cols)) return;
    const float2 a = split(x[0]), b = split(x[1]), d = split(x[2]), e = split(x[3]);
    if constexpr (BF16) {
      const __nv_bfloat162 q[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(b.x, b.y),
                                   __floats2bfloat162_rn(d.x, d.y), __floats2bfloat162_rn(e.x, e.y)};
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(v.p) + off + c) = *reinterpret_cast<const uint4*>(q);
    } else {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(v.p) + off + c);
      p[0] = make_float4(a.x, a.y, b.x, b.y);
      p[1] = make_float4(d.x, d.y, e.x, e.y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<L>(k, j, t);
      const float2 e = split(x[j >> 1]);
      if (c < cols) store_elem(v.p, off + c, BF16, (j & 1) ? e.y : e.x);
    }
  }
}

__device__ __forceinline__ float total(F2 a) {
  const float2 v = split(a);
  return v.x + v.y;
}

// Sums over the threads of a row.  More than one warp: through shared memory with one
// barrier; `turn` alternates two buffers, so the next sum does not overtake this one's reads.
template <class L, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float (*red)[N][32], int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = warp_sum(s[i]);
  if constexpr (L::kWarps > 1) {
    float(*b)[32] = red[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) b[i][threadIdx.x >> 5] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < L::kWarps; ++w) t += b[i][w];
      s[i] = t;
    }
  }
}

// The block's groups hold the same columns: the first adds the others' sums.
template <class L>
__device__ __forceinline__ void join_groups(F2 (*d)[4], F2* own, int group, int t) {
  __syncthreads();
#pragma unroll
  for (int e = 0; e < L::NV * 4; ++e) own[(group * L::NV * 4 + e) * L::TPR + t] = d[e >> 2][e & 3];
  __syncthreads();
  if (group == 0) {
#pragma unroll
    for (int e = 0; e < L::NV * 4; ++e)
#pragma unroll
      for (int g = 1; g < L::kGroups; ++g)
        d[e >> 2][e & 3] = add2(d[e >> 2][e & 3], own[(g * L::NV * 4 + e) * L::TPR + t]);
  }
}

// ------------------------------------------------------------------ rows through shared memory
//
// Rows arrive by bulk copies in a ring of stages per row group, so that the bytes in flight
// do not take registers.  A stage holds x, or x, dy and skip.  A bulk copy moves whole
// 16-byte units: it takes those that hold the row, and the row starts at its address modulo
// 16 in its slot.  (Bytes beside the row in its first and last unit are copied, not used.)
// A stage's refill is issued by one thread of the group after the sums of the next row,
// which every thread reaches only when it has read this row for the last time.
//
// Bound by HBM where rows are long, by the issue of the row sums' instructions where a warp has
// a short row, by the launch for few rows.  Captured calls (us, and of the measured copy
// bandwidth): forward bf16 32768 x 4096 91.4 (91%), 32768 x 768 18.0 (87%), 8 x 768 3.1; backward
// bf16 32768 x 4096 130 (96%), 16384 x 768 24.2 (65%, with the join of its parameter gradients),
// fp32 1001 x 1023 with unaligned rows 9.5.
//
// A copy that does not land within the budget is recorded in the status word; the group
// then carries on without waiting, so that every barrier is still met, and leaves.

__device__ int32_t g_norm_status[2];  // code, wait site

constexpr int kSiteNormRow = 5;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ const uint8_t* row_address(const EpiView& v, int64_t r) {
  return static_cast<const uint8_t*>(v.p) + r * v.ld * (v.bf16 ? 2 : 4);
}

// Where a row starts in its first 16-byte unit: at 0 in VEC calls.
template <class L>
__device__ __forceinline__ uint32_t within_unit(const void* row) {
  return L::VEC ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
}

// Bytes of the 16-byte units that hold a row of `bytes`, and their copy.
template <class L>
__device__ __forceinline__ uint32_t unit_bytes(const void* row, uint32_t bytes) {
  return (within_unit<L>(row) + bytes + 15u) & ~15u;
}

template <class L>
__device__ __forceinline__ void request_row(void* slot, const uint8_t* row, uint32_t bytes, uint64_t* bar) {
  bulk_load(slot, row - within_unit<L>(row), unit_bytes<L>(row, bytes), bar);
}

// Group k of a staged row, zero past the last column.
template <class L>
__device__ __forceinline__ void staged_group(const uint8_t* row, int bf16, int k, int t, int cols, F2 (&x)[4]) {
  if constexpr (!L::VEC) {
    float e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = column<L>(k, j, t);
      e[j] = c < cols ? load_elem(row, c, bf16) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = pair(e[2 * j], e[2 * j + 1]);
  } else {
    const int c = column<L>(k, 0, t);
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    if (bf16) {
      if (exists<L>(c, cols)) a = *reinterpret_cast<const uint4*>(row + 2 * c);
      const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = pair(__uint_as_float(q[j] << 16), __uint_as_float(q[j] & 0xFFFF0000u));
    } else {
      if (exists<L>(c, cols)) {
        a = *reinterpret_cast<const uint4*>(row + 4 * c);
        b = *reinterpret_cast<const uint4*>(row + 4 * c + 16);
      }
      x[0] = pair(__uint_as_float(a.x), __uint_as_float(a.y));
      x[1] = pair(__uint_as_float(a.z), __uint_as_float(a.w));
      x[2] = pair(__uint_as_float(b.x), __uint_as_float(b.y));
      x[3] = pair(__uint_as_float(b.z), __uint_as_float(b.w));
    }
  }
}

// The ring of one row group: stage s of a phase holds the group's (s + S n)-th row.
struct Ring {
  uint64_t* full;
  uint8_t* base;
  uint32_t stage_bytes;
  int stages;
  const Watchdog& wd;

  __device__ __forceinline__ uint8_t* stage(int s) const { return base + s * stage_bytes; }
  __device__ __forceinline__ void wait(int s, uint32_t phase) const {
    if (!*wd.abort) mbar_wait(&full[s], phase, wd, kSiteNormRow);
  }
};

// The phase of each stage's latest copy (kept by the thread that issues them).
struct Asked {
  uint32_t any = 0, parity = 0;

  __device__ __forceinline__ void add(int s) {
    const uint32_t bit = 1u << s;
    if (any & bit) parity ^= bit;
    any |= bit;
  }
};

// After a wait ran out, copies may still be in flight: none may land in memory that the
// block no longer owns.  (Otherwise every copy has been waited for.)
__device__ __forceinline__ void settle_ring(const Ring& ring, int t, const Asked& asked) {
  if (t != 0 || !*ring.wd.abort) return;
  const unsigned long long budget = ring.wd.budget > 2000000000ull ? ring.wd.budget : 2000000000ull;
  const uint64_t t0 = global_timer_ns();
  for (int s = 0; s < ring.stages; ++s)
    while (((asked.any >> s) & 1u) && !mbar_try_wait(&ring.full[s], (asked.parity >> s) & 1u) &&
           global_timer_ns() - t0 < budget) {
    }
}

template <class L>
__global__ void __launch_bounds__(L::kThreads, L::kForward) muon_layer_norm_ring_kernel(
    const __grid_constant__ NormParams p) {
  extern __shared__ __align__(128) uint8_t rows[];
  __shared__ float red[2][1][32];
  __shared__ uint64_t full[L::kGroups][kMaxStages];
  __shared__ int abort_flag;
  const int t = threadIdx.x % L::TPR, group = threadIdx.x / L::TPR;
  if (threadIdx.x == 0) abort_flag = 0;
  if (t == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&full[group][s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const Watchdog wd{&abort_flag, g_norm_status, p.timeout_ns};
  const uint32_t bytes = static_cast<uint32_t>(p.cols) * (L::BF16 ? 2 : 4), slot = slot_bytes(bytes);
  const Ring ring{full[group], rows + static_cast<uint32_t>(group * p.stages) * slot, slot, p.stages, wd};
  Asked asked;
  const int64_t step = static_cast<int64_t>(gridDim.x) * L::kGroups;
  int64_t r = static_cast<int64_t>(blockIdx.x) * L::kGroups + group;
  auto request = [&](int s, int64_t row) {
    asked.add(s);
    const uint8_t* x = row_address(p.x, row);
    mbar_arrive_expect_tx(&ring.full[s], unit_bytes<L>(x, bytes));
    request_row<L>(ring.stage(s), x, bytes, &ring.full[s]);
  };
  if (t == 0)
    for (int s = 0; s < p.stages; ++s)
      if (r + s * step < p.rows) request(s, r + s * step);
  F2 gain[L::NV][4], bias[L::NV][4];
#pragma unroll
  for (int k = 0; k < L::NV; ++k) {
#pragma unroll
    for (int j = 0; j < 4; ++j) gain[k][j] = pair(1.f), bias[k][j] = pair(0.f);
    if (p.gain.p != nullptr) load_group<L>(p.gain, k, t, p.cols, gain[k]);
    if (p.bias.p != nullptr) load_group<L>(p.bias, k, t, p.cols, bias[k]);
  }
  const float inv = 1.f / static_cast<float>(p.cols);
  int turn = 0, s = 0;
  uint32_t phase = 0;
  for (; r < p.rows; r += step) {
    ring.wait(s, phase);
    F2 x[L::NV][4], acc = pair(0.f);
    const uint8_t* row = ring.stage(s) + within_unit<L>(row_address(p.x, r));
#pragma unroll
    for (int k = 0; k < L::NV; ++k) {
      staged_group<L>(row, L::BF16, k, t, p.cols, x[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc = add2(acc, x[k][j]);
    }
    fence_proxy_async_smem();  // these reads come before the copy that refills the stage
    if constexpr (L::kWarps == 1) __syncwarp();
    float sum[1] = {total(acc)};
    row_sums<L, 1>(sum, red, turn);
    if (t == 0 && r + p.stages * step < p.rows) request(s, r + p.stages * step);
    const float mean = sum[0] * inv;
    acc = pair(0.f);
    const F2 shift = pair(-mean);
#pragma unroll
    for (int k = 0; k < L::NV; ++k) {
      if constexpr (L::VEC) {
        if (exists<L>(column<L>(k, 0, t), p.cols)) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[k][j] = add2(x[k][j], shift);
            acc = fma2(x[k][j], x[k][j], acc);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[k][j] = add2(x[k][j], pair(column<L>(k, 2 * j, t) < p.cols ? -mean : 0.f,
                                       column<L>(k, 2 * j + 1, t) < p.cols ? -mean : 0.f));
          acc = fma2(x[k][j], x[k][j], acc);
        }
      }
    }
    sum[0] = total(acc);
    row_sums<L, 1>(sum, red, turn);
    const float rstd = rsqrtf(fmaf(sum[0], inv, p.eps));
    const F2 scale = pair(rstd);
#pragma unroll
    for (int k = 0; k < L::NV; ++k) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[k][j] = fma2(mul2(x[k][j], scale), gain[k][j], bias[k][j]);
      store_group<L, L::BF16>(p.y, r * p.y.ld, k, t, p.cols, x[k]);
    }
    if (t == 0) {
      if (p.mean != nullptr) p.mean[r] = mean;
      if (p.rstd != nullptr) p.rstd[r] = rstd;
    }
    if (++s == p.stages) {
      s = 0;
      phase ^= 1u;
    }
  }
  settle_ring(ring, t, asked);
}

template <class L>
__global__ void __launch_bounds__(L::kThreads, L::kBackward) muon_layer_norm_backward_ring_kernel(
    const __grid_constant__ NormGradParams p) {
  extern __shared__ __align__(128) uint8_t rows[];
  __shared__ float red[2][2][32];
  __shared__ uint64_t full[L::kGroups][kMaxStages];
  __shared__ int abort_flag;
  const int t = threadIdx.x % L::TPR, group = threadIdx.x / L::TPR;
  if (threadIdx.x == 0) abort_flag = 0;
  if (t == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&full[group][s], 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const Watchdog wd{&abort_flag, g_norm_status, p.timeout_ns};
  const uint32_t bytes = static_cast<uint32_t>(p.cols) * (L::BF16 ? 2 : 4);
  const uint32_t skip_bytes = p.skip.p == nullptr ? 0u : static_cast<uint32_t>(p.cols) * (p.skip.bf16 ? 2 : 4);
  const uint32_t slot = slot_bytes(bytes), stage = 2 * slot + (skip_bytes ? slot_bytes(skip_bytes) : 0u);
  const Ring ring{full[group], rows + static_cast<uint32_t>(group * p.stages) * stage, stage, p.stages, wd};
  Asked asked;
  const int64_t step = static_cast<int64_t>(gridDim.x) * L::kGroups;
  int64_t r = static_cast<int64_t>(blockIdx.x) * L::kGroups + group;
  auto request = [&](int s, int64_t row) {
    asked.add(s);
    const uint8_t *x = row_address(p.x, row), *dy = row_address(p.dy, row), *skip = row_address(p.skip, row);
    uint32_t all = unit_bytes<L>(x, bytes) + unit_bytes<L>(dy, bytes);
    if (skip_bytes) all += unit_bytes<L>(skip, skip_bytes);
    mbar_arrive_expect_tx(&ring.full[s], all);
    request_row<L>(ring.stage(s), x, bytes, &ring.full[s]);
    request_row<L>(ring.stage(s) + slot, dy, bytes, &ring.full[s]);
    if (skip_bytes) request_row<L>(ring.stage(s) + 2 * slot, skip, skip_bytes, &ring.full[s]);
  };
  if (t == 0)
    for (int s = 0; s < p.stages; ++s)
      if (r + s * step < p.rows) request(s, r + s * step);
  F2 gain[L::NV][4], dgain[L::NV][4], dbias[L::NV][4];
#pragma unroll
  for (int k = 0; k < L::NV; ++k) {
#pragma unroll
    for (int j = 0; j < 4; ++j) gain[k][j] = pair(1.f), dgain[k][j] = pair(0.f), dbias[k][j] = pair(0.f);
    if (p.gain.p != nullptr) load_group<L>(p.gain, k, t, p.cols, gain[k]);
  }
  const float inv = 1.f / static_cast<float>(p.cols);
  float nmean = r < p.rows ? p.mean[r] : 0.f, nrstd = r < p.rows ? p.rstd[r] : 0.f;
  int turn = 0, s = 0, last = -1;
  uint32_t phase = 0;
  for (; r < p.rows; r += step) {
    const float mean = nmean, rstd = nrstd;
    if (r + step < p.rows) {
      nmean = p.mean[r + step];
      nrstd = p.rstd[r + step];
    }
    // h = (x - mean) rstd, the difference first: x rstd - mean rstd in one operation would lose
    // |mean| rstd 2^-24 of h.  Past the last column dy is 0 and h harmless.
    const F2 scale = pair(rstd), shift = pair(-mean);
    ring.wait(s, phase);
    const uint8_t* xrow = ring.stage(s) + within_unit<L>(row_address(p.x, r));
    const uint8_t* dyrow = ring.stage(s) + slot + within_unit<L>(row_address(p.dy, r));
    F2 aq2 = pair(0.f), aqh2 = pair(0.f);
#pragma unroll
    for (int k = 0; k < L::NV; ++k) {
      F2 x[4], dy[4];
      staged_group<L>(xrow, L::BF16, k, t, p.cols, x);
      staged_group<L>(dyrow, L::BF16, k, t, p.cols, dy);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 h = mul2(add2(x[j], shift), scale), q = mul2(dy[j], gain[k][j]);
        dgain[k][j] = fma2(dy[j], h, dgain[k][j]);
        dbias[k][j] = add2(dbias[k][j], dy[j]);
        aq2 = add2(aq2, q);
        aqh2 = fma2(q, h, aqh2);
      }
    }
    float sum[2] = {total(aq2), total(aqh2)};
    row_sums<L, 2>(sum, red, turn);
    if (t == 0 && last >= 0 && r + (p.stages - 1) * step < p.rows) request(last, r + (p.stages - 1) * step);
    if (p.dx.p != nullptr) {
      // dx = (q - aq - (x - mean) (rstd aqh)) rstd + skip
      const F2 c0 = pair(-sum[0] * inv), c1 = pair(-rstd * (sum[1] * inv));
#pragma unroll
      for (int k = 0; k < L::NV; ++k) {
        F2 x[4], dy[4];
        staged_group<L>(xrow, L::BF16, k, t, p.cols, x);
        staged_group<L>(dyrow, L::BF16, k, t, p.cols, dy);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = fma2(dy[j], gain[k][j], fma2(add2(x[j], shift), c1, c0));
        if (skip_bytes) {
          const uint8_t* skip = ring.stage(s) + 2 * slot + within_unit<L>(row_address(p.skip, r));
          staged_group<L>(skip, p.skip.bf16, k, t, p.cols, dy);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = fma2(x[j], scale, dy[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = mul2(x[j], scale);
        }
        store_group<L, L::BF16>(p.dx, r * p.dx.ld, k, t, p.cols, x);
      }
    }
    fence_proxy_async_smem();  // this row's reads come before the copy that refills its stage
    if constexpr (L::kWarps == 1) __syncwarp();
    last = s;
    if (++s == p.stages) {
      s = 0;
      phase ^= 1u;
    }
  }
  settle_ring(ring, t, asked);
  if (p.partial == nullptr) return;
  __syncthreads();  // the ring's memory is free: every group has read its last row
  F2* own = reinterpret_cast<F2*>(rows);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    F2(*d)[4] = which == 0 ? dgain : dbias;
    if constexpr (L::kGroups > 1) join_groups<L>(d, own, group, t);
    if (group == 0) {
      float* out = p.partial + (static_cast<int64_t>(blockIdx.x) * 2 + which) * p.cols;
      const EpiView o{out, 0, 0, L::VEC ? 1 : 0};
#pragma unroll
      for (int k = 0; k < L::NV; ++k) store_group<L, false>(o, 0, k, t, p.cols, d[k]);
    }
  }
}

// ------------------------------------------------------------------ wider rows

constexpr int kWideThreads = 512;

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

// One row per block, read three times (from L2 after the first).
__global__ void __launch_bounds__(kWideThreads) muon_layer_norm_wide_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[33];
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const int64_t xo = r * p.x.ld, yo = r * p.y.ld;
    float s = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += kWideThreads) s += load_elem(p.x.p, xo + c, p.x.bf16);
    const float mean = block_sum(s, red) / static_cast<float>(p.cols);
    s = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
      const float d = load_elem(p.x.p, xo + c, p.x.bf16) - mean;
      s = fmaf(d, d, s);
    }
    const float rstd = 1.f / sqrtf(block_sum(s, red) / static_cast<float>(p.cols) + p.eps);
    for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
      float v = (load_elem(p.x.p, xo + c, p.x.bf16) - mean) * rstd;
      if (p.gain.p != nullptr) v *= load_elem(p.gain.p, c, p.gain.bf16);
      if (p.bias.p != nullptr) v += load_elem(p.bias.p, c, p.bias.bf16);
      store_elem(p.y.p, yo + c, p.y.bf16, v);
    }
    if (threadIdx.x == 0) {
      if (p.mean != nullptr) p.mean[r] = mean;
      if (p.rstd != nullptr) p.rstd[r] = rstd;
    }
  }
}

__global__ void __launch_bounds__(kWideThreads) muon_layer_norm_dx_wide_kernel(
    const __grid_constant__ NormGradParams p) {
  __shared__ float red[33];
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const float mean = p.mean[r], rstd = p.rstd[r];
    float sq = 0.f, sqh = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
      float q = load_elem(p.dy.p, r * p.dy.ld + c, p.dy.bf16);
      if (p.gain.p != nullptr) q *= load_elem(p.gain.p, c, p.gain.bf16);
      sq += q;
      sqh = fmaf(q, (load_elem(p.x.p, r * p.x.ld + c, p.x.bf16) - mean) * rstd, sqh);
    }
    const float aq = block_sum(sq, red) / static_cast<float>(p.cols);
    const float aqh = block_sum(sqh, red) / static_cast<float>(p.cols);
    for (int c = threadIdx.x; c < p.cols; c += kWideThreads) {
      float q = load_elem(p.dy.p, r * p.dy.ld + c, p.dy.bf16);
      if (p.gain.p != nullptr) q *= load_elem(p.gain.p, c, p.gain.bf16);
      const float h = (load_elem(p.x.p, r * p.x.ld + c, p.x.bf16) - mean) * rstd;
      float v = rstd * (q - aq - h * aqh);
      if (p.skip.p != nullptr) v += load_elem(p.skip.p, r * p.skip.ld + c, p.skip.bf16);
      store_elem(p.dx.p, r * p.dx.ld + c, p.dx.bf16, v);
    }
  }
}

// Partial column sums of wide rows: block (b, s) takes 32 columns and every slices-th group
// of 8 rows.
__global__ void __launch_bounds__(256) muon_layer_norm_columns_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ float sg[8][33], sb[8][33];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float dg = 0.f, db = 0.f;
  if (c < p.cols)
    for (int64_t r = blockIdx.y * 8 + w; r < p.rows; r += int64_t(8) * gridDim.y) {
      const float dy = load_elem(p.dy.p, r * p.dy.ld + c, p.dy.bf16);
      const float h = (load_elem(p.x.p, r * p.x.ld + c, p.x.bf16) - p.mean[r]) * p.rstd[r];
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

// ------------------------------------------------------------------ parameter gradients

// Adds the slices' partial sums: 32 columns of one gradient per block, 32 warps over the
// slices with eight loads each on their way (a few hundred slices, so a few latencies).
__global__ void __launch_bounds__(1024) muon_layer_norm_join_kernel(const __grid_constant__ NormGradParams p) {
  __shared__ float sum[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, which = blockIdx.y;
  const int c = blockIdx.x * 32 + lane;
  float* out = which == 0 ? p.dgain : p.dbias;
  if (out == nullptr) return;
  float t = 0.f;
  if (c < p.cols) {
    const float* o = p.partial + static_cast<int64_t>(which) * p.cols + c;
#pragma unroll 8
    for (int s = w; s < p.slices; s += 32) t += o[static_cast<int64_t>(s) * 2 * p.cols];
  }
  sum[w][lane] = t;
  __syncthreads();
  if (w == 0 && c < p.cols) {
    t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += sum[k][lane];
    out[c] = p.accumulate ? out[c] + t : t;
  }
}

cudaError_t norm_status(int32_t (&out)[2], bool clear, cudaStream_t s) {
  const int32_t zero[2] = {0, 0};
  if (clear) return cudaMemcpyToSymbolAsync(g_norm_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
  return cudaMemcpyFromSymbolAsync(out, g_norm_status, sizeof(out), 0, cudaMemcpyDeviceToHost, s);
}

}  // namespace muon

namespace {
using namespace muon;

constexpr int kSms = 148;             // of the one part this library is built for
constexpr int kWidest = 512 * 2 * 8;  // columns of a row that a ring serves

bool sizes_ok(int64_t rows, int64_t cols) { return rows >= 0 && rows <= kMaxRows && cols >= 1 && cols <= kMaxSide; }

// Whether every row of the call can be moved 8 elements at a time.
bool whole_groups(int64_t cols, std::initializer_list<const EpiView*> views) {
  if (cols % 8 != 0) return false;
  for (const EpiView* v : views)
    if (v->p != nullptr && v->vec == 0) return false;
  return true;
}

// Blocks of a row kernel: what the SMs can hold at once, `per_sm` blocks each.
int64_t row_blocks(int64_t rows, int groups, int per_sm) {
  return std::max<int64_t>(1, std::min<int64_t>(ceil_div(rows, groups), int64_t(kSms) * per_sm));
}

// Calls f(threads per row, groups of 8 per thread) as compile-time constants for this width.
template <class F>
muon_status_t with_shape(int64_t cols, F&& f) {
  const int64_t g = ceil_div(cols, 8);
#define MUON_SHAPE(T, N) \
  if (g <= (T) * (N)) return f(std::integral_constant<int, T>(), std::integral_constant<int, N>())
  MUON_SHAPE(32, 1);
  MUON_SHAPE(32, 2);
  MUON_SHAPE(32, 3);
  MUON_SHAPE(32, 4);
  MUON_SHAPE(128, 2);
  MUON_SHAPE(256, 2);
  MUON_SHAPE(256, 3);
  MUON_SHAPE(512, 2);
#undef MUON_SHAPE
  return MUON_ERR_UNSUPPORTED_SHAPE;
}

// Shared memory and stages of a launch: as many stages as fit beside the other blocks of the
// SM, two to four, and `least` bytes for the final sums.
struct RingSize {
  int stages, bytes;
};

RingSize ring_size(int64_t stage_bytes, int groups, int per_sm, int64_t least) {
  const int64_t budget = (232448 / per_sm - 3 * 1024) / (groups * stage_bytes);
  const int64_t stages = std::max<int64_t>(2, std::min<int64_t>(kMaxStages, budget));
  return {static_cast<int>(stages), static_cast<int>(std::max(least, stages * groups * stage_bytes))};
}

template <auto Kernel, class P>  // (the kernel itself, not its type, so that each has its own static)
muon_status_t launch_rows(const P& p, int64_t blocks, int threads, int smem, cudaStream_t s) {
  static thread_local int configured_device = -1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MUON_ERR_CUDA;
  if (configured_device != dev) {
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448 - 2048) != cudaSuccess)
      return MUON_ERR_CUDA;
    configured_device = dev;
  }
  return queued(launch_dependent(Kernel, p, dim3(static_cast<unsigned>(blocks)), threads, s, smem));
}

template <int T, int N, bool BF16, int VEC>
muon_status_t run_norm(NormParams p, cudaStream_t s) {
  using L = Rows<T, N, BF16, VEC>;
  const RingSize ring = ring_size(slot_bytes(p.cols * (BF16 ? 2 : 4)), L::kGroups, L::kForward, 0);
  p.stages = ring.stages;
  return launch_rows<muon_layer_norm_ring_kernel<L>>(p, row_blocks(p.rows, L::kGroups, L::kForward), L::kThreads,
                                                     ring.bytes, s);
}

// Row blocks of the backward pass, each with a partial sum of its own.
template <int T, int N>
int64_t grad_blocks(int64_t rows) {
  using L = Rows<T, N, true, kFull>;
  return row_blocks(rows, L::kGroups, L::kBackward);
}

template <int T, int N, bool BF16, int VEC>
muon_status_t run_norm_grad(NormGradParams p, cudaStream_t s) {
  using L = Rows<T, N, BF16, VEC>;
  const int64_t stage = 2 * slot_bytes(p.cols * (BF16 ? 2 : 4)) +
                        (p.skip.p == nullptr ? 0 : slot_bytes(p.cols * (p.skip.bf16 ? 2 : 4)));
  const RingSize ring = ring_size(stage, L::kGroups, L::kBackward, L::kGroups > 1 ? L::kThreads * N * 8 * 4 : 0);
  p.stages = ring.stages;
  return launch_rows<muon_layer_norm_backward_ring_kernel<L>>(p, p.slices, L::kThreads, ring.bytes, s);
}

int slices_for(const muon_layer_norm_grad_t* d) {
  if (d->cols > kWidest) return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, ceil_div(d->rows, 64))));
  int64_t n = 1;
  with_shape(d->cols, [&](auto t, auto k) {
    n = grad_blocks<t(), k()>(d->rows);
    return MUON_OK;
  });
  return static_cast<int>(n);
}

size_t norm_grad_bytes(const muon_layer_norm_grad_t* d) {
  if ((d->dgain == nullptr && d->dbias == nullptr) || d->rows == 0) return 0;
  return kHeaderBytes + static_cast<size_t>(slices_for(d)) * 2 * static_cast<size_t>(d->cols) * sizeof(float);
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
  p.x = epi_view(d->x, d->rows, d->cols);
  p.gain = epi_view(d->gain, 1, d->cols);
  p.bias = epi_view(d->bias, 1, d->cols);
  p.y = epi_view(d->y, d->rows, d->cols);
  p.mean = d->mean;
  p.rstd = d->rstd;
  p.rows = d->rows;
  p.cols = static_cast<int32_t>(d->cols);
  p.eps = d->eps;
  p.timeout_ns = layers_wait_ns();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->cols > kWidest)
    return queued(launch_dependent(muon_layer_norm_wide_kernel, p,
                                   dim3(static_cast<unsigned>(row_blocks(d->rows, 1, 4))), kWideThreads, s));
  const bool vec = whole_groups(d->cols, {&p.x, &p.y, &p.gain, &p.bias}), bf16 = p.x.bf16 != 0;
  return with_shape(d->cols, [&](auto t, auto n) {
    // Forward, the checks for missing columns cost instructions but some shapes are quicker with
    // them; why is not known.  At 2^27 bf16 elements, us with and without: 256 columns 125, 111;
    // 512 99, 106; 768 104, 103; 1024 105, 101; 2048 101, 105; 4096 91, 101; 6144 96, 99; 8192
    // 110, 107.  At 2^26 fp32 elements: 256 104, 102; 512 102, 103; 768 93, 105; 1024 98, 107;
    // 2048 95, 97; 4096 101, 95; 6144 104, 102; 8192 111, 108.  So a warp's row and the widest
    // leave them out in bf16, a block's row in fp32 (bf16 512 and fp32 2048 lose 7% and 2% by
    // that).  Backward they always cost: 4096 bf16 149, 131.
    constexpr bool wide32 = t() >= 128, full16 = t() == 32 || t() == 512;
    const bool full = d->cols == t() * n() * 8;
    if (vec && full && bf16 && full16) return run_norm<t(), n(), true, full16 ? kFull : kGroups8>(p, s);
    if (vec && full && !bf16 && wide32) return run_norm<t(), n(), false, wide32 ? kFull : kGroups8>(p, s);
    if (vec) return bf16 ? run_norm<t(), n(), true, kGroups8>(p, s) : run_norm<t(), n(), false, kGroups8>(p, s);
    return bf16 ? run_norm<t(), n(), true, kLoose>(p, s) : run_norm<t(), n(), false, kLoose>(p, s);
  });
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
  if (d->dx.data == nullptr && !grads && d->rows > 0) ops.fail(MUON_ERR_INVALID_ARG);
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
  if (d->rows == 0) {  // the sums are empty
    const size_t n = static_cast<size_t>(d->cols) * 4;
    if (!d->accumulate && ((d->dgain != nullptr && cudaMemsetAsync(d->dgain, 0, n, s) != cudaSuccess) ||
                           (d->dbias != nullptr && cudaMemsetAsync(d->dbias, 0, n, s) != cudaSuccess)))
      return MUON_ERR_CUDA;
    return MUON_OK;
  }
  NormGradParams p{};
  p.dy = epi_view(d->dy, d->rows, d->cols);
  p.x = epi_view(d->x, d->rows, d->cols);
  p.gain = epi_view(d->gain, 1, d->cols);
  p.skip = epi_view(d->skip, d->rows, d->cols);
  p.dx = epi_view(d->dx, d->rows, d->cols);
  p.mean = d->mean;
  p.rstd = d->rstd;
  p.dgain = d->dgain;
  p.dbias = d->dbias;
  p.partial = grads ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kHeaderBytes) : nullptr;
  p.rows = d->rows;
  p.cols = static_cast<int32_t>(d->cols);
  p.accumulate = d->accumulate;
  p.timeout_ns = layers_wait_ns();
  p.slices = slices_for(d);
  if (d->cols > kWidest) {
    if (d->dx.data != nullptr)
      st = queued(launch_dependent(muon_layer_norm_dx_wide_kernel, p,
                                   dim3(static_cast<unsigned>(row_blocks(d->rows, 1, 4))), kWideThreads, s));
    if (st == MUON_OK && grads)
      st = queued(launch_dependent(
          muon_layer_norm_columns_kernel, p,
          dim3(static_cast<unsigned>(ceil_div(d->cols, 32)), static_cast<unsigned>(p.slices)), 256, s));
  } else {
    const bool vec = whole_groups(d->cols, {&p.x, &p.dy, &p.gain, &p.skip, &p.dx}), bf16 = p.x.bf16 != 0;
    st = with_shape(d->cols, [&](auto t, auto n) {
      const bool full = d->cols == t() * n() * 8;
      if (vec && full)
        return bf16 ? run_norm_grad<t(), n(), true, kFull>(p, s) : run_norm_grad<t(), n(), false, kFull>(p, s);
      if (vec)
        return bf16 ? run_norm_grad<t(), n(), true, kGroups8>(p, s) : run_norm_grad<t(), n(), false, kGroups8>(p, s);
      return bf16 ? run_norm_grad<t(), n(), true, kLoose>(p, s) : run_norm_grad<t(), n(), false, kLoose>(p, s);
    });
  }
  if (st != MUON_OK || !grads) return st;
  return queued(launch_dependent(muon_layer_norm_join_kernel, p, dim3(static_cast<unsigned>(ceil_div(d->cols, 32)), 2),
                                 1024, s));
}
