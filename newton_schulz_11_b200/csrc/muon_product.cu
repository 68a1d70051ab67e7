// The products of the layers on the 5th-generation tensor cores (tcgen05, sm_100a).
//
//   D[M x N] = sum_k A(m, k) B(n, k), then the epilogue of muon_epilogue.cuh
//
// Two warp-specialised kernels, one for large products and one for small ones, serve x W^T
// (both operands contiguous along k), dy W (W contiguous along its side) and dy^T x (both
// contiguous along their sides): the majorness of each operand is a run-time property of the
// launch.
//
// Operand precision.  A bf16 operand is read as it is.  An fp32 operand comes as three bf16
// terms, x = h + m + l exactly (pack_terms), and the product as the sum of the term products
// whose size is at least 2^-16 of the whole: h h, h m, m h, m m, h l, l h (six), or h b, m b,
// l b against a bf16 operand (three).  The large products walk the k-blocks of a piece once
// per term product, the smallest first, all into one accumulator (a second one would not fit
// tensor memory); the small ones walk them once, see Walk.
//
// Sums.  The tensor cores add 16 products at a time to the fp32 accumulator and truncate.
// Left alone that costs about 1.1e-9 K relative for zero-mean data (measured: 9e-6 at
// K = 8192, 1.9e-5 at K = 16384) and up to 6e-9 K for products of one sign (1.3e-5 at K = 4096,
// 7.8e-4 at K = 131072): far below a bf16 output's half step up to K = 4096 but not below
// fp32's.  The Sum variants and the small products therefore end the accumulation after 512 of
// k (5e-7 by the same rate; 256 where an operand is fp32, measured 2.8e-7), read the accumulator
// into registers and add it there with rounding to nearest; large products with bf16 results
// do so after 2048 of k where the reduction is longer than 4096.
#include <cuda_runtime.h>

#include <algorithm>

#include "muon_epilogue.cuh"
#include "muon_layers_host.h"

namespace muon {

__device__ int32_t g_layers_status[2];  // code, wait site

enum ProductSite : int {
  kSiteLoad = 1,      // producer: a stage to be consumed
  kSiteAccFree = 2,   // MMA issuer: an accumulator to be read
  kSiteStage = 3,     // MMA issuer: a stage to be filled
  kSiteAccReady = 4,  // epilogue: an accumulator to be finished
};

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// The box lands in this CTA; its bytes complete on the leader CTA's mbarrier.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster, int32_t c0,
                                                 int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar_cluster)
      : "memory");
}

template <int NC>
__device__ __forceinline__ void tmem_load_row(uint32_t taddr, uint32_t (&v)[NC]) {
  if constexpr (NC == 32)
    tmem_ld_32x32b_x32(taddr, v);
  else
    tmem_ld_32x32b_x16(taddr, v);
  tmem_wait_ld();
}

// 16 columns of this thread's lane, written.
__device__ __forceinline__ void tmem_store_row16(uint32_t taddr, const float* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "f"(x[8]), "f"(x[9]),
      "f"(x[10]), "f"(x[11]), "f"(x[12]), "f"(x[13]), "f"(x[14]), "f"(x[15])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Sums of columns over the rows: block b takes 64 columns, 8 a thread, and every slices-th
// group of 32 rows.  256 threads.  U rows a thread are on their way at once: the row loop is
// written out per type, since a load that branches on its operand's layout is not hoisted above
// the one before it (one row at a time: 2000 x 2000 fp32 5.4 us, 4.6 like this; 16384 x 768 bf16
// 9.5, 7.0; riding under both gradients of 8192 x 4096 x 1024, 145 and 132).
template <int U, bool BF16>
__device__ __forceinline__ int64_t sum_rows(const ColumnSumTask& p, int64_t r, int c, F2 (&s)[4]) {
  constexpr int kWords = BF16 ? 1 : 2;
  const int64_t step = int64_t(32) * p.slices, pitch = p.src.ld * (BF16 ? 2 : 4);
  const uint8_t* at = static_cast<const uint8_t*>(p.src.p) + r * pitch + c * (BF16 ? 2 : 4);
  for (; r + (U - 1) * step < p.rows; r += U * step, at += U * step * pitch) {
    uint4 v[U][kWords];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < kWords; ++k) v[u][k] = *reinterpret_cast<const uint4*>(at + u * step * pitch + 16 * k);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t w[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w,
                             v[u][kWords - 1].x, v[u][kWords - 1].y, v[u][kWords - 1].z, v[u][kWords - 1].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[j] = add2(s[j], BF16 ? EpiRow<16>::value(w[j])
                               : pair(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1])));
    }
  }
  return r;
}

template <int U>
__device__ __forceinline__ void column_sums(const ColumnSumTask& p, int b, float (*red)[64]) {
  const int g = threadIdx.x & 7, w = threadIdx.x >> 3;
  const int blocks = (p.cols + 63) / 64;
  const int slice = b / blocks, c0 = (b - slice * blocks) * 64;
  const int c = c0 + g * 8;
  F2 s[4] = {0ull, 0ull, 0ull, 0ull};  // zeros
  if (c < p.cols) {
    int64_t r = slice * 32 + w;
    if (p.src.vec > 0 && c + 8 <= p.cols)
      r = p.src.bf16 ? sum_rows<U, true>(p, r, c, s) : sum_rows<U / 2, false>(p, r, c, s);
    for (; r < p.rows; r += int64_t(32) * p.slices) {
      F2 x[4];
      load_pairs<8>(p.src, r * p.src.ld + c, p.cols - c, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = add2(s[j], x[j]);
    }
  }
  named_barrier(1, 256);  // an earlier task's sums have been read
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(&red[w][g * 8 + 2 * j]) = split(s[j]);
  named_barrier(1, 256);
  const int o = c0 + threadIdx.x;
  if (threadIdx.x < 64 && o < p.cols) {
    float t = red[0][threadIdx.x];
#pragma unroll
    for (int k = 1; k < 32; ++k) t += red[k][threadIdx.x];
    if (p.slices == 1)
      p.out[o] = p.accumulate ? p.out[o] + t : t;
    else
      p.partial[static_cast<int64_t>(slice) * p.cols + o] = t;
  }
}

// The blocks of a product's launch that sum columns instead.
__device__ __forceinline__ void run_column_sums(const ProductParams& p, uint8_t* smem) {
  griddep_wait();
  griddep_launch_dependents();
  if (threadIdx.x >= 256) return;
  float(*red)[64] = reinterpret_cast<float(*)[64]>(smem);
  for (int b = static_cast<int>(blockIdx.x) - p.sum_from; b < p.sum_tasks; b += p.sum_blocks)
    column_sums<16>(p.sum, b, red);
}

// ------------------------------------------------------------------ large products
//
// A CTA pair shares a tile of 256 x 256 (tcgen05.mma.cta_group::2): each CTA stages its own
// 128 rows of A and of B, 64 deep, 32 KB per k-block for 128 x 256 x 64 of work, in seven
// stages; one thread of the leader CTA issues the MMAs; the two accumulators let the
// epilogue of one tile run under the products of the next.  Persistent over a list of tiles.
// SUM: the reduction in pieces added in registers.  FLIP: the tile's rows are the output's
// columns.
//
// Bound by the tensor cores (under the power cap) where k is long: 8192 x 4096 x 14336 (tokens,
// in, out) with the kept pre-activation in 690 us, 1394 TF/s; by the epilogue's traffic and the
// last wave where it is short: 16384 x 768 x 768 with a residual in 27 us (192 tiles are 2.6
// waves of 74), 2.8 TB/s; and dy^T x of 8192 x 4096 x 1024, 64 tiles for 74 pairs, in 75 us.
template <bool SUM_, bool FLIP_>
struct Pair {
  static constexpr int TM = 256, TN = 256;
  static constexpr bool SUM = SUM_, FLIP = FLIP_;
  static constexpr int BK = kProductBK;
  static constexpr int kABytes = 128 * BK * 2;
  static constexpr int kStageBytes = 2 * kABytes;
  static constexpr int S = 7;
  static constexpr int kBarOff = S * kStageBytes;
  static constexpr int kSmemBytes = kBarOff + 256 + 1024;
  // Epilogue warps.  (16, with half the columns each, measured 3-8% slower: 29.5 against
  // 27.2 us at 16384x768x768 with residual, 210 against 197 us at 8192x4096x4096.)
  static constexpr int NEPI = 8;
  static constexpr int kThreads = 64 + 32 * NEPI;
  static constexpr int NCW = TN * 4 / NEPI;       // accumulator columns per epilogue thread
  static constexpr int GC = 16;               // finished at a time; the common epilogue: 32
  static constexpr int kTmemCols = 2 * TN;
  // Whether the common epilogue has code of its own.  Beside the sums' registers it spills: in
  // pieces of 2048 of k, 8192 x 4096 x 14336 took 745 us with it and 708 without.
  static constexpr bool kPlain = !FLIP && !SUM;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert((2 * S + 5) * 8 + 16 <= 256, "barrier area");
};

// One unit of work: a tile and a range of k-blocks.
struct Unit {
  int i, j, split, kb0, kb1;
};

// Tiles are walked in bands of 8 along M, so that the tiles in flight at one time share
// rows of A and of B in L2.
__device__ __forceinline__ Unit decode_unit(const ProductParams& p, int t) {
  const int tiles = p.tiles_m * p.tiles_n;
  Unit u;
  u.split = t / tiles;
  const int q = t - u.split * tiles;
  const int band = q / (8 * p.tiles_n);
  const int first = 8 * band;
  const int height = p.tiles_m - first < 8 ? p.tiles_m - first : 8;
  const int in = q - band * 8 * p.tiles_n;
  u.j = in / height;
  u.i = first + (in - u.j * height);
  u.kb0 = u.split * p.kb_per_split;
  u.kb1 = u.kb0 + p.kb_per_split < p.nk ? u.kb0 + p.kb_per_split : p.nk;
  return u;
}

// One operand's k-block into `dst`: 128 of its side from side0, 64 of k from k0, its bytes
// completing on the leader's barrier.  K-major: one box of 64 k x 128; side-major: two boxes
// of 64 x 64 k.
__device__ __forceinline__ void load_pair_operand(uint8_t* dst, const CUtensorMap* map, int mn, int side0, int k0,
                                                  uint32_t bar_cluster) {
  if (mn) {
    tma_load_2d_pair(dst, map, bar_cluster, side0, k0);
    tma_load_2d_pair(dst + 8192, map, bar_cluster, side0 + 64, k0);
  } else {
    tma_load_2d_pair(dst, map, bar_cluster, k0, side0);
  }
}

// Descriptor of the kk-th 16 of k: K-major rows of 128 B, 32 B per slice; side-major k-rows of
// 128 B, 2 KB per slice, the next 64 of the side 8 KB on.
__device__ __forceinline__ uint64_t slice_desc(uint32_t addr, int mn, int kk) {
  return mn ? smem_desc_sw128(addr + kk * 2048u, 8192u, 1024u) : smem_desc_sw128(addr + kk * 32u, 16u, 1024u);
}

__device__ __forceinline__ void settle_wait(uint64_t* bar, uint32_t parity, unsigned long long budget) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < budget) {
  }
}

// Lane 0 waits, the warp learns the outcome.
__device__ __forceinline__ bool warp_waits(uint64_t* bar, uint32_t parity, const Watchdog& w, int site) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, w, site) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

template <class L>
__global__ void __launch_bounds__(L::kThreads, 1) muon_product_pair_kernel(const __grid_constant__ ProductParams p) {
  constexpr int S = L::S, TN = L::TN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);  // used in the leader CTA
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;  // used in the leader CTA: every epilogue warp of the pair arrives
  uint64_t* tdown = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tdown + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* peer_issued = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);  // leader CTA
  __shared__ uint64_t pdone;  // leader CTA: the peer's producer has finished

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int worker = blockIdx.x >> 1;
  const int workers = p.sum_from >> 1;
  const int units = p.tiles_m * p.tiles_n * p.splits;
  if (static_cast<int>(blockIdx.x) >= p.sum_from) return run_column_sums(p, smem);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * L::NEPI);
    }
    mbar_init(tdown, 1);
    mbar_init(&pdone, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.map_a[0]);
    tma_prefetch_desc(&p.map_b[0]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, L::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Watchdog wd{abort_flag, g_layers_status, p.timeout_ns};
  // waits on the way out, for copies and MMAs in flight, end by themselves
  const unsigned long long tb = p.timeout_ns > 2000000000ull ? p.timeout_ns : 2000000000ull;
  griddep_wait();  // everything read or written below may belong to the launch before
  griddep_launch_dependents();

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer (each CTA)
    // Load i of a CTA goes to stage i % S in phase i / S; the leader arms each phase for the
    // whole pair's bytes.
    if (lane == 0) {
      const uint32_t full0 = map_to_rank(smem_u32(full), 0);
      int s = 0;
      uint32_t ph = 0, issued = 0;
      bool ok = true;
      for (int t = worker; ok && t < units; t += workers) {
        const Unit u = decode_unit(p, t);
        const int a0 = L::TM * u.i + 128 * rank;
        const int b0 = TN * u.j + 128 * rank;
        for (int pb = u.kb0; ok && pb < u.kb1; pb += p.piece) {
          const int pe = pb + p.piece < u.kb1 ? pb + p.piece : u.kb1;
          for (int g = 0; ok && g < p.nseg; ++g) {
            const CUtensorMap* ma = &p.map_a[p.seg_a[g]];
            const CUtensorMap* mb = &p.map_b[p.seg_b[g]];
            for (int kb = pb; kb < pe; ++kb) {
              if (!mbar_wait(&empty[s], ph ^ 1u, wd, kSiteLoad)) {
                ok = false;
                break;
              }
              uint8_t* sa = smem + s * L::kStageBytes;
              if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * L::kStageBytes);
              const uint32_t fb = full0 + 8u * static_cast<uint32_t>(s);
              const int k0 = kb * L::BK;
              load_pair_operand(sa, ma, p.a_mn, a0, k0, fb);
              load_pair_operand(sa + L::kABytes, mb, p.b_mn, b0, k0, fb);
              ++issued;
              if (++s == S) {
                s = 0;
                ph ^= 1u;
              }
            }
          }
        }
      }
      // Before the CTAs part, every copy in flight has landed.  A load below
      // min(own, peer's) - S has: both producers waited for its stage to be consumed again.
      // After a timeout the two may have stopped at different counts: the peer reports its
      // own, and the leader completes or arms the difference, phase by phase in order.
      if (rank != 0) {
        st_cluster_u32(map_to_rank(smem_u32(const_cast<uint32_t*>(peer_issued)), 0), issued);
        mbar_arrive_cluster(map_to_rank(smem_u32(&pdone), 0));
      } else {
        const uint32_t own = issued;
        uint32_t peer = own;
        const uint64_t t0 = global_timer_ns();
        bool known;
        while (!(known = mbar_try_wait_cluster(&pdone, 0)) && global_timer_ns() - t0 < tb) {
        }
        if (known) peer = *peer_issued;
        const uint32_t both = own < peer ? own : peer, most = own > peer ? own : peer;
        for (uint32_t i = both >= static_cast<uint32_t>(S) ? both - S : 0u; i < most; ++i) {
          uint64_t* bar = &full[i % S];
          if (i >= own)
            mbar_arrive_expect_tx(bar, L::kStageBytes);
          else if (i >= peer)
            mbar_complete_tx(bar, L::kStageBytes);
          settle_wait(bar, (i / S) & 1u, tb);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (leader CTA)
    if (lane == 0) {
      if (rank == 0) {
        const uint32_t idesc = idesc_bf16_f32(L::TM, TN, p.a_mn, p.b_mn);
        int s = 0, acc = 0;
        uint32_t ph = 0, aph = 0;
        bool ok = true;
        for (int t = worker; ok && t < units; t += workers) {
          const Unit u = decode_unit(p, t);
          for (int pb = u.kb0; ok && pb < u.kb1; pb += p.piece) {
            const int pe = pb + p.piece < u.kb1 ? pb + p.piece : u.kb1;
            const int blocks = (pe - pb) * p.nseg;
            if (!mbar_wait(&tempty[acc], aph ^ 1u, wd, kSiteAccFree)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t dtm = tmem_base + static_cast<uint32_t>(acc * TN);
            for (int kb = 0; kb < blocks; ++kb) {
              if (!mbar_wait(&full[s], ph, wd, kSiteStage)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t sa = smem_u32(smem + s * L::kStageBytes);
              const uint32_t sb = sa + L::kABytes;
#pragma unroll
              for (int kk = 0; kk < L::BK / 16; ++kk)
                umma_bf16_pair(dtm, slice_desc(sa, p.a_mn, kk), slice_desc(sb, p.b_mn, kk), idesc,
                               (kb | kk) != 0 ? 1u : 0u);
              umma_commit_pair(&empty[s], 0x3);
              if (++s == S) {
                s = 0;
                ph ^= 1u;
              }
            }
            if (!ok) break;
            umma_commit_pair(&tfull[acc], 0x3);
            if (++acc == 2) {
              acc = 0;
              aph ^= 1u;
            }
          }
        }
        // Every MMA has finished before either CTA releases tensor memory or leaves.
        umma_commit_pair(tdown, 0x3);
      }
      settle_wait(tdown, 0, tb);
    }
  } else {
    // ---------------------------------------------------------------- epilogue (each CTA)
    const int ew = warp - 2;
    const int q4 = warp & 3;  // tensor memory lanes 32 q4 .. 32 q4 + 31 belong to this warp
    const int h = ew >> 2;    // which NCW of the tile's columns
    const int r = q4 * 32 + lane;
    const uint32_t tempty0 = map_to_rank(smem_u32(tempty), 0);
    int acc = 0;
    uint32_t aph = 0;
    bool ok = true;
    for (int t = worker; ok && t < units; t += workers) {
      const Unit u = decode_unit(p, t);
      const int64_t row = static_cast<int64_t>(L::TM) * u.i + 128 * rank + r;
      const int64_t col = static_cast<int64_t>(TN) * u.j + h * L::NCW;
      float* part = p.partial == nullptr ? nullptr : p.partial + u.split * p.split_stride;
      EpiRow<32> at;
      // the common epilogue, where all of the warp's rows and columns exist
      const bool plain =
          L::kPlain && p.e.plain && part == nullptr && row - lane + 32 <= p.e.rows && col + L::NCW <= p.e.cols;
      if constexpr (!L::FLIP) {  // the epilogue's inputs move while the tile's products run
        if (plain) at.start(p.e, row, col);
        if (part == nullptr && t + workers < units) {  // the next tile's inputs, a tile ahead
          const Unit nx = decode_unit(p, t + workers);
          const int64_t nrow = static_cast<int64_t>(L::TM) * nx.i + 128 * rank + r;
          const int64_t ncol = static_cast<int64_t>(TN) * nx.j + h * L::NCW;
          if (nrow < p.e.rows && ncol < p.e.cols) {
            const int width = p.e.cols - ncol < L::NCW ? static_cast<int>(p.e.cols - ncol) : L::NCW;
            prefetch_row(p.e.slope, nrow, ncol, width);
            prefetch_row(p.e.add, nrow, ncol, width);
          }
        }
        if constexpr (L::kPlain) {
          if (plain) at.fetch(0);
        }
      }
      uint32_t tacc = 0;
      auto await = [&]() {
        __syncwarp();
        ok = warp_waits(&tfull[acc], aph, wd, kSiteAccReady);
        tc_fence_after();
        tacc = tmem_base + static_cast<uint32_t>(acc * TN + h * L::NCW) + (static_cast<uint32_t>(q4 * 32) << 16);
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + 8u * static_cast<uint32_t>(acc));
        if (++acc == 2) {
          acc = 0;
          aph ^= 1u;
        }
      };
      await();
      if constexpr (L::SUM) {
        if (u.kb1 - u.kb0 > p.piece) {
          // Pieces are added in registers; the whole sum goes back to the last piece's
          // columns, so that the code below finds it where a single piece would be.
          float sum[L::NCW];
#pragma unroll
          for (int j = 0; j < L::NCW; ++j) sum[j] = 0.f;
          for (int pb = u.kb0; ok;) {
#pragma unroll
            for (int c = 0; c < L::NCW; c += 16) {
              uint32_t v[16];
              tmem_load_row<16>(tacc + c, v);
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[c + j] += __uint_as_float(v[j]);
            }
            pb += p.piece;
            if (pb >= u.kb1) break;
            release();
            await();
          }
          if (ok) {
#pragma unroll
            for (int c = 0; c < L::NCW; c += 16) tmem_store_row16(tacc + c, &sum[c]);
            tmem_wait_st();
          }
        }
      }
      if (!ok) break;
      if constexpr (L::kPlain) {
        if (plain) {
#pragma unroll 1
          for (int c = 0; c < L::NCW; c += 32) {
            uint32_t v[32];
            tmem_load_row<32>(tacc + c, v);
            if (c + 32 == L::NCW) release();  // the last read
            F2 x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = pair(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            at.finish(p.e, col + c, c, c + 32 < L::NCW, x);
          }
          continue;
        }
      }
      // Everything else, in short steps: the code of a step has every choice in it, and a
      // small product is over before a long one is in the instruction cache.
      constexpr int GC = L::GC;
#pragma unroll 1
      for (int c = 0; c < L::NCW; c += GC) {
        uint32_t v[GC];
        __syncwarp();  // lanes may have parted over edges
        tmem_load_row<GC>(tacc + c, v);
        if (c + GC == L::NCW) release();  // the last read
        if constexpr (!L::FLIP) {  // (a split reduction never runs flipped: its partial sums are aligned)
          if (part != nullptr) {
            float x[GC];
#pragma unroll
            for (int j = 0; j < GC; ++j) x[j] = __uint_as_float(v[j]);
            const EpiView out{part, p.ld_partial, 0, 2};
            if (row < p.e.rows && col + c < p.ld_partial) store_segment<GC>(out, row * out.ld + col + c, GC, x);
            continue;
          }
        }
        F2 x[GC / 2];
#pragma unroll
        for (int j = 0; j < GC / 2; ++j) x[j] = pair(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
        if constexpr (L::FLIP)
          finish_column<GC>(p.e, col + c, row, x);
        else
          finish_segment<GC>(p.e, row, col + c, x);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing arrives on, or lands in, either CTA after this
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, L::kTmemCols);
  }
}

// ------------------------------------------------------------------ small products
//
// One tile of 128 x TN per cluster of 1, 2, 4 or 8 CTAs that split the reduction.  A small
// product is bound by latency: by the few SMs its tiles would occupy (an SM takes in about
// 64 bytes a cycle from L2: 12 k-blocks of 128 x 128 tiles take 5 us on one CTA), and by the
// instructions of its epilogue.  The cluster divides both: each CTA sums its k-blocks in
// tensor memory, leaves its tile in its own shared memory (the ring's, whose loads have all
// been consumed), and finishes a share of the columns, adding the others' sums through
// distributed shared memory in the order of the ranks.  No second launch, no workspace.
// Two products of one call that both are small share a launch, each with its own number of
// CTAs per tile.
//
// Measured (captured calls, us): 1 x 1024 x 4096 6.5, 1 x 4096 x 4096 13 (2.6 TB/s of weights),
// 16 x 4096 x 14336 30 (3.9 TB/s), 512 x 1024 x 4096 12.4; both gradients of 256 x 768 x 768 with
// fp32 weights 12.3, with the layout of the terms.
template <int TN_, bool FLIP_>
struct Small {
  static constexpr int TN = TN_;
  static constexpr bool FLIP = FLIP_;
  static constexpr int BK = kProductBK;
  static constexpr int kABytes = 128 * BK * 2;
  static constexpr int kBBytes = TN * BK * 2;
  static constexpr int S = 14;  // loads of one operand term that the ring holds
  static constexpr int kBarOff = S * kABytes;
  static constexpr int kPairs = kBarOff / (kABytes + kBBytes) < S ? kBarOff / (kABytes + kBBytes) : S;
  static constexpr int kSmemBytes = kBarOff + 512 + 1024;
  static constexpr int NEPI = 8;
  static constexpr int kThreads = 64 + 32 * NEPI;
  static constexpr int NCW = TN / 2;  // accumulator columns per epilogue thread
  static constexpr int GC = TN < 128 ? 8 : 16;  // finished at a time
  static constexpr int kTmemCols = 4 * TN;
  static_assert(kSmemBytes <= 232448, "shared memory of a block");
  static_assert(128 * TN * 4 <= kBarOff, "the tile fits the ring");
  static_assert((2 * S + 5) * 8 + 16 <= 512, "barrier area");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// As load_pair_operand, ROWS of the side, completing on this CTA's barrier.
template <int ROWS>
__device__ __forceinline__ void load_operand(uint8_t* dst, const CUtensorMap* map, int mn, int side0, int k0,
                                             uint64_t* bar) {
  if (mn) {
#pragma unroll
    for (int b = 0; b < ROWS / 64; ++b) tma_load_2d(dst + b * 8192, map, bar, side0 + 64 * b, k0);
  } else {
    tma_load_2d(dst, map, bar, k0, side0);
  }
}

// A staged tile: 4 columns of a row in 16 bytes, the rows of a column group side by side, so
// that a warp's 32 rows are conflict-free to write and to read.
__device__ __forceinline__ uint32_t staged_at(int row, int col) {
  return static_cast<uint32_t>(((col >> 2) * 128 + row) * 16);
}

// The walk of a k-block: the operand terms in the order they are loaded (side 0: the tile's
// rows; term 0 leading, 1 middle, 2 low), and the term products with the loads they use, wait
// for and are the last to use.  Each term is loaded once a k-block (a walk per term product
// loads two per product, 12 instead of 6), and the order frees them early.  The leading terms'
// product has an accumulator of its own: beside it the others are corrections, 2^-8 and less
// of its size, whose own truncation is nothing.  Gradients of 515 x 770 x 1030 in fp32: 34.9 us,
// 47.5 with a walk per term product; of 256 x 768 x 768 with fp32 weights 14.2 and 23.1.  (With
// the tables read at run time, not unrolled, the issuing thread was the bound: 68 and 17.)
struct WalkStep {
  int a, b, need, correction, frees;  // frees: bit per load
};
template <int WALK>
struct Walk;
template <>
struct Walk<kWalkOne> {
  static constexpr int kLoads = 2, kSteps = 1, kRing = 0;  // a place holds both loads: Small::kPairs of them
  int side[2] = {0, 1}, term[2] = {0, 0};
  WalkStep step[1] = {{0, 1, 1, 0, 1}};
};
template <>
struct Walk<kWalkRows> {
  static constexpr int kLoads = 4, kSteps = 3, kRing = 12;
  int side[4] = {0, 1, 0, 0}, term[4] = {2, 0, 1, 0};
  WalkStep step[3] = {{0, 1, 2, 1, 1}, {2, 1, 3, 1, 4}, {3, 1, 4, 0, 2 + 8}};
};
template <>
struct Walk<kWalkCols> {
  static constexpr int kLoads = 4, kSteps = 3, kRing = 12;
  int side[4] = {1, 0, 1, 1}, term[4] = {2, 0, 1, 0};
  WalkStep step[3] = {{1, 0, 2, 1, 1}, {1, 2, 3, 1, 4}, {1, 3, 4, 0, 2 + 8}};
};
template <>
struct Walk<kWalkBoth> {
  static constexpr int kLoads = 6, kSteps = 6, kRing = 12;
  int side[6] = {0, 1, 0, 1, 0, 1}, term[6] = {2, 0, 1, 1, 0, 2};
  // l h, m h, m m, h h, h m, h l
  WalkStep step[6] = {{0, 1, 2, 1, 1}, {2, 1, 3, 1, 0}, {2, 3, 4, 1, 4},
                                      {4, 1, 5, 0, 2}, {4, 3, 5, 1, 8}, {4, 5, 6, 1, 16 + 32}};
};

struct SmallBars {
  uint64_t *full, *empty, *tfull, *tempty;
};

// The producer's loads of k-blocks [kb0, kb1); `budget` bounds the last wait, for the copies
// still in flight.
template <class L, class W>
__device__ __forceinline__ void small_loads(const ProductParams& p, uint8_t* smem, const SmallBars& bar,
                                            const Watchdog& wd, int i, int j, int kb0, int kb1,
                                            unsigned long long budget) {
  constexpr W w{};
  constexpr bool joint = W::kSteps == 1;
  constexpr int kPlaces = joint ? L::kPairs : W::kRing, kPlace = joint ? L::kABytes + L::kBBytes : L::kABytes;
  int s = 0;
  uint32_t ph = 0, issued = 0;
  bool ok = true;
  for (int kb = kb0; ok && kb < kb1; ++kb) {
#pragma unroll
    for (int l = 0; l < W::kLoads; ++l) {
      uint8_t* dst = smem + s * kPlace + l * L::kABytes;
      uint64_t* full = &bar.full[joint ? s : s + l];
      if (!joint || l == 0) {
        ok = mbar_wait(&bar.empty[s + l], ph ^ 1u, wd, kSiteLoad);
        if (!ok) break;
        mbar_arrive_expect_tx(full, joint ? L::kABytes + L::kBBytes : w.side[l] == 0 ? L::kABytes : L::kBBytes);
      }
      if (w.side[l] == 0)
        load_operand<128>(dst, &p.map_a[w.term[l]], p.a_mn, 128 * i, kb * L::BK, full);
      else
        load_operand<L::TN>(dst, &p.map_b[w.term[l]], p.b_mn, L::TN * j, kb * L::BK, full);
      if (!joint || l == 0) ++issued;
    }
    if ((s += joint ? 1 : W::kLoads) == kPlaces) {
      s = 0;
      ph ^= 1u;
    }
  }
  // every copy in flight has landed before anything else is put there
  for (uint32_t l = issued >= static_cast<uint32_t>(kPlaces) ? issued - kPlaces : 0u; l < issued; ++l)
    settle_wait(&bar.full[l % kPlaces], (l / kPlaces) & 1u, budget);
}

// The MMA issuer's half.
template <class L, class W>
__device__ __forceinline__ void small_products(const ProductParams& p, uint8_t* smem, const SmallBars& bar,
                                               const Watchdog& wd, uint32_t tmem_base, int kb0, int kb1) {
  constexpr W w{};
  constexpr int TN = L::TN;
  constexpr bool joint = W::kSteps == 1;
  constexpr int kPlaces = joint ? L::kPairs : W::kRing, kPlace = joint ? L::kABytes + L::kBBytes : L::kABytes;
  const uint32_t idesc = idesc_bf16_f32(128, TN, p.a_mn, p.b_mn);
  int s = 0, acc = 0;
  uint32_t ph = 0, aph = 0;
  for (int pb = kb0; pb < kb1; pb += p.piece) {
    const int pe = pb + p.piece < kb1 ? pb + p.piece : kb1;
    if (!mbar_wait(&bar.tempty[acc], aph ^ 1u, wd, kSiteAccFree)) return;
    tc_fence_after();
    const uint32_t dtm = tmem_base + static_cast<uint32_t>(2 * acc * TN);
    for (int kb = pb; kb < pe; ++kb) {
      const uint32_t base = smem_u32(smem + s * kPlace);
      int there = 0, begun = 0;
#pragma unroll
      for (int t = 0; t < W::kSteps; ++t) {
        const WalkStep step = w.step[t];
#pragma unroll
        for (int l = 0; l < W::kLoads; ++l)
          if (l >= there && l < step.need)
            if (!mbar_wait(&bar.full[s + l], ph, wd, kSiteStage)) return;
        there = step.need;
        tc_fence_after();
        const uint32_t sa = base + step.a * L::kABytes, sb = base + step.b * L::kABytes;
        const uint32_t d = dtm + static_cast<uint32_t>(step.correction * TN);
        const bool later = begun >> step.correction & 1;
#pragma unroll
        for (int kk = 0; kk < L::BK / 16; ++kk)
          umma_bf16(d, slice_desc(sa, p.a_mn, kk), slice_desc(sb, p.b_mn, kk), idesc,
                    kk != 0 || later || kb != pb ? 1u : 0u);
        begun |= 1 << step.correction;
#pragma unroll
        for (int l = 0; l < W::kLoads; ++l)
          if (step.frees >> l & 1) umma_commit(&bar.empty[s + l]);
      }
      if ((s += joint ? 1 : W::kLoads) == kPlaces) {
        s = 0;
        ph ^= 1u;
      }
    }
    umma_commit(&bar.tfull[acc]);
    if (++acc == 2) {
      acc = 0;
      aph ^= 1u;
    }
  }
}

template <class L>
__global__ void __launch_bounds__(L::kThreads, 1) muon_product_small_kernel(const __grid_constant__ ProductGroup g) {
  constexpr int S = L::S, TN = L::TN, GC = L::GC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* tdown = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tdown + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (static_cast<int>(blockIdx.x) >= g.p[0].sum_from) return run_column_sums(g.p[0], smem);
  const int second = static_cast<int>(blockIdx.x) >= g.first_blocks;
  const ProductParams& p = g.p[second];
  const int block = static_cast<int>(blockIdx.x) - (second ? g.first_blocks : 0);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // the p.splits CTAs of a tile are neighbours in the cluster, from rank `first` on
  const int in_cluster = static_cast<int>(cluster_rank());
  const int rank = in_cluster & (p.splits - 1), first = in_cluster - rank;
  const int tile = block / p.splits;
  const int j = tile / p.tiles_m, i = tile - j * p.tiles_m;
  const bool live = j < p.tiles_n;  // the last cluster may have CTAs left over
  // k-blocks of this CTA; of `parts` CTAs that have any (the others help with the epilogue)
  const int per = (p.nk + p.splits - 1) / p.splits, parts = (p.nk + per - 1) / per;
  const int kb0 = live ? min(per * rank, p.nk) : 0, kb1 = live ? min(kb0 + per, p.nk) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], L::NEPI);
    }
    mbar_init(tdown, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.map_a[0]);
    tma_prefetch_desc(&p.map_b[0]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Watchdog wd{abort_flag, g_layers_status, p.timeout_ns};
  const SmallBars bar{full, empty, tfull, tempty};
  const unsigned long long tb = p.timeout_ns > 2000000000ull ? p.timeout_ns : 2000000000ull;
  griddep_wait();  // everything read or written below may belong to the launch before
  griddep_launch_dependents();

  // The share of the tile that this thread finishes: row r of the tile, 16 columns at a time.
  const int e = static_cast<int>(threadIdx.x) - 64;
  const int r = e & 127, q0 = rank + p.splits * (e >> 7);
  const int64_t row = static_cast<int64_t>(128) * i + r;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      switch (p.walk) {
        case kWalkOne: small_loads<L, Walk<kWalkOne>>(p, smem, bar, wd, i, j, kb0, kb1, tb); break;
        case kWalkRows: small_loads<L, Walk<kWalkRows>>(p, smem, bar, wd, i, j, kb0, kb1, tb); break;
        case kWalkCols: small_loads<L, Walk<kWalkCols>>(p, smem, bar, wd, i, j, kb0, kb1, tb); break;
        default: small_loads<L, Walk<kWalkBoth>>(p, smem, bar, wd, i, j, kb0, kb1, tb);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      switch (p.walk) {
        case kWalkOne: small_products<L, Walk<kWalkOne>>(p, smem, bar, wd, tmem_base, kb0, kb1); break;
        case kWalkRows: small_products<L, Walk<kWalkRows>>(p, smem, bar, wd, tmem_base, kb0, kb1); break;
        case kWalkCols: small_products<L, Walk<kWalkCols>>(p, smem, bar, wd, tmem_base, kb0, kb1); break;
        default: small_products<L, Walk<kWalkBoth>>(p, smem, bar, wd, tmem_base, kb0, kb1);
      }
      umma_commit(tdown);
      settle_wait(tdown, 0, tb);
    }
  } else {
    // ---------------------------------------------------------------- sums, and the tile's staging
    const int q4 = warp & 3;          // tensor memory lanes 32 q4 .. 32 q4 + 31 belong to this warp
    const int c0 = ((warp - 2) >> 2) * L::NCW;
    const int lane_row = q4 * 32 + lane;
    if constexpr (!L::FLIP) {  // the epilogue's inputs move while the products run
      const int64_t col = static_cast<int64_t>(TN) * j + GC * q0;
      if (q0 < TN / GC && row < p.e.rows && col < p.e.cols) {
        prefetch_row(p.e.slope, row, col, 1);
        prefetch_row(p.e.add, row, col, 1);
      }
    }
    float sum[L::NCW];
#pragma unroll
    for (int c = 0; c < L::NCW; ++c) sum[c] = 0.f;
    int acc = 0;
    uint32_t aph = 0;
    bool ok = true;
    for (int pb = kb0; pb < kb1; pb += p.piece) {
      ok = warp_waits(&tfull[acc], aph, wd, kSiteAccReady);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tacc =
          tmem_base + static_cast<uint32_t>(2 * acc * TN + c0) + (static_cast<uint32_t>(q4 * 32) << 16);
      if (p.nseg > 1) {
#pragma unroll
        for (int c = 0; c < L::NCW; c += 16) {
          uint32_t v[16];
          tmem_load_row<16>(tacc + TN + c, v);
#pragma unroll
          for (int k = 0; k < 16; ++k) sum[c + k] += __uint_as_float(v[k]);
        }
      }
#pragma unroll
      for (int c = 0; c < L::NCW; c += 16) {
        uint32_t v[16];
        tmem_load_row<16>(tacc + c, v);
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[c + k] += __uint_as_float(v[k]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      if (++acc == 2) {
        acc = 0;
        aph ^= 1u;
      }
    }
    if (ok && kb0 < kb1) {  // the last accumulator is complete: every stage of the ring has been consumed
#pragma unroll
      for (int c = 0; c < L::NCW; c += 4)
        *reinterpret_cast<float4*>(smem + staged_at(lane_row, c0 + c)) =
            make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
    }
  }

  __syncwarp();
  cluster_sync();  // every CTA's tile is staged
  if (warp >= 2 && live && !*abort_flag) {
#pragma unroll 1
    for (int q = q0; q < TN / GC; q += 2 * p.splits) {
      F2 v[GC / 2];
#pragma unroll
      for (int k = 0; k < GC / 2; ++k) v[k] = 0ull;  // zeros
#pragma unroll 1
      for (int c = 0; c < parts; c += 2) {  // two CTAs' sums on their way at once
        float4 a[2][GC / 4];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (c + k < parts) {
            const uint32_t base = map_to_rank(smem_u32(smem), static_cast<uint32_t>(first + c + k)) + staged_at(r, GC * q);
#pragma unroll
            for (int l = 0; l < GC / 4; ++l) a[k][l] = ld_cluster_f4(base + l * 2048u);
          }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (c + k < parts) {
#pragma unroll
            for (int l = 0; l < GC / 4; ++l) {
              v[2 * l] = add2(v[2 * l], pair(a[k][l].x, a[k][l].y));
              v[2 * l + 1] = add2(v[2 * l + 1], pair(a[k][l].z, a[k][l].w));
            }
          }
      }
      const int64_t col = static_cast<int64_t>(TN) * j + GC * q;
      if constexpr (L::FLIP)  // row: a column of the output; col: the first of 16 of its rows
        finish_column<GC>(p.e, col, row, v);
      else
        finish_segment<GC>(p.e, row, col, v);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nobody reads this CTA's tile any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
}

// ------------------------------------------------------------------ before and after the products

// Calls f(row, group of 8 columns) over the sweep, for block `b` of it.
template <class F>
__device__ __forceinline__ void run_sweep(const Sweep& s, int b, F&& f) {
  const int along = 1 << s.shift, deep = 256 >> s.shift;
  const int rb = b / s.col_blocks, cb = b - rb * s.col_blocks;
  const int g0 = (cb << s.shift) + (threadIdx.x & (along - 1));
  for (int64_t r = static_cast<int64_t>(rb) * deep + (threadIdx.x >> s.shift); r < s.rows;
       r += static_cast<int64_t>(s.row_blocks) * deep)
    for (int g = g0; g < s.groups; g += s.col_blocks << s.shift) f(r, g);
}

// x = h + m + l: each term takes the leading 8 bits of what is left, truncated, so the three
// hold the 24 bits of an fp32 value exactly and none overflows (only terms below 2^-133 are
// lost).  A bf16 source is copied to rows that TMA can read.
// An infinity in one operand meets every term of the other: inf * 0 of an absent m or l would
// make the sum NaN.  So a term that nothing is left for is 2^-60 of the value, which no finite
// sum shows, and an infinity goes into all three: then every term product has the sign of the
// whole one.
// Bound by HBM for large operands and by the launch for small ones: 4 bytes read and 6 written
// an element, about 2 us of the 12.3 of both gradients of 256 x 768 x 768.  Two rows at a time,
// and one test for eight elements, made x W^T of 4096 x 1024 x 1024 in fp32 16% and both
// gradients of 1000 x 1000 x 1000 13% quicker (50 and 39 us).
__device__ __forceinline__ void pack_terms(const PackTask& p, int64_t at, float (&x)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  if (top > 0x7F800000u) {  // a NaN stays one without its low half
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (isnan(x[j])) x[j] = __uint_as_float(0x7FC00000u);
  }
  float least[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) least[j] = fabsf(x[j]) * 0x1p-60f;
  for (int t = 0;;) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __byte_perm(__float_as_uint(x[2 * j]), __float_as_uint(x[2 * j + 1]), 0x7632);
    *reinterpret_cast<uint4*>(p.dst + t * p.term_stride + at) = make_uint4(w[0], w[1], w[2], w[3]);
    if (++t == p.terms) break;
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // (an infinity leaves NaN, of which and infinity the larger is infinity)
      const float h = __uint_as_float(__float_as_uint(x[j]) & 0xFFFF0000u);
      x[j] = copysignf(fmaxf(fabsf(x[j] - h), least[j]), h);
    }
  }
}

// Two rows a thread and step, so that two loads are on their way.
__device__ __forceinline__ void pack_rows(const PackTask& p, int b) {
  const Sweep& s = p.sweep;
  const int along = 1 << s.shift, deep = 256 >> s.shift;
  const int rb = b / s.col_blocks, cb = b - rb * s.col_blocks;
  const int g0 = (cb << s.shift) + (threadIdx.x & (along - 1));
  const int64_t step = static_cast<int64_t>(s.row_blocks) * deep;
  const bool wide = !p.src.bf16 && p.src.vec > 0;
  for (int64_t r = static_cast<int64_t>(rb) * deep + (threadIdx.x >> s.shift); r < s.rows; r += 2 * step) {
    const bool two = r + step < s.rows;
    for (int g = g0; g < s.groups; g += s.col_blocks << s.shift) {
      const int c = g * 8;
      float x[8], y[8];
      if (wide && c + 8 <= p.cols) {
        const float* at = static_cast<const float*>(p.src.p) + r * p.src.ld + c;
        const float* next = two ? at + step * p.src.ld : at;
        const float4 x0 = *reinterpret_cast<const float4*>(at), x1 = *reinterpret_cast<const float4*>(at + 4);
        const float4 y0 = *reinterpret_cast<const float4*>(next), y1 = *reinterpret_cast<const float4*>(next + 4);
        x[0] = x0.x, x[1] = x0.y, x[2] = x0.z, x[3] = x0.w, x[4] = x1.x, x[5] = x1.y, x[6] = x1.z, x[7] = x1.w;
        y[0] = y0.x, y[1] = y0.y, y[2] = y0.z, y[3] = y0.w, y[4] = y1.x, y[5] = y1.y, y[6] = y1.z, y[7] = y1.w;
      } else {
        load_segment<8>(p.src, r * p.src.ld + c, p.cols - c, x);
        if (two) load_segment<8>(p.src, (r + step) * p.src.ld + c, p.cols - c, y);
      }
      pack_terms(p, r * p.ld_dst + c, x);
      if (two) pack_terms(p, (r + step) * p.ld_dst + c, y);
    }
  }
}

__global__ void __launch_bounds__(256) muon_prepare_kernel(const __grid_constant__ PrepareParams p) {
  __shared__ float red[32][64];
  griddep_wait();
  griddep_launch_dependents();
  int i = 0;
  while (static_cast<int>(blockIdx.x) >= p.begin[i + 1]) ++i;
  const int b = static_cast<int>(blockIdx.x) - p.begin[i];
  if (i < p.packs) {
    pack_rows(p.pack[i], b);
  } else {
    column_sums<8>(p.sum, b, red);
  }
}

// Adds the partial sums of a split reduction in the order of the splits, then the epilogue.
__device__ __forceinline__ void join_group(const JoinTask& p, int64_t m, int g) {
  const int64_t n = static_cast<int64_t>(g) * 8;
  const float* src = p.partial + m * p.ld_partial + n;
  F2 v[4] = {0ull, 0ull, 0ull, 0ull};  // zeros
#pragma unroll 8
  for (int s = 0; s < p.splits; ++s) {
    const float4 a = *reinterpret_cast<const float4*>(src + s * p.split_stride);
    const float4 b = *reinterpret_cast<const float4*>(src + s * p.split_stride + 4);
    v[0] = add2(v[0], pair(a.x, a.y));
    v[1] = add2(v[1], pair(a.z, a.w));
    v[2] = add2(v[2], pair(b.x, b.y));
    v[3] = add2(v[3], pair(b.z, b.w));
  }
  finish_segment<8>(p.e, m, n, v);
}

// The slices of the column sums: 32 columns per block, 8 warps over the slices.
__device__ __forceinline__ void join_column_sums(const ColumnSumTask& p, int b, float (*red)[32]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = b * 32 + lane;
  float t = 0.f;
  if (c < p.cols) {
#pragma unroll 8
    for (int s = w; s < p.slices; s += 8) t += p.partial[static_cast<int64_t>(s) * p.cols + c];
  }
  red[w][lane] = t;
  __syncthreads();
  if (w == 0 && c < p.cols) {
    for (int k = 1; k < 8; ++k) t += red[k][lane];
    p.out[c] = p.accumulate ? p.out[c] + t : t;
  }
}

__global__ void __launch_bounds__(256) muon_finish_kernel(const __grid_constant__ FinishParams p) {
  __shared__ float red[8][32];
  griddep_wait();
  griddep_launch_dependents();
  int i = 0;
  while (static_cast<int>(blockIdx.x) >= p.begin[i + 1]) ++i;
  const int b = static_cast<int>(blockIdx.x) - p.begin[i];
  if (i < p.joins) {
    const JoinTask& t = p.join[i];
    run_sweep(t.sweep, b, [&](int64_t r, int g) { join_group(t, r, g); });
  } else {
    join_column_sums(p.sum, b, red);
  }
}

// ------------------------------------------------------------------ launches

template <class L>
static cudaError_t launch_pair(ProductParams& p, int sms, cudaStream_t stream) {
  auto* kernel = muon_product_pair_kernel<L>;
  static thread_local int configured_device = -1;
  static thread_local int resident = 0;  // pairs that can run at once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sms / 2 * 2, 1, 1);
    cfg.blockDim = dim3(L::kThreads, 1, 1);
    cfg.dynamicSmemBytes = L::kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return e;
    resident = clusters > 0 ? clusters : 1;
    configured_device = dev;
  }
  p.sum_from = 2 * std::min(p.tiles_m * p.tiles_n * p.splits, resident);
  return launch_dependent(kernel, p, dim3(static_cast<unsigned>(p.sum_from + p.sum_blocks)), L::kThreads, stream,
                          L::kSmemBytes, 2);
}

template <class L>
static cudaError_t launch_small(ProductGroup& g, int blocks, cudaStream_t stream) {
  auto* kernel = muon_product_small_kernel<L>;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  g.p[0].sum_from = blocks;
  return launch_dependent(kernel, g, dim3(static_cast<unsigned>(blocks + g.p[0].sum_blocks)), L::kThreads, stream,
                          L::kSmemBytes, g.cluster);
}

cudaError_t launch_product_pair(int tile, ProductParams& p, int sms, cudaStream_t stream) {
  switch (tile) {
    case kPair256: return launch_pair<Pair<false, false>>(p, sms, stream);
    case kPair256Sum: return launch_pair<Pair<true, false>>(p, sms, stream);
    case kFlipPair256: return launch_pair<Pair<false, true>>(p, sms, stream);
    case kFlipPair256Sum: return launch_pair<Pair<true, true>>(p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_product_small(int tile, ProductGroup& g, int blocks, cudaStream_t stream) {
  switch (tile) {
    case kOne128: return launch_small<Small<128, false>>(g, blocks, stream);
    case kFlip128: return launch_small<Small<128, true>>(g, blocks, stream);
    case kFlip32: return launch_small<Small<32, true>>(g, blocks, stream);
    case kFlip64: return launch_small<Small<64, true>>(g, blocks, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_prepare(const PrepareParams& p, cudaStream_t stream) {
  return launch_dependent(muon_prepare_kernel, p, dim3(static_cast<unsigned>(p.begin[p.packs + 1])), 256, stream);
}

cudaError_t launch_finish(const FinishParams& p, cudaStream_t stream) {
  return launch_dependent(muon_finish_kernel, p, dim3(static_cast<unsigned>(p.begin[p.joins + 1])), 256, stream);
}

}  // namespace muon

extern "C" muon_status_t muon_layers_status(void* stream, int clear, int32_t* device_status, int32_t* where) {
  if (device_status == nullptr) return MUON_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t product[2] = {0, 0}, norm[2] = {0, 0};
  const int32_t zero[2] = {0, 0};
  if (cudaMemcpyFromSymbolAsync(product, muon::g_layers_status, sizeof(product), 0, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      muon::norm_status(norm, false, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return MUON_ERR_CUDA;
  if (clear && (cudaMemcpyToSymbolAsync(muon::g_layers_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s) !=
                    cudaSuccess ||
                muon::norm_status(norm, true, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess))
    return MUON_ERR_CUDA;
  const int32_t* first = product[0] != 0 ? product : norm;
  *device_status = first[0];
  if (where != nullptr) *where = first[1];
  return MUON_OK;
}
