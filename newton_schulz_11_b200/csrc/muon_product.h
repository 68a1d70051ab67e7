// Parameters of the layer products, shared by their host planner and kernels.
//
// A product is D[M x N] = sum_k A(m, k) B(n, k) followed by one epilogue:
//   v = sum + bias[n];  preact[m, n] = v;  v = act(v);  v *= act'(slope[m, n]);  v += add[m, n]
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "muon_params.h"

namespace muon {

// One operand of the epilogue.  vec: rows may be accessed 32 (2) or 16 (1) bytes at a time
// from any column that is a multiple of 8; 0: one element at a time.
struct EpiView {
  void* p;
  int64_t ld;
  int32_t bf16;
  int32_t vec;
};

struct Epilogue {
  EpiView bias, preact, slope, add, out;
  int64_t rows, cols;  // of the output
  int32_t act, slope_act;
  int32_t plain;  // all but the bias bf16, in rows of whole 32-byte units; a 32-byte aligned bias
};

constexpr int kTerms = 3;                // bf16 terms of an fp32 operand
constexpr int kMaxSegments = 6;          // products of two such operands that are kept
constexpr int kProductBK = 64;           // reduction depth of a k-block

// How a product is tiled.  The flipped tiles hold the output's columns on their M side (the
// lanes of tensor memory), so that a warp's 32 lanes are neighbouring columns of one row:
// they take few tokens, whose tile would be mostly empty the other way round, and outputs
// whose rows cannot be accessed 16 bytes at a time, element by element in whole lines.
enum ProductTile : int {
  kPair256 = 0,     // 256 x 256 on a CTA pair, the whole reduction in tensor memory
  kPair256Sum,      // the same, the reduction in pieces that are added in registers
  kFlipPair256,
  kFlipPair256Sum,
  kOne128,          // 128 x 128 per cluster, in pieces (the small products, see muon_product.cu)
  kFlip128,
  kFlip32,          // 128 columns x 32 tokens
  kFlip64,          // 128 columns x 64 tokens
};

struct TileShape {
  int m, n;  // rows and columns of the tile
  bool pair, flip, sum;
};

constexpr TileShape kTileShapes[] = {
    {256, 256, true, false, false}, {256, 256, true, false, true}, {256, 256, true, true, false},
    {256, 256, true, true, true},   {128, 128, false, false, true}, {128, 128, false, true, true},
    {128, 32, false, true, true},   {128, 64, false, true, true},
};

// Column sums of a matrix, in `slices` partial sums over its rows.
struct ColumnSumTask {
  EpiView src;
  float* out;
  float* partial;  // [slices][cols]
  int64_t rows;
  int32_t cols, accumulate, slices;
};

// How a small product walks a k-block: by how many terms its operands have.
enum ProductWalk : int { kWalkOne = 0, kWalkRows, kWalkCols, kWalkBoth };

struct ProductParams {
  CUtensorMap map_a[kTerms];  // operand on the tile's M side
  CUtensorMap map_b[kTerms];  // operand on the tile's N side
  Epilogue e;
  int32_t a_mn, b_mn;         // majorness: 0 = contiguous along k, 1 = along the side
  int32_t tiles_m, tiles_n;
  int32_t nk;                 // k-blocks of the whole reduction
  int32_t splits;             // small products: CTAs of a cluster that share a tile (a power of two)
  int32_t kb_per_split;       // large products
  int32_t piece;              // k-blocks per piece
  int32_t nseg;
  uint8_t seg_a[8], seg_b[8]; // large products: the terms of each segment, smallest products first
  int32_t walk;               // small products: ProductWalk
  float* partial;             // large products: [splits][e.rows][ld_partial] for the end, or nullptr
  int64_t ld_partial, split_stride;
  unsigned long long timeout_ns;
  // The bias gradient rides along where the products leave SMs idle: blocks from sum_from on
  // (a whole number of clusters) run its sum_tasks instead.
  ColumnSumTask sum;
  int32_t sum_from, sum_tasks, sum_blocks;
};

// One launch of small products: the second, if any, from block first_blocks on.
struct ProductGroup {
  ProductParams p[2];
  int32_t first_blocks, cluster;
};

// bf16 operand map of a matrix with rows of ld elements: boxes of 64 columns x box_rows rows.
bool encode_operand_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows);

cudaError_t launch_product_pair(int tile, ProductParams& p, int sms, cudaStream_t stream);
cudaError_t launch_product_small(int tile, ProductGroup& g, int blocks, cudaStream_t stream);

// How 256-thread blocks cover rows x groups of 8 columns: 2^shift threads along a row.
struct Sweep {
  int64_t rows;
  int32_t groups, shift;
  int32_t row_blocks, col_blocks;
};

inline Sweep make_sweep(int64_t rows, int64_t groups, int64_t most_blocks) {
  Sweep s{rows, static_cast<int32_t>(groups), 0, 1, 1};
  while (s.shift < 8 && (int64_t(1) << s.shift) < groups) ++s.shift;
  const int64_t rb = (rows + (256 >> s.shift) - 1) / (256 >> s.shift);
  s.row_blocks = static_cast<int32_t>(rb < most_blocks ? rb : most_blocks);
  const int64_t cb = (groups + (int64_t(1) << s.shift) - 1) >> s.shift, room = most_blocks / s.row_blocks;
  s.col_blocks = static_cast<int32_t>(cb < room ? cb : room > 1 ? room : 1);
  return s;
}

inline int sweep_blocks(const Sweep& s) { return s.row_blocks * s.col_blocks; }

// An operand laid out for the tensor cores: [terms][sweep.rows][ld_dst].
struct PackTask {
  EpiView src;
  __nv_bfloat16* dst;
  int64_t ld_dst, term_stride;
  int32_t cols, terms;
  Sweep sweep;
};

// What precedes the products of a call, in one launch: blocks [begin[i], begin[i + 1]) run
// task i, the column sums last.
struct PrepareParams {
  PackTask pack[3];
  ColumnSumTask sum;
  int32_t packs;
  int32_t begin[5];
};

// The end of a split reduction.
struct JoinTask {
  Epilogue e;
  const float* partial;
  int64_t ld_partial, split_stride;
  int32_t splits;
  Sweep sweep;
};

// What follows the products, likewise.
struct FinishParams {
  JoinTask join[2];
  ColumnSumTask sum;
  int32_t joins;
  int32_t begin[4];
};

cudaError_t launch_prepare(const PrepareParams& p, cudaStream_t stream);
cudaError_t launch_finish(const FinishParams& p, cudaStream_t stream);

// Launches with programmatic stream serialisation: every kernel of the layers waits
// (griddepcontrol.wait) before it touches what the launch before may have written.
template <class K, class P>
cudaError_t launch_dependent(K kernel, const P& p, dim3 grid, int threads, cudaStream_t stream, int smem = 0,
                             int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return counted(cudaLaunchKernelEx(&cfg, kernel, p));
}

}  // namespace muon
