// Parameters of the layer products, shared by their host planner and kernels.
//
// A product is D[M x N] = sum_k A(m, k) B(n, k) followed by one epilogue:
//   v = sum + bias[n];  preact[m, n] = v;  v = act(v);  v *= act'(slope[m, n]);  v += add[m, n]
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

enum ProductTile : int {
  kPair256 = 0,     // 256 x 256 on a CTA pair, the whole reduction in tensor memory
  kPair256Sum = 1,  // the same, the reduction in pieces that are added in registers
  kOne128 = 2,      // 128 x 128 on one CTA, in pieces
  kFlip32 = 3,      // few tokens: 128 features x 32 tokens on one CTA, in pieces
  kFlip64 = 4,      // 128 features x 64 tokens
};

struct ProductParams {
  CUtensorMap map_a[kTerms];  // operand on the tile's M side
  CUtensorMap map_b[kTerms];  // operand on the tile's N side
  Epilogue e;
  int32_t a_mn, b_mn;         // majorness: 0 = contiguous along k, 1 = along the side
  int32_t tiles_m, tiles_n;
  int32_t nk;                 // k-blocks of the whole reduction
  int32_t splits, kb_per_split;
  int32_t piece;              // k-blocks per piece
  int32_t nseg;
  uint8_t seg_a[8], seg_b[8]; // the terms of each segment, smallest products first
  float* partial;             // [splits][e.rows][ld_partial] for the join kernel, or nullptr
  int64_t ld_partial, split_stride;
  unsigned long long timeout_ns;
};

// bf16 operand map of a matrix with rows of ld elements: boxes of 64 columns x box_rows rows.
bool encode_operand_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows);

int product_tile_m(int tile);
int product_tile_n(int tile);
cudaError_t launch_product(int tile, const ProductParams& p, int sms, cudaStream_t stream);

struct JoinParams {
  Epilogue e;
  const float* partial;
  int64_t ld_partial, split_stride;
  int32_t splits;
};
cudaError_t launch_join(const JoinParams& p, int sms, cudaStream_t stream);

struct PackParams {
  const void* src;
  __nv_bfloat16* dst;  // [terms][rows][ld_dst]
  int64_t rows, ld_src, ld_dst, term_stride;
  int32_t cols, src_bf16, terms, vec;
};
cudaError_t launch_pack(const PackParams& p, int sms, cudaStream_t stream);

}  // namespace muon
