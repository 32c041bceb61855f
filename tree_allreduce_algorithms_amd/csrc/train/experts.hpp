// The experts' products: what the host hands to the kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ar.h"

namespace ar {

// Up to kOrderOnce pairs the order is one launch, whose blocks have a wave for each
// 64 pairs and count all of the list: 8,192 pairs of 64 experts 5.0 us, 8.8 with
// their parts counted by a launch before; 32,768 8.8 and 9.2; 65,536 of 128 14.2 and
// 9.9.  Longer lists are counted so, a part a block, kOrderBlocks at most, since
// each block reads all blocks' counts.
constexpr uint32_t kOrderWaves = 16;
constexpr uint64_t kOrderOnce = 32768;
constexpr uint32_t kOrderBlockPairs = 4096;
constexpr uint32_t kOrderBlocks = 64;

// Blocks that are counted apart.
inline uint32_t order_blocks(uint64_t pairs) {
  if (pairs <= kOrderOnce) return 0;
  const uint64_t n = (pairs + kOrderBlockPairs - 1) / kOrderBlockPairs;
  return n > kOrderBlocks ? kOrderBlocks : static_cast<uint32_t>(n);
}

struct OrderArgs {
  const int32_t* indices;
  uint32_t pairs, block_pairs, blocks;
  int32_t experts;
  int32_t* order;
  int32_t* position;
  int32_t* offsets;
  uint32_t* counts;       // [blocks][experts], or null: the list is short
};
// Each block's pairs of each expert; the order itself.
hipError_t launch_expert_order_count(const OrderArgs& a, hipStream_t stream);
hipError_t launch_expert_order_place(const OrderArgs& a, hipStream_t stream);

// The token of a pair, pair / top_k: by a product with `reciprocal` = ceil(2^32 /
// top_k) where pairs * top_k <= 2^32 makes that exact, else (0) by a division.
struct TokenOf {
  uint32_t top_k, reciprocal;
};
inline TokenOf token_of(uint64_t pairs, uint32_t top_k) {
  const uint64_t two32 = 1ull << 32;
  return {top_k, top_k > 1 && pairs * top_k <= two32 ? static_cast<uint32_t>((two32 + top_k - 1) / top_k) : 0};
}

// Products by expert.  `line` is the distance of a weight's lines: of its rows
// (in) where the columns (out) are contiguous, of its columns otherwise.
struct ProductArgs {
  const void* x;
  const void* w;
  void* y;
  const int32_t* order;    // null: x's rows are the pairs in order
  const int32_t* offsets;
  uint64_t x_stride, w_expert, w_line;
  uint32_t x_rows, pairs, in, out, tiles_n;
  int32_t experts;
  TokenOf token;
};

// Blocks of a launch; one has less than 2^32 threads of at most 512 a block.
constexpr uint64_t kMaxProductBlocks = (1u << 23) - 1;
uint64_t expert_product_blocks(uint64_t pairs, int experts, uint64_t out, bool by_out, bool direct);
uint64_t expert_weight_grad_blocks(int experts, uint64_t in, uint64_t out, bool direct);

// Bytes that 32-bit offsets reach from one base (see tile.hpp).
constexpr uint64_t kProductReach = 0x80000000ull;

hipError_t launch_expert_product(const ProductArgs& a, bool out_contiguous, bool direct, hipStream_t stream);

struct WeightGradArgs {
  const void* x;
  const void* dy;
  void* dw;
  const int32_t* order;
  const int32_t* offsets;
  uint64_t x_stride, dy_stride;
  uint32_t x_rows, pairs, in, out, tiles_n;
  uint32_t tiles, tiles_xcd;    // of an expert; an XCD's of these
  uint32_t xcds;                // that share an expert's tiles: all or half
  uint32_t parts;               // blocks that share a tile's rows
  int32_t experts;
  TokenOf token;
};
uint32_t expert_weight_grad_parts(uint64_t pairs, int experts, uint64_t in, uint64_t out);
// With more than one part a.dw has that many float32 arrays of its size, which the
// second call adds up into dw.
hipError_t launch_expert_weight_grad(const WeightGradArgs& a, ar_dtype_t dw_dtype, bool direct, hipStream_t stream);
hipError_t launch_expert_add_parts(const WeightGradArgs& a, void* dw, ar_dtype_t dw_dtype, hipStream_t stream);

struct CombineArgs {
  const void* y;
  const void* dout;          // gradient only
  const int32_t* position;
  const int32_t* offsets;    // gradient only
  const float* weights;
  void* out;                 // the tokens' sums, or dy
  float* dweights;
  uint64_t y_stride, dout_stride;
  uint32_t tokens, pairs, size;
  int32_t experts, top_k;
};
hipError_t launch_expert_combine(const CombineArgs& a, hipStream_t stream);
hipError_t launch_expert_combine_grad(const CombineArgs& a, hipStream_t stream);

}  // namespace ar
