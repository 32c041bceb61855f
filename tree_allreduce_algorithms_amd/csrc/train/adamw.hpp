// AdamW plans: what the host lays out and the kernels read.
//
// A plan is one image, identical in host and device memory:
//   AdamwHead     sizes and types (the host reads them)
//   AdamwSums     the norm's partial sums and results (device only)
//   tensors       one AdamwTensor per tensor that has elements
//   tiles         one AdamwTile per unit of work
// All offsets are from the image's start.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ar.h"

namespace ar {

constexpr uint32_t kAdamwMagic = 0x41573031u;
constexpr uint32_t kAdamwTile = 4096;       // elements of a tile

// A launch has less than 2^32 threads.  A step has up to four blocks of 256 a
// tile, a decoding one.
constexpr uint32_t kAdamwMaxTiles = (1u << 22) - 1;
constexpr uint32_t kAdamwMaxDecodeTiles = (1u << 24) - 1;

// A 32-bit step whose reads come to this much or less goes through the caches
// for them, a longer one past them.  Norm and step back to back, float32
// throughout: 256 MiB 83 us through and 97 past, 320 MiB 103 and 122, 400 MiB
// 154 and 145, 1 GiB 391 and 369.
constexpr uint64_t kKeepBytes = 320ull << 20;

// An eps (with its bias correction) beside which the float32 root and
// reciprocal of a step would be wrong: below 2^25 times the roots (1.1e-19)
// that are taken as 0, or so large that its reciprocal is subnormal, which is
// taken as 0 too.  Such a step's updates are computed in float64.
inline bool wide_eps(double eps) { return eps < 4e-12 || eps > 1e37; }

// Blocks of a norm, and how many of them make a group: the sums of a group's
// blocks, and those of the groups, are added up by one block.
constexpr uint32_t kMaxNormBlocks = 1024;
constexpr uint32_t kNormGroup = 32;
constexpr uint32_t kNormGroups = kMaxNormBlocks / kNormGroup;

struct AdamwHead {
  uint32_t magic;
  uint32_t tensors;
  uint32_t tiles;
  uint32_t tile_elements;
  int32_t param_dtype;
  int32_t grad_dtype;
  int32_t state_bits;
  int32_t has_copy;
  uint64_t bytes;
  uint64_t sums_at;
  uint64_t tensors_at;
  uint64_t tiles_at;
  uint64_t touched;       // bytes that a step reads
};

struct AdamwSums {
  double of_block[kMaxNormBlocks];
  double of_group[kNormGroups];
  // how many have left their sum, 0 between calls; each in a line of its own
  struct alignas(256) Counter {
    uint32_t count;
  } arrived[kNormGroups], groups_arrived;
  alignas(256) float factor;                // of the last norm
};

struct AdamwTensor {
  void* p;
  const void* g;
  void* copy;
  void* m;
  void* v;
  float* ms;
  float* vs;
  uint64_t count;
  uint32_t vec;      // every pointer allows four elements per access
  uint32_t pad[3];
};

struct AdamwTile {
  uint32_t tensor;
  uint32_t index;    // elements [index, index + 1) * kAdamwTile of it
};

struct AdamwNormArgs {
  char* plan;
  uint64_t sums_at, tensors_at, tiles_at;
  uint32_t tiles;
  double max_norm;
  double grad_scale;
  float* norm;
};

struct AdamwStepArgs {
  char* plan;
  uint64_t sums_at, tensors_at, tiles_at;
  int clip;
  float factor;               // without clip
  float lr_wd;
  float lr, eps;              // with the bias corrections, see updated()
  double b1, one_b1;          // beta, 1 - beta
  double b2, one_b2;
  double root_b2, root_one_b2;
  double eps64;               // eps before its rounding
  int far;                    // wide_eps(eps64)
};

hipError_t launch_adamw_norm(const AdamwNormArgs& a, ar_dtype_t grad_dtype, hipStream_t stream);
hipError_t launch_adamw_step(const AdamwStepArgs& a, uint32_t tiles, ar_dtype_t param_dtype,
                             ar_dtype_t grad_dtype, int state_bits, bool copy, bool keep, hipStream_t stream);
hipError_t launch_adamw_dequantize(const void* codes, const float* scales, uint64_t count,
                                   bool is_signed, float* out, hipStream_t stream);

}  // namespace ar
