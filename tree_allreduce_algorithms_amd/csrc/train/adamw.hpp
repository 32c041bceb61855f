// AdamW plans: what the host lays out and the kernels read.
//
// A plan is one image, identical in host and device memory:
//   AdamwHead     sizes and types (host reads), and the norm's results
//   partials      kMaxNormBlocks doubles (device only)
//   tensors       one AdamwTensor per tensor that has elements
//   tiles         one AdamwTile per unit of work
// All offsets are from the image's start.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ar.h"

namespace ar {

constexpr uint32_t kAdamwMagic = 0x41573031u;
constexpr uint32_t kMaxNormBlocks = 2048;
constexpr uint32_t kAdamwStep = 1024;       // elements a block handles at a time
constexpr uint32_t kMaxTileSteps = 4;

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
  uint64_t partials_at;
  uint64_t tensors_at;
  uint64_t tiles_at;
  // device side: the last norm's factor, and how many blocks of the running
  // norm have left their partial sum (0 between calls)
  float factor;
  uint32_t arrived;
  uint64_t pad;
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
  uint32_t index;    // elements [index, index + 1) * tile_elements of it
};

struct AdamwNormArgs {
  char* plan;
  uint64_t partials_at, tensors_at, tiles_at;
  uint32_t tiles, tile_elements;
  double max_norm;
  double grad_scale;
  float* norm;
};

struct AdamwStepArgs {
  char* plan;
  uint64_t tensors_at, tiles_at;
  uint32_t tile_elements;
  int clip;
  float factor;                     // without clip
  float lr, lr_wd, eps, bc1, bc2;   // bc = 1 - beta^step
  double b1, one_b1, b2, one_b2;
};

hipError_t launch_adamw_norm(const AdamwNormArgs& a, ar_dtype_t grad_dtype, hipStream_t stream);
hipError_t launch_adamw_step(const AdamwStepArgs& a, uint32_t tiles, ar_dtype_t param_dtype,
                             ar_dtype_t grad_dtype, int state_bits, bool copy, hipStream_t stream);
hipError_t launch_adamw_dequantize(const void* codes, const float* scales, uint64_t count,
                                   bool is_signed, float* out, hipStream_t stream);

}  // namespace ar
