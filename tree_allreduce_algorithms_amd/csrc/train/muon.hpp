// Muon plans: what the host lays out and the kernels read.
//
// A plan is one image, identical in host and device memory:
//   MuonHead      sizes and types (the host reads them)
//   matrices      one MuonMatrix per matrix
//   chunks        one MuonChunk per unit of element-wise work
//   squares       one MuonTile per tile of X X^T on or above the diagonal
//   polys         the same for the polynomial of X X^T, whose tiles cost otherwise
//   tiles         one MuonTile per tile of X
//                 (all dealt to the XCDs, with entries of none between)
//   norms         MuonNorm per matrix (device only), then a double per chunk
//   arrived       a counter for each tile in parts (device only), 0 between calls
// All offsets are from the image's start.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ar.h"

namespace ar {

constexpr uint32_t kMuonMagic = 0x4d553031u;
constexpr uint32_t kMuonChunk = 8192;         // elements of a chunk of a matrix
constexpr uint64_t kMuonMaxTiles = (1u << 22) - 1;
constexpr uint32_t kMuonXcds = 8;            // blocks come to them in turn
// elements of one padded matrix: 32-bit offsets reach 2^31 bytes of 16 bits
constexpr uint64_t kMuonMaxElements = 1ull << 30;
constexpr int kMuonMaxSteps = 32;

struct MuonHead {
  uint32_t magic;
  uint32_t matrices;
  uint32_t chunks;
  uint32_t squares;          // entries of the tables
  uint32_t polys;
  uint32_t tiles;
  uint32_t side;             // of a tile of X: 64 or 128
  uint32_t square_side;      // of a tile of X X^T
  int32_t param_dtype;
  int32_t grad_dtype;
  int32_t has_copy;
  uint16_t longest, shortest;      // 64 or 128: no matrix's longer and shorter side is more; 0, 0
  uint64_t bytes;
  uint64_t workspace;        // bytes
  uint64_t matrices_at, chunks_at, squares_at, polys_at, tiles_at, norms_at, sums_at, arrived_at;
  uint64_t parts_at;         // in the workspace: the parts' sums
};

struct MuonMatrix {
  void* p;
  const void* g;
  void* copy;
  float* m;
  uint64_t x[2], gram, poly;       // in the workspace; the small parts lie behind the large
  uint64_t x_plane, gram_plane;    // bytes of a plane
  uint32_t rows, cols;
  uint32_t height, width;          // of X: the shorter and the longer side, padded to whole tiles
  uint32_t tall;                   // X is the transposed matrix
  uint32_t vec;                    // four elements of a row may be accessed at once
  uint32_t flat;                   // and four from any fourth element on
  uint32_t first_chunk, chunks;
  float by_shape, by_size;         // sqrt(max(1, rows / cols)), sqrt(max(rows, cols))
  uint32_t pad;
};

struct MuonChunk {
  uint32_t matrix, index;
};

// A tile of a product, or a part of its k: the parts leave their sums in the
// workspace, and the last to arrive adds them up, in their order.
constexpr uint32_t kMuonNoMatrix = 0xffffffffu;
struct MuonTile {
  uint32_t matrix;           // kMuonNoMatrix: nothing to do
  uint16_t m, n;
  uint32_t first, steps;     // of kMuonStep k
  uint32_t part, parts;
  uint32_t slot;             // of its first part's sums
  uint32_t counter;
};
constexpr uint32_t kMuonStep = 32;

struct MuonNorm {
  uint32_t arrived;          // chunks that have left their sum; 0 between calls
  uint32_t pad;
  double inverse;            // 1 / (|u| + eps)
  uint32_t rest[12];
};

struct MuonStepArgs {
  char* plan;
  char* workspace;
  uint64_t matrices_at, chunks_at, squares_at, polys_at, tiles_at, norms_at, sums_at, arrived_at, parts_at;
  float momentum, grad_scale, lr, lr_wd;
  double eps;
  float rms;                 // 0: scaled by shape
  int nesterov, last;        // last: the final product updates the parameters
  int from;                  // which of the two X is read
  int steps;                 // all of them, for launch_muon_whole
};

hipError_t launch_muon_momentum(const MuonStepArgs& a, uint32_t chunks, ar_dtype_t grad_dtype, hipStream_t stream);
hipError_t launch_muon_start(const MuonStepArgs& a, uint32_t tiles, uint32_t side, ar_dtype_t grad_dtype,
                             hipStream_t stream);
hipError_t launch_muon_gram(const MuonStepArgs& a, uint32_t squares, uint32_t side, hipStream_t stream);
hipError_t launch_muon_poly(const MuonStepArgs& a, uint32_t squares, uint32_t side, hipStream_t stream);
hipError_t launch_muon_apply(const MuonStepArgs& a, uint32_t tiles, uint32_t side, ar_dtype_t param_dtype, bool copy,
                             hipStream_t stream);

// Steps of matrices of up to `longest` by `shortest` (64 or 128), a block each.
hipError_t launch_muon_whole(const MuonStepArgs& a, uint32_t matrices, uint32_t longest, uint32_t shortest,
                             ar_dtype_t param_dtype, ar_dtype_t grad_dtype, bool copy, hipStream_t stream);

}  // namespace ar
