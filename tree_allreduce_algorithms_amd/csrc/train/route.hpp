// The expert router: what the entry points hand to the kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kernels.hpp"

namespace ar {

// A router call's sums (AR_ROUTE_WORKSPACE bytes of device memory).  Every
// block leaves a row of S_e and of counts; the last block of a group adds up
// the group's rows, the last group the groups'.  The counters are 0 between
// calls, each in a line of its own; the rest needs no clearing.
constexpr int kRouteBlocks = 256;
constexpr int kRouteGroups = 64;

struct RouteSums {
  struct alignas(256) Counter {
    uint32_t count;
  } arrived[kRouteGroups], groups_arrived;
  uint32_t tokens_of_block[kRouteBlocks];            // that live
  uint32_t tokens_of_group[kRouteGroups];
  // [group or block][experts]: S_e as float32 in the high word, counts in the low
  uint64_t of_group[kRouteGroups * AR_MAX_EXPERTS];
  uint64_t of_block[kRouteBlocks * AR_MAX_EXPERTS];
};
static_assert(sizeof(RouteSums) <= AR_ROUTE_WORKSPACE, "the workspace's documented size");

struct RouteArgs {
  RankPtrs logits;
  RankPtrs masks;                  // p[0] NULL: none
  RouteSums* sums;
  int32_t* indices;
  float* weights;
  int32_t* counts;
  float* loss;
  float* share;
  uint64_t row_stride;             // elements
  uint32_t tokens;                 // of a rank
  uint32_t rows_per_block;         // blocks (x, rank): tokens [x, x + 1) * rows_per_block
  uint32_t group;                  // blocks of a rank whose sums are joined first
  int nranks, experts, top_k, renormalize;
};

struct RouteGradArgs {
  RankPtrs logits;
  RankPtrs masks;
  RankPtrs dweights;               // p[0] NULL: none
  const int32_t* indices;
  const float* share;
  const float* dloss;              // NULL: 0
  void* dlogits;
  uint64_t row_stride;
  uint32_t tokens;
  uint32_t rows_per_block;
  int nranks, experts, top_k, renormalize;
};

// rows_per_block and group are set by the launchers.
hipError_t launch_route(const RouteArgs& a, ar_dtype_t dtype, hipStream_t stream);
hipError_t launch_route_grad(const RouteGradArgs& a, ar_dtype_t dtype, hipStream_t stream);

}  // namespace ar
