// The expert router: what the entry points hand to the kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kernels.hpp"

namespace ar {

// A router call's sums (AR_ROUTE_WORKSPACE bytes of device memory).  Every
// block leaves a row of S_e and of counts; the last block of a group adds the
// group's up and onto the totals, whole numbers, in which the order of adding
// does not show.  Totals and counters are 0 between calls, the counters each in
// a line of its own; the rows need no clearing.
constexpr int kRouteBlocks = 256;
constexpr int kRouteGroups = 64;

struct RouteSums {
  struct alignas(256) Counter {
    uint32_t count;
  } arrived[kRouteGroups], groups_arrived;
  uint32_t tokens;                                 // that live
  uint32_t not_finite;                             // a sum of probabilities was not
  uint64_t share[AR_MAX_EXPERTS];                  // S_e in steps of 2^-32
  uint32_t counts[AR_MAX_RANKS * AR_MAX_EXPERTS];  // [rank][experts]
  uint32_t tokens_of_block[kRouteBlocks];
  // [block][experts]: S_e as float32 in the high word, counts in the low
  uint64_t of_block[kRouteBlocks * AR_MAX_EXPERTS];
};
static_assert(sizeof(RouteSums) <= AR_ROUTE_WORKSPACE, "the workspace's documented size");

// One pointer a rank, for at most N ranks: kernels take them by value, and a
// launch with room for 8 ranks in its arguments costs the host about 1 us less
// than one with room for 64 (2.3 us against 3.5 for 16 and 1,600 bytes).
template <int N> struct Pointers {
  const void* p[N];
};
constexpr int kFewRanks = 8;

struct RouteShape {
  uint64_t row_stride;             // elements
  uint32_t tokens;                 // of a rank
  uint32_t rows_per_block;         // blocks (x, rank): tokens [x, x + 1) * rows_per_block
  uint32_t group;                  // blocks of a rank whose sums are joined first
  int nranks, experts, top_k, renormalize;
};

template <int N> struct RouteArgs : RouteShape {
  Pointers<N> logits;
  Pointers<N> masks;               // p[0] NULL: none
  RouteSums* sums;
  int32_t* indices;
  float* weights;
  int32_t* counts;
  float* loss;
  float* share;
};

template <int N> struct RouteGradArgs : RouteShape {
  Pointers<N> logits;
  Pointers<N> masks;
  Pointers<N> dweights;            // p[0] NULL: none
  const int32_t* indices;
  const float* share;
  const float* dloss;              // NULL: 0
  void* dlogits;
};

// rows_per_block and group are set by the launchers.
template <int N> hipError_t launch_route(const RouteArgs<N>& a, ar_dtype_t dtype, hipStream_t stream);
template <int N> hipError_t launch_route_grad(const RouteGradArgs<N>& a, ar_dtype_t dtype, hipStream_t stream);

}  // namespace ar
