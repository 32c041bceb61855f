// C entry points of the expert router: checks and dispatch.
#include "train/route.hpp"

#include <cstring>
#include <limits>

#include "launch.hpp"

namespace {

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

ar_status_t check(const void* const* logits, const uint8_t* const* masks, const ar_route_shape_t* s) {
  if (logits == nullptr || s == nullptr) return AR_ERROR_INVALID_ARGUMENT;
  if (s->nranks < 1 || s->nranks > AR_MAX_RANKS || s->experts < 1 || s->top_k < 1 ||
      s->top_k > s->experts || s->row_stride < static_cast<size_t>(s->experts))
    return AR_ERROR_INVALID_ARGUMENT;
  if (s->dtype != AR_FLOAT32 && s->dtype != AR_BFLOAT16) return AR_ERROR_UNSUPPORTED;
  if (s->experts > AR_MAX_EXPERTS || s->top_k > AR_MAX_TOP_K) return AR_ERROR_UNSUPPORTED;
  const size_t most = std::numeric_limits<int32_t>::max();
  if (s->tokens > most / s->nranks) return AR_ERROR_UNSUPPORTED;
  if (s->tokens == 0) return AR_SUCCESS;
  if (s->row_stride > std::numeric_limits<uintptr_t>::max() / 4 / s->tokens)
    return AR_ERROR_INVALID_ARGUMENT;
  const uintptr_t size = s->dtype == AR_FLOAT32 ? 4 : 2;
  for (int r = 0; r < s->nranks; ++r) {
    if (logits[r] == nullptr || !aligned(logits[r], size)) return AR_ERROR_INVALID_ARGUMENT;
    if (masks != nullptr && masks[r] == nullptr) return AR_ERROR_INVALID_ARGUMENT;
  }
  return AR_SUCCESS;
}

template <int N, class P> void fill(ar::Pointers<N>* to, P const* from, const ar_route_shape_t* s) {
  std::memset(to, 0, sizeof(*to));
  if (from == nullptr || s->tokens == 0) return;
  for (int r = 0; r < s->nranks; ++r) to->p[r] = from[r];
}

void fill_shape(ar::RouteShape* a, const ar_route_shape_t* s) {
  a->row_stride = s->row_stride;
  a->tokens = static_cast<uint32_t>(s->tokens);
  a->rows_per_block = 0;
  a->group = 0;
  a->nranks = s->nranks;
  a->experts = s->experts;
  a->top_k = s->top_k;
  a->renormalize = s->renormalize != 0;
}

template <int N>
hipError_t route(const void* const* logits, const uint8_t* const* masks, const ar_route_shape_t* shape,
                 int32_t* indices, float* weights, int32_t* counts, float* loss, float* share,
                 void* workspace, hipStream_t stream) {
  ar::RouteArgs<N> a;
  fill(&a.logits, logits, shape);
  fill(&a.masks, masks, shape);
  fill_shape(&a, shape);
  a.sums = static_cast<ar::RouteSums*>(workspace);
  a.indices = indices;
  a.weights = weights;
  a.counts = counts;
  a.loss = loss;
  a.share = share;
  return ar::launch_route(a, shape->dtype, stream);
}

template <int N>
hipError_t route_grad(const void* const* logits, const uint8_t* const* masks, const ar_route_shape_t* shape,
                      const int32_t* indices, const float* share, const float* const* dweights,
                      const float* dloss, void* dlogits, hipStream_t stream) {
  ar::RouteGradArgs<N> a;
  fill(&a.logits, logits, shape);
  fill(&a.masks, masks, shape);
  fill(&a.dweights, dweights, shape);
  fill_shape(&a, shape);
  a.indices = indices;
  a.share = share;
  a.dloss = dloss;
  a.dlogits = dlogits;
  return ar::launch_route_grad(a, shape->dtype, stream);
}

}  // namespace

extern "C" {

ar_status_t ar_route(const void* const* logits, const uint8_t* const* masks,
                     const ar_route_shape_t* shape, int32_t* indices, float* weights,
                     int32_t* counts, float* loss, float* share, void* workspace,
                     hipStream_t stream) {
  const ar_status_t st = check(logits, masks, shape);
  if (st != AR_SUCCESS) return st;
  if (counts == nullptr || loss == nullptr || share == nullptr || workspace == nullptr ||
      (shape->tokens != 0 && (indices == nullptr || weights == nullptr)))
    return AR_ERROR_INVALID_ARGUMENT;
  if (!aligned(indices, 4) || !aligned(weights, 4) || !aligned(counts, 4) || !aligned(loss, 4) ||
      !aligned(share, 4) || !aligned(workspace, 16))
    return AR_ERROR_INVALID_ARGUMENT;
  return ar::launch_status(ar::enqueue([&] {
    return (shape->nranks <= ar::kFewRanks ? route<ar::kFewRanks> : route<AR_MAX_RANKS>)(
        logits, masks, shape, indices, weights, counts, loss, share, workspace, stream);
  }));
}

ar_status_t ar_route_grad(const void* const* logits, const uint8_t* const* masks,
                          const ar_route_shape_t* shape, const int32_t* indices,
                          const float* share, const float* const* dweights, const float* dloss,
                          void* dlogits, hipStream_t stream) {
  const ar_status_t st = check(logits, masks, shape);
  if (st != AR_SUCCESS) return st;
  if (shape->tokens == 0) return AR_SUCCESS;
  if (indices == nullptr || share == nullptr || dlogits == nullptr || !aligned(indices, 4) ||
      !aligned(share, 4) || !aligned(dloss, 4) ||
      !aligned(dlogits, shape->dtype == AR_FLOAT32 ? 4 : 2))
    return AR_ERROR_INVALID_ARGUMENT;
  if (dweights != nullptr)
    for (int r = 0; r < shape->nranks; ++r)
      if (dweights[r] == nullptr || !aligned(dweights[r], 4)) return AR_ERROR_INVALID_ARGUMENT;
  return ar::launch_status(ar::enqueue([&] {
    return (shape->nranks <= ar::kFewRanks ? route_grad<ar::kFewRanks> : route_grad<AR_MAX_RANKS>)(
        logits, masks, shape, indices, share, dweights, dloss, dlogits, stream);
  }));
}

}  // extern "C"
