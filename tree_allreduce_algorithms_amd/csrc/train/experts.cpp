// C entry points of the experts' products: checks and dispatch.
#include "train/experts.hpp"

#include <limits>

#include "launch.hpp"

namespace {

constexpr uint64_t kMost = std::numeric_limits<int32_t>::max();

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Whether rows of `size` elements of `width` bytes, `stride` elements apart, fit the
// address space.
bool fits(const void* p, uint64_t rows, uint64_t stride, uint64_t size, uint64_t width) {
  if (rows == 0 || size == 0) return true;
  const uint64_t room = (std::numeric_limits<uintptr_t>::max() - reinterpret_cast<uintptr_t>(p)) / width;
  return size <= room && (rows == 1 || stride <= (room - size) / (rows - 1));
}

ar_status_t check(const ar_expert_rows_t* r) {
  if (r == nullptr || r->experts < 1 || r->in < 1 || r->out < 1) return AR_ERROR_INVALID_ARGUMENT;
  if (r->dtype != AR_BFLOAT16 || r->experts > AR_MAX_EXPERTS || r->pairs > kMost || r->x_rows > kMost ||
      r->in > kMost || r->out > kMost)
    return AR_ERROR_UNSUPPORTED;
  if (r->offsets == nullptr || !aligned(r->offsets, 4) || !aligned(r->order, 4) ||
      (r->order != nullptr && r->top_k < 1))
    return AR_ERROR_INVALID_ARGUMENT;
  if (r->x_rows != 0 && (r->x == nullptr || !aligned(r->x, 2) || (r->x_rows > 1 && r->x_stride < r->in) ||
                         !fits(r->x, r->x_rows, r->x_stride, r->in, 2)))
    return AR_ERROR_INVALID_ARGUMENT;
  if (r->order == nullptr && r->x_rows < r->pairs) return AR_ERROR_INVALID_ARGUMENT;
  return AR_SUCCESS;
}

// Whether the `n` bytes at p and the rows at q (see fits) share none.
bool apart(const void* p, uint64_t n, const void* q, uint64_t rows, uint64_t stride, uint64_t size, uint64_t width) {
  if (rows == 0 || size == 0 || q == nullptr) return true;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p), other = reinterpret_cast<uintptr_t>(q);
  return lo + n <= other || other + ((rows - 1) * stride + size) * width <= lo;
}

// Rows of 16-byte pieces within the reach of 32-bit offsets.  Others go through registers
// (65,536 rows of 14,336 times 14,336 x 4,096 take 8.0 ms straight to LDS; 131,072, which
// are past the reach, 26.2 ms instead of 16).
bool wide(const void* p, uint64_t rows, uint64_t stride, uint64_t size) {
  return aligned(p, 16) && size % 8 == 0 && (rows < 2 || (stride % 8 == 0 && stride <= ar::kProductReach / 2 / rows)) &&
         size <= ar::kProductReach / 2;
}

ar_status_t check_sums(const void* y, uint64_t y_stride, uint64_t pairs, uint64_t size, ar_dtype_t dtype,
                       const int32_t* position, uint64_t tokens, int top_k) {
  if (size < 1 || top_k < 1) return AR_ERROR_INVALID_ARGUMENT;
  if (dtype != AR_BFLOAT16 || pairs > kMost || tokens > kMost / static_cast<uint64_t>(top_k) || size > kMost)
    return AR_ERROR_UNSUPPORTED;
  if ((size - 1) / 8 / 256 >= 65535) return AR_ERROR_UNSUPPORTED;
  if (tokens != 0 && (position == nullptr || !aligned(position, 4))) return AR_ERROR_INVALID_ARGUMENT;
  if (pairs != 0 && (y == nullptr || !aligned(y, 2) || (pairs > 1 && y_stride < size) ||
                     !fits(y, pairs, y_stride, size, 2)))
    return AR_ERROR_INVALID_ARGUMENT;
  return AR_SUCCESS;
}

}  // namespace

extern "C" {

size_t ar_expert_order_workspace(size_t pairs, int experts) {
  if (experts < 1 || experts > AR_MAX_EXPERTS || pairs > kMost) return 0;
  return static_cast<size_t>(ar::order_blocks(pairs)) * experts * sizeof(uint32_t);
}

ar_status_t ar_expert_order(const int32_t* indices, size_t pairs, int experts, int32_t* order,
                            int32_t* position, int32_t* offsets, void* workspace, hipStream_t stream) {
  if (experts < 1) return AR_ERROR_INVALID_ARGUMENT;
  if (experts > AR_MAX_EXPERTS || pairs > kMost) return AR_ERROR_UNSUPPORTED;
  if (offsets == nullptr || !aligned(offsets, 4) ||
      (pairs != 0 && (indices == nullptr || order == nullptr || position == nullptr)))
    return AR_ERROR_INVALID_ARGUMENT;
  if (!aligned(indices, 4) || !aligned(order, 4) || !aligned(position, 4) || !aligned(workspace, 16) ||
      (workspace == nullptr && ar_expert_order_workspace(pairs, experts) != 0))
    return AR_ERROR_INVALID_ARGUMENT;
  ar::OrderArgs a;
  a.indices = indices;
  a.pairs = static_cast<uint32_t>(pairs);
  a.experts = experts;
  a.order = order;
  a.position = position;
  a.offsets = offsets;
  // whole rounds of a block's waves, and no block without pairs
  const uint64_t blocks = ar::order_blocks(pairs), unit = ar::kOrderWaves * 64;
  a.counts = blocks != 0 ? static_cast<uint32_t*>(workspace) : nullptr;
  a.block_pairs = static_cast<uint32_t>(blocks == 0 ? unit : ((pairs + blocks - 1) / blocks + unit - 1) / unit * unit);
  a.blocks = pairs == 0 ? 1 : static_cast<uint32_t>((pairs - 1) / a.block_pairs + 1);
  hipError_t err = hipSuccess;
  if (a.counts != nullptr) err = ar::enqueue([&] { return ar::launch_expert_order_count(a, stream); });
  if (err == hipSuccess) err = ar::enqueue([&] { return ar::launch_expert_order_place(a, stream); });
  return ar::launch_status(err);
}

ar_status_t ar_expert_matmul(const ar_expert_rows_t* r, const void* weight, size_t expert_stride,
                             size_t in_stride, size_t out_stride, void* y, hipStream_t stream) {
  const ar_status_t st = check(r);
  if (st != AR_SUCCESS) return st;
  if (weight == nullptr || !aligned(weight, 2)) return AR_ERROR_INVALID_ARGUMENT;
  // columns next to each other, or rows; where a size is 1 its stride says nothing
  const bool by_out = (out_stride == 1 || r->out == 1) && (r->in == 1 || in_stride >= r->out);
  const bool by_in = (in_stride == 1 || r->in == 1) && (r->out == 1 || out_stride >= r->in);
  if (!by_out && !by_in) return AR_ERROR_INVALID_ARGUMENT;
  const uint64_t lines = by_out ? r->in : r->out, length = by_out ? r->out : r->in;
  const uint64_t line = lines == 1 ? length : by_out ? in_stride : out_stride;
  if (!fits(weight, lines, line, length, 2) ||
      !fits(weight, r->experts, expert_stride, (lines - 1) * line + length, 2))
    return AR_ERROR_INVALID_ARGUMENT;
  if (r->pairs == 0) return AR_SUCCESS;
  if (y == nullptr || !aligned(y, 2) || !fits(y, r->pairs, r->out, r->out, 2)) return AR_ERROR_INVALID_ARGUMENT;
  const uint64_t x_stride = r->x_rows > 1 ? r->x_stride : r->in, w_expert = r->experts > 1 ? expert_stride : 0;
  const bool direct = wide(r->x, r->x_rows, x_stride, r->in) && wide(weight, lines, line, length) && w_expert % 8 == 0;
  if (ar::expert_product_blocks(r->pairs, r->experts, r->out, by_out, direct) > ar::kMaxProductBlocks)
    return AR_ERROR_UNSUPPORTED;
  ar::ProductArgs a;
  a.x = r->x;
  a.w = weight;
  a.y = y;
  a.order = r->order;
  a.offsets = r->offsets;
  a.x_stride = x_stride;
  a.w_expert = w_expert;
  a.w_line = line;
  a.x_rows = static_cast<uint32_t>(r->x_rows);
  a.pairs = static_cast<uint32_t>(r->pairs);
  a.in = static_cast<uint32_t>(r->in);
  a.out = static_cast<uint32_t>(r->out);
  a.tiles_n = 0;
  a.experts = r->experts;
  a.token = ar::token_of(r->pairs, r->order != nullptr ? r->top_k : 1);
  return ar::launch_status(ar::enqueue([&] { return ar::launch_expert_product(a, by_out, direct, stream); }));
}

size_t ar_expert_weight_grad_workspace(size_t pairs, int experts, size_t in, size_t out) {
  if (experts < 1 || experts > AR_MAX_EXPERTS || in < 1 || out < 1 || in > kMost || out > kMost || pairs > kMost) return 0;
  const uint32_t parts = ar::expert_weight_grad_parts(pairs, experts, in, out);
  // (with parts there are at most 256 tiles of 128 x 256 float32)
  return parts > 1 ? parts * sizeof(float) * experts * in * out : 0;
}

ar_status_t ar_expert_weight_grad(const ar_expert_rows_t* r, const void* dy, size_t dy_stride, void* dw,
                                  ar_dtype_t dw_dtype, void* workspace, hipStream_t stream) {
  const ar_status_t st = check(r);
  if (st != AR_SUCCESS) return st;
  if (dw_dtype != AR_FLOAT32 && dw_dtype != AR_BFLOAT16) return AR_ERROR_UNSUPPORTED;
  const uint64_t size = dw_dtype == AR_FLOAT32 ? 4 : 2;
  if (dw == nullptr || !aligned(dw, size) || r->in > std::numeric_limits<uint64_t>::max() / r->out / r->experts ||
      !fits(dw, 1, 0, r->in * r->out * r->experts, size))
    return AR_ERROR_INVALID_ARGUMENT;
  if (r->pairs != 0 && (dy == nullptr || !aligned(dy, 2) || (r->pairs > 1 && dy_stride < r->out) ||
                        !fits(dy, r->pairs, dy_stride, r->out, 2)))
    return AR_ERROR_INVALID_ARGUMENT;
  // dw may be a part of a larger buffer of the caller's: nothing that is read lies in it
  const uint64_t bytes = static_cast<uint64_t>(r->experts) * r->in * r->out * size;
  if (!apart(dw, bytes, r->x, r->x_rows, r->x_stride, r->in, 2) ||
      !apart(dw, bytes, dy, r->pairs, dy_stride, r->out, 2) || !apart(dw, bytes, r->offsets, 1, 0, r->experts + 1, 4) ||
      !apart(dw, bytes, r->order, 1, 0, r->pairs, 4))
    return AR_ERROR_INVALID_ARGUMENT;
  const uint64_t x_stride = r->x_rows > 1 ? r->x_stride : r->in, y_stride = r->pairs > 1 ? dy_stride : r->out;
  const bool direct = wide(r->x, r->x_rows, x_stride, r->in) && wide(dy, r->pairs, y_stride, r->out);
  if (ar::expert_weight_grad_blocks(r->experts, r->in, r->out, direct) > ar::kMaxProductBlocks)
    return AR_ERROR_UNSUPPORTED;
  const uint32_t parts = ar::expert_weight_grad_parts(r->pairs, r->experts, r->in, r->out);
  if (parts > 1 && (workspace == nullptr || !aligned(workspace, 16))) return AR_ERROR_INVALID_ARGUMENT;
  ar::WeightGradArgs a;
  a.x = r->x;
  a.dy = dy;
  a.dw = dw;
  a.order = r->order;
  a.offsets = r->offsets;
  a.x_stride = x_stride;
  a.dy_stride = y_stride;
  a.x_rows = static_cast<uint32_t>(r->x_rows);
  a.pairs = static_cast<uint32_t>(r->pairs);
  a.in = static_cast<uint32_t>(r->in);
  a.out = static_cast<uint32_t>(r->out);
  a.tiles_n = a.tiles = a.tiles_xcd = a.xcds = 0;
  a.parts = parts;
  a.experts = r->experts;
  a.token = ar::token_of(r->pairs, r->order != nullptr ? r->top_k : 1);
  if (parts > 1) a.dw = workspace;
  hipError_t err = ar::enqueue(
      [&] { return ar::launch_expert_weight_grad(a, parts > 1 ? AR_FLOAT32 : dw_dtype, direct, stream); });
  if (err == hipSuccess && parts > 1)
    err = ar::enqueue([&] { return ar::launch_expert_add_parts(a, dw, dw_dtype, stream); });
  return ar::launch_status(err);
}

ar_status_t ar_expert_combine(const void* y, size_t y_stride, size_t pairs, size_t size, ar_dtype_t dtype,
                              const int32_t* position, const float* weights, size_t tokens, int top_k,
                              void* out, hipStream_t stream) {
  const ar_status_t st = check_sums(y, y_stride, pairs, size, dtype, position, tokens, top_k);
  if (st != AR_SUCCESS) return st;
  // the kernel counts the choices by up to four at a time in an int
  if (static_cast<uint64_t>(top_k) > kMost - 3) return AR_ERROR_UNSUPPORTED;
  if (tokens == 0) return AR_SUCCESS;
  if (out == nullptr || !aligned(out, 2) || !aligned(weights, 4) || !fits(out, tokens, size, size, 2))
    return AR_ERROR_INVALID_ARGUMENT;
  ar::CombineArgs a = {};
  a.y = y;
  a.position = position;
  a.weights = weights;
  a.out = out;
  a.y_stride = pairs > 1 ? y_stride : size;
  a.tokens = static_cast<uint32_t>(tokens);
  a.pairs = static_cast<uint32_t>(pairs);
  a.size = static_cast<uint32_t>(size);
  a.top_k = top_k;
  return ar::launch_status(ar::enqueue([&] { return ar::launch_expert_combine(a, stream); }));
}

ar_status_t ar_expert_combine_grad(const void* dout, size_t dout_stride, const void* y, size_t y_stride,
                                   size_t pairs, size_t size, ar_dtype_t dtype, const int32_t* position,
                                   const int32_t* offsets, int experts, const float* weights, size_t tokens,
                                   int top_k, void* dy, float* dweights, hipStream_t stream) {
  const ar_status_t st = check_sums(y, y_stride, pairs, size, dtype, position, tokens, top_k);
  if (st != AR_SUCCESS) return st;
  if (experts < 1) return AR_ERROR_INVALID_ARGUMENT;
  if (experts > AR_MAX_EXPERTS) return AR_ERROR_UNSUPPORTED;
  if (tokens == 0 && pairs == 0) return AR_SUCCESS;
  if (offsets == nullptr || !aligned(offsets, 4)) return AR_ERROR_INVALID_ARGUMENT;
  if (tokens != 0 && (dout == nullptr || !aligned(dout, 2) || weights == nullptr || !aligned(weights, 4) ||
                      dweights == nullptr || !aligned(dweights, 4) || (tokens > 1 && dout_stride < size) ||
                      !fits(dout, tokens, dout_stride, size, 2)))
    return AR_ERROR_INVALID_ARGUMENT;
  if (pairs != 0 && (dy == nullptr || !aligned(dy, 2) || !fits(dy, pairs, size, size, 2)))
    return AR_ERROR_INVALID_ARGUMENT;
  ar::CombineArgs a = {};
  a.y = y;
  a.dout = dout;
  a.position = position;
  a.offsets = offsets;
  a.weights = weights;
  a.out = dy;
  a.dweights = dweights;
  a.y_stride = pairs > 1 ? y_stride : size;
  a.dout_stride = tokens > 1 ? dout_stride : size;
  a.tokens = static_cast<uint32_t>(tokens);
  a.pairs = static_cast<uint32_t>(pairs);
  a.size = static_cast<uint32_t>(size);
  a.experts = experts;
  a.top_k = top_k;
  return ar::launch_status(ar::enqueue([&] { return ar::launch_expert_combine_grad(a, stream); }));
}

}  // extern "C"
