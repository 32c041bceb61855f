// C entry points of the AdamW step: checks, plans, hyperparameters.
#include "train/adamw.hpp"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>
#include <new>
#include <vector>

#include "launch.hpp"

namespace {

using ar::AdamwHead;
using ar::AdamwTensor;
using ar::AdamwTile;

constexpr uint64_t align16(uint64_t x) { return (x + 15) / 16 * 16; }

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

struct Layout {
  uint32_t tensors = 0;     // with elements
  uint64_t tiles = 0;
  uint64_t tensors_at = 0, tiles_at = 0, bytes = 0;
};

constexpr uint64_t sums_at() { return (sizeof(AdamwHead) + 255) / 256 * 256; }

Layout layout_of(const ar_adamw_tensor_t* t, int n) {
  Layout l;
  for (int i = 0; i < n; ++i) {
    if (t[i].count == 0) continue;
    ++l.tensors;
    l.tiles += (t[i].count - 1) / ar::kAdamwTile + 1;
  }
  l.tensors_at = sums_at() + sizeof(ar::AdamwSums);
  l.tiles_at = align16(l.tensors_at + l.tensors * sizeof(AdamwTensor));
  l.bytes = align16(l.tiles_at + l.tiles * sizeof(AdamwTile));
  return l;
}

struct Range {
  uintptr_t lo, hi;
  bool written;
};

// A tensor's size in bytes must fit the address space; `at` gets the range.
bool range_of(const void* p, uint64_t count, uint64_t size, bool written, std::vector<Range>* at) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (count > (std::numeric_limits<uintptr_t>::max() - lo) / size) return false;
  at->push_back({lo, lo + count * size, written});
  return true;
}

ar_status_t check(const ar_adamw_tensor_t* t, int n, ar_dtype_t pd, ar_dtype_t gd, int bits) {
  if (t == nullptr || n < 1) return AR_ERROR_INVALID_ARGUMENT;
  const bool types = (pd == AR_FLOAT32 || pd == AR_BFLOAT16) && (gd == AR_FLOAT32 || gd == AR_BFLOAT16);
  if (!types || (bits != 8 && bits != 32)) return AR_ERROR_UNSUPPORTED;
  const uint64_t psize = pd == AR_FLOAT32 ? 4 : 2, gsize = gd == AR_FLOAT32 ? 4 : 2;
  const uint64_t ssize = bits / 8;
  std::vector<Range> ranges;
  bool first = true, copies = false;
  for (int i = 0; i < n; ++i) {
    const ar_adamw_tensor_t& x = t[i];
    if (x.count == 0) continue;
    if (x.param == nullptr || x.grad == nullptr || x.exp_avg == nullptr || x.exp_avg_sq == nullptr)
      return AR_ERROR_INVALID_ARGUMENT;
    if (!aligned(x.param, psize) || !aligned(x.grad, gsize) || !aligned(x.exp_avg, ssize) ||
        !aligned(x.exp_avg_sq, ssize) || !aligned(x.copy, 2) || !aligned(x.exp_avg_scale, 4) ||
        !aligned(x.exp_avg_sq_scale, 4))
      return AR_ERROR_INVALID_ARGUMENT;
    if ((x.exp_avg_scale != nullptr) != (bits == 8) || (x.exp_avg_sq_scale != nullptr) != (bits == 8))
      return AR_ERROR_INVALID_ARGUMENT;
    if (first) copies = x.copy != nullptr;
    first = false;
    if ((x.copy != nullptr) != copies || (copies && pd != AR_FLOAT32)) return AR_ERROR_INVALID_ARGUMENT;
    const uint64_t blocks = (x.count - 1) / AR_ADAMW_BLOCK + 1;
    bool fits = range_of(x.param, x.count, psize, true, &ranges) &&
                range_of(x.grad, x.count, gsize, false, &ranges) &&
                range_of(x.exp_avg, x.count, ssize, true, &ranges) &&
                range_of(x.exp_avg_sq, x.count, ssize, true, &ranges);
    if (fits && copies) fits = range_of(x.copy, x.count, 2, true, &ranges);
    if (fits && bits == 8)
      fits = range_of(x.exp_avg_scale, blocks, 4, true, &ranges) &&
             range_of(x.exp_avg_sq_scale, blocks, 4, true, &ranges);
    if (!fits) return AR_ERROR_INVALID_ARGUMENT;
  }
  // no written range may meet another: in order of their starts, each range
  // must begin after the furthest end of the written ones before it, and a
  // written one after the furthest end of all before it
  std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end_all = 0, end_written = 0;
  for (const Range& r : ranges) {
    if (r.lo < end_written || (r.written && r.lo < end_all)) return AR_ERROR_INVALID_ARGUMENT;
    end_all = std::max(end_all, r.hi);
    if (r.written) end_written = std::max(end_written, r.hi);
  }
  return AR_SUCCESS;
}

// No exception leaves a C entry: the host running out of memory is reported
// as a request that cannot be served.
ar_status_t check_noexcept(const ar_adamw_tensor_t* t, int n, ar_dtype_t pd, ar_dtype_t gd, int bits) {
  try {
    return check(t, n, pd, gd, bits);
  } catch (const std::bad_alloc&) {
    return AR_ERROR_UNSUPPORTED;
  }
}

bool plan_ok(const AdamwHead* h, const void* device) {
  return h != nullptr && device != nullptr && aligned(device, 16) && h->magic == ar::kAdamwMagic;
}

}  // namespace

extern "C" {

size_t ar_adamw_plan_bytes(const ar_adamw_tensor_t* tensors, int ntensors, ar_dtype_t param_dtype,
                           ar_dtype_t grad_dtype, int state_bits) {
  if (check_noexcept(tensors, ntensors, param_dtype, grad_dtype, state_bits) != AR_SUCCESS) return 0;
  const Layout l = layout_of(tensors, ntensors);
  return l.tiles > ar::kAdamwMaxTiles ? 0 : l.bytes;
}

ar_status_t ar_adamw_plan(const ar_adamw_tensor_t* tensors, int ntensors, ar_dtype_t param_dtype,
                          ar_dtype_t grad_dtype, int state_bits, void* plan, size_t bytes) {
  const ar_status_t st = check_noexcept(tensors, ntensors, param_dtype, grad_dtype, state_bits);
  if (st != AR_SUCCESS) return st;
  const Layout l = layout_of(tensors, ntensors);
  if (l.tiles > ar::kAdamwMaxTiles) return AR_ERROR_UNSUPPORTED;
  if (plan == nullptr || bytes < l.bytes || !aligned(plan, 8)) return AR_ERROR_INVALID_ARGUMENT;

  char* base = static_cast<char*>(plan);
  std::memset(base, 0, l.bytes);
  AdamwHead* h = reinterpret_cast<AdamwHead*>(base);
  h->magic = ar::kAdamwMagic;
  h->tensors = l.tensors;
  h->tiles = static_cast<uint32_t>(l.tiles);
  h->tile_elements = ar::kAdamwTile;
  h->param_dtype = param_dtype;
  h->grad_dtype = grad_dtype;
  h->state_bits = state_bits;
  h->bytes = l.bytes;
  h->sums_at = sums_at();
  h->tensors_at = l.tensors_at;
  h->tiles_at = l.tiles_at;
  // no norm yet: a step that clips all the same shows it
  reinterpret_cast<ar::AdamwSums*>(base + h->sums_at)->factor = std::numeric_limits<float>::quiet_NaN();
  AdamwTensor* out = reinterpret_cast<AdamwTensor*>(base + l.tensors_at);
  AdamwTile* tile = reinterpret_cast<AdamwTile*>(base + l.tiles_at);
  const uintptr_t pquad = param_dtype == AR_FLOAT32 ? 16 : 8, gquad = grad_dtype == AR_FLOAT32 ? 16 : 8;
  const uintptr_t squad = state_bits == 32 ? 16 : 4;
  const uint64_t read = (param_dtype == AR_FLOAT32 ? 4 : 2) + (grad_dtype == AR_FLOAT32 ? 4 : 2) + state_bits / 4;
  uint32_t k = 0;
  for (int i = 0; i < ntensors; ++i) {
    const ar_adamw_tensor_t& x = tensors[i];
    if (x.count == 0) continue;
    h->has_copy = x.copy != nullptr;
    h->touched += x.count * read;
    const bool vec = aligned(x.param, pquad) && aligned(x.grad, gquad) && aligned(x.copy, 8) &&
                     aligned(x.exp_avg, squad) && aligned(x.exp_avg_sq, squad);
    out[k] = {x.param, x.grad, x.copy, x.exp_avg, x.exp_avg_sq, x.exp_avg_scale, x.exp_avg_sq_scale,
              x.count, vec ? 1u : 0u, {0, 0, 0}};
    const uint64_t n = (x.count - 1) / ar::kAdamwTile + 1;
    for (uint64_t j = 0; j < n; ++j) *tile++ = {k, static_cast<uint32_t>(j)};
    ++k;
  }
  return AR_SUCCESS;
}

ar_status_t ar_adamw_grad_norm(const void* plan, void* device_plan, double max_norm,
                               double grad_scale, float* norm, hipStream_t stream) {
  const AdamwHead* h = static_cast<const AdamwHead*>(plan);
  if (!plan_ok(h, device_plan) || !(max_norm >= 0.0) || !std::isfinite(grad_scale) || !aligned(norm, 4))
    return AR_ERROR_INVALID_ARGUMENT;
  ar::AdamwNormArgs a;
  a.plan = static_cast<char*>(device_plan);
  a.sums_at = h->sums_at;
  a.tensors_at = h->tensors_at;
  a.tiles_at = h->tiles_at;
  a.tiles = h->tiles;
  a.max_norm = max_norm;
  a.grad_scale = grad_scale;
  a.norm = norm;
  return ar::launch_status(ar::enqueue(
      [&] { return ar::launch_adamw_norm(a, static_cast<ar_dtype_t>(h->grad_dtype), stream); }));
}

ar_status_t ar_adamw_step(const void* plan, void* device_plan, const ar_adamw_step_t* s,
                          hipStream_t stream) {
  const AdamwHead* h = static_cast<const AdamwHead*>(plan);
  if (!plan_ok(h, device_plan) || s == nullptr) return AR_ERROR_INVALID_ARGUMENT;
  const double all[] = {s->lr, s->beta1, s->beta2, s->eps, s->weight_decay, s->grad_scale};
  for (double x : all)
    if (!std::isfinite(x)) return AR_ERROR_INVALID_ARGUMENT;
  if (s->lr < 0 || s->eps < 0 || s->weight_decay < 0 || s->step < 1 || s->beta1 < 0 || s->beta1 >= 1 ||
      s->beta2 < 0 || s->beta2 >= 1)
    return AR_ERROR_INVALID_ARGUMENT;
  if (h->tiles == 0) return AR_SUCCESS;
  hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
  if (stream != nullptr && hipStreamIsCapturing(stream, &capture) == hipSuccess &&
      capture != hipStreamCaptureStatusNone)
    return AR_ERROR_UNSUPPORTED;

  ar::AdamwStepArgs a;
  a.plan = static_cast<char*>(device_plan);
  a.tensors_at = h->tensors_at;
  a.sums_at = h->sums_at;
  a.tiles_at = h->tiles_at;
  a.clip = s->clip != 0;
  a.factor = static_cast<float>(s->grad_scale);
  const double bc1 = 1.0 - std::pow(s->beta1, static_cast<double>(s->step));
  const double bc2 = 1.0 - std::pow(s->beta2, static_cast<double>(s->step));
  a.lr = static_cast<float>(s->lr * std::sqrt(bc2) / bc1);
  a.eps64 = s->eps * std::sqrt(bc2);
  a.eps = static_cast<float>(a.eps64);
  a.far = ar::wide_eps(a.eps64);
  a.lr_wd = static_cast<float>(s->lr * s->weight_decay);
  a.b1 = s->beta1;
  a.one_b1 = 1.0 - s->beta1;
  a.b2 = s->beta2;
  a.one_b2 = 1.0 - s->beta2;
  a.root_b2 = std::sqrt(a.b2);
  a.root_one_b2 = std::sqrt(a.one_b2);
  return ar::launch_status(ar::enqueue([&] {
    return ar::launch_adamw_step(a, h->tiles, static_cast<ar_dtype_t>(h->param_dtype),
                                 static_cast<ar_dtype_t>(h->grad_dtype), h->state_bits,
                                 h->has_copy != 0, h->touched <= ar::kKeepBytes, stream);
  }));
}

ar_status_t ar_adamw_dequantize(const void* codes, const float* scales, size_t count, int is_signed,
                                float* out, hipStream_t stream) {
  if (count == 0) return AR_SUCCESS;
  if (codes == nullptr || scales == nullptr || out == nullptr || !aligned(scales, 4) || !aligned(out, 4))
    return AR_ERROR_INVALID_ARGUMENT;
  const uintptr_t c = reinterpret_cast<uintptr_t>(codes), s = reinterpret_cast<uintptr_t>(scales);
  const uintptr_t o = reinterpret_cast<uintptr_t>(out);
  const uint64_t blocks = (count - 1) / AR_ADAMW_BLOCK + 1;
  if (count > (std::numeric_limits<uintptr_t>::max() - std::max(std::max(c, s), o)) / 4)
    return AR_ERROR_INVALID_ARGUMENT;
  if ((count - 1) / ar::kAdamwTile + 1 > ar::kAdamwMaxDecodeTiles) return AR_ERROR_UNSUPPORTED;
  const uintptr_t oe = o + count * 4;
  if ((c < oe && o < c + count) || (s < oe && o < s + blocks * 4)) return AR_ERROR_INVALID_ARGUMENT;
  return ar::launch_status(ar::enqueue(
      [&] { return ar::launch_adamw_dequantize(codes, scales, count, is_signed != 0, out, stream); }));
}

}  // extern "C"
