// C entry points of the Muon step: checks, plans, hyperparameters.
#include "train/muon.hpp"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>
#include <new>
#include <vector>

#include "launch.hpp"

namespace {

using ar::MuonChunk;
using ar::MuonHead;
using ar::MuonMatrix;
using ar::MuonNorm;
using ar::MuonTile;

constexpr uint64_t kMost = std::numeric_limits<uintptr_t>::max();

constexpr uint64_t up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

uint64_t size_of(ar_dtype_t t) { return t == AR_FLOAT32 ? 4 : 2; }

bool empty(const ar_muon_tensor_t& t) { return t.count == 0 || t.rows == 0 || t.cols == 0; }

struct Range {
  uintptr_t lo, hi;
  bool written;
};

// All of the tensors' checks but the number of tiles.
ar_status_t check(const ar_muon_tensor_t* t, int n, ar_dtype_t pd, ar_dtype_t gd) {
  if (t == nullptr || n < 1) return AR_ERROR_INVALID_ARGUMENT;
  if ((pd != AR_FLOAT32 && pd != AR_BFLOAT16) || (gd != AR_FLOAT32 && gd != AR_BFLOAT16)) return AR_ERROR_UNSUPPORTED;
  std::vector<Range> ranges;
  bool first = true, copies = false;
  for (int i = 0; i < n; ++i) {
    const ar_muon_tensor_t& x = t[i];
    if (empty(x)) continue;
    if (x.param == nullptr || x.grad == nullptr || x.momentum == nullptr || !aligned(x.param, size_of(pd)) ||
        !aligned(x.grad, size_of(gd)) || !aligned(x.momentum, 4) || !aligned(x.copy, 2))
      return AR_ERROR_INVALID_ARGUMENT;
    if (first) copies = x.copy != nullptr;
    first = false;
    if ((x.copy != nullptr) != copies || (copies && pd != AR_FLOAT32)) return AR_ERROR_INVALID_ARGUMENT;
    if (x.rows > ar::kMuonMaxElements || x.cols > ar::kMuonMaxElements ||
        up(x.rows, 128) * up(x.cols, 128) > ar::kMuonMaxElements ||
        up(std::min(x.rows, x.cols), 128) > 65535 * 64ull || up(std::max(x.rows, x.cols), 128) > 65535 * 64ull)
      return AR_ERROR_UNSUPPORTED;
    const uint64_t each = static_cast<uint64_t>(x.rows) * x.cols;
    if (x.count > kMost / 4 / each) return AR_ERROR_INVALID_ARGUMENT;
    const uint64_t count = x.count * each;
    const auto add = [&](const void* p, uint64_t size, bool written) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
      if (count > (kMost - lo) / size) return false;
      ranges.push_back({lo, lo + count * size, written});
      return true;
    };
    if (!add(x.param, size_of(pd), true) || !add(x.grad, size_of(gd), false) || !add(x.momentum, 4, true) ||
        (copies && !add(x.copy, 2, true)))
      return AR_ERROR_INVALID_ARGUMENT;
  }
  // no written range may meet another (see the AdamW plan)
  std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end_all = 0, end_written = 0;
  for (const Range& r : ranges) {
    if (r.lo < end_written || (r.written && r.lo < end_all)) return AR_ERROR_INVALID_ARGUMENT;
    end_all = std::max(end_all, r.hi);
    if (r.written) end_written = std::max(end_written, r.hi);
  }
  return AR_SUCCESS;
}

ar_status_t check_noexcept(const ar_muon_tensor_t* t, int n, ar_dtype_t pd, ar_dtype_t gd) {
  try {
    return check(t, n, pd, gd);
  } catch (const std::bad_alloc&) {
    return AR_ERROR_UNSUPPORTED;
  }
}

struct Layout {
  uint64_t matrices = 0, chunks = 0, squares = 0, tiles = 0, side = 0;
  uint64_t matrices_at = 0, chunks_at = 0, squares_at = 0, tiles_at = 0, norms_at = 0, sums_at = 0;
  uint64_t bytes = 0, workspace = 0;
  bool fits = true;
};

// Sizes with tiles of `side`.
Layout layout_with(const ar_muon_tensor_t* t, int n, uint64_t side) {
  Layout l;
  l.side = side;
  for (int i = 0; i < n && l.fits; ++i) {
    if (empty(t[i])) continue;
    const uint64_t count = t[i].count, rows = t[i].rows, cols = t[i].cols;
    const uint64_t height = up(std::min(rows, cols), side), width = up(std::max(rows, cols), side);
    const uint64_t h = height / side, w = width / side;
    const uint64_t chunks = (rows * cols - 1) / ar::kMuonChunk + 1;
    // every count below is bounded by these before it is multiplied
    if (count > ar::kMuonMaxTiles / std::max({h * (h + 1) / 2, h * w, chunks})) {
      l.fits = false;
      break;
    }
    l.matrices += count;
    l.chunks += count * chunks;
    l.squares += count * (h * (h + 1) / 2);
    l.tiles += count * h * w;
    l.workspace += count * (2 * up(height * width * 4, 256) + 2 * up(height * height * 4, 256));
    l.fits = l.chunks <= ar::kMuonMaxTiles && l.squares <= ar::kMuonMaxTiles && l.tiles <= ar::kMuonMaxTiles;
  }
  l.matrices_at = up(sizeof(MuonHead), 256);
  l.chunks_at = up(l.matrices_at + l.matrices * sizeof(MuonMatrix), 256);
  l.squares_at = up(l.chunks_at + l.chunks * sizeof(MuonChunk), 256);
  l.tiles_at = up(l.squares_at + l.squares * sizeof(MuonTile), 256);
  l.norms_at = up(l.tiles_at + l.tiles * sizeof(MuonTile), 256);
  l.sums_at = up(l.norms_at + l.matrices * sizeof(MuonNorm), 256);
  l.bytes = up(l.sums_at + l.chunks * sizeof(double), 256);
  return l;
}

Layout layout_of(const ar_muon_tensor_t* t, int n) {
  const Layout wide = layout_with(t, n, 128);
  if (wide.fits && wide.squares >= 128) return wide;
  const Layout narrow = layout_with(t, n, 64);
  return narrow.fits ? narrow : wide;
}

bool plan_ok(const MuonHead* h) { return h != nullptr && aligned(h, 8) && h->magic == ar::kMuonMagic; }

}  // namespace

extern "C" {

size_t ar_muon_plan_bytes(const ar_muon_tensor_t* tensors, int ntensors, ar_dtype_t param_dtype,
                          ar_dtype_t grad_dtype) {
  if (check_noexcept(tensors, ntensors, param_dtype, grad_dtype) != AR_SUCCESS) return 0;
  const Layout l = layout_of(tensors, ntensors);
  return l.fits ? l.bytes : 0;
}

ar_status_t ar_muon_plan(const ar_muon_tensor_t* tensors, int ntensors, ar_dtype_t param_dtype,
                         ar_dtype_t grad_dtype, void* plan, size_t bytes) {
  const ar_status_t st = check_noexcept(tensors, ntensors, param_dtype, grad_dtype);
  if (st != AR_SUCCESS) return st;
  const Layout l = layout_of(tensors, ntensors);
  if (!l.fits) return AR_ERROR_UNSUPPORTED;
  if (plan == nullptr || bytes < l.bytes || !aligned(plan, 8)) return AR_ERROR_INVALID_ARGUMENT;

  char* base = static_cast<char*>(plan);
  std::memset(base, 0, l.bytes);
  MuonHead* h = reinterpret_cast<MuonHead*>(base);
  h->magic = ar::kMuonMagic;
  h->matrices = static_cast<uint32_t>(l.matrices);
  h->chunks = static_cast<uint32_t>(l.chunks);
  h->squares = static_cast<uint32_t>(l.squares);
  h->tiles = static_cast<uint32_t>(l.tiles);
  h->side = static_cast<uint32_t>(l.side);
  h->param_dtype = param_dtype;
  h->grad_dtype = grad_dtype;
  h->bytes = l.bytes;
  h->workspace = l.workspace;
  h->matrices_at = l.matrices_at;
  h->chunks_at = l.chunks_at;
  h->squares_at = l.squares_at;
  h->tiles_at = l.tiles_at;
  h->norms_at = l.norms_at;
  h->sums_at = l.sums_at;
  MuonMatrix* matrix = reinterpret_cast<MuonMatrix*>(base + l.matrices_at);
  MuonChunk* chunk = reinterpret_cast<MuonChunk*>(base + l.chunks_at);
  MuonTile* square = reinterpret_cast<MuonTile*>(base + l.squares_at);
  MuonTile* tile = reinterpret_cast<MuonTile*>(base + l.tiles_at);
  uint32_t k = 0, chunks = 0;
  uint64_t at = 0;
  for (int i = 0; i < ntensors; ++i) {
    const ar_muon_tensor_t& x = tensors[i];
    if (empty(x)) continue;
    h->has_copy = x.copy != nullptr;
    const uint64_t each = static_cast<uint64_t>(x.rows) * x.cols;
    for (uint64_t c = 0; c < x.count; ++c, ++k) {
      MuonMatrix& m = matrix[k];
      m.p = static_cast<char*>(x.param) + c * each * size_of(param_dtype);
      m.g = static_cast<const char*>(x.grad) + c * each * size_of(grad_dtype);
      m.copy = x.copy == nullptr ? nullptr : static_cast<char*>(x.copy) + c * each * 2;
      m.m = x.momentum + c * each;
      m.rows = static_cast<uint32_t>(x.rows);
      m.cols = static_cast<uint32_t>(x.cols);
      m.tall = x.rows > x.cols;
      m.height = static_cast<uint32_t>(up(std::min(x.rows, x.cols), l.side));
      m.width = static_cast<uint32_t>(up(std::max(x.rows, x.cols), l.side));
      m.x_plane = static_cast<uint64_t>(m.height) * m.width * 2;
      m.gram_plane = static_cast<uint64_t>(m.height) * m.height * 2;
      for (uint64_t* to : {&m.x[0], &m.x[1]}) {
        *to = at;
        at += up(2 * m.x_plane, 256);
      }
      for (uint64_t* to : {&m.gram, &m.poly}) {
        *to = at;
        at += up(2 * m.gram_plane, 256);
      }
      m.first_chunk = chunks;
      m.chunks = static_cast<uint32_t>((each - 1) / ar::kMuonChunk + 1);
      chunks += m.chunks;
      const double r = static_cast<double>(x.rows), w = static_cast<double>(x.cols);
      m.by_shape = static_cast<float>(std::sqrt(std::max(1.0, r / w)));
      m.by_size = static_cast<float>(std::sqrt(std::max(r, w)));
      for (uint32_t j = 0; j < m.chunks; ++j) *chunk++ = {k, j};
      const uint32_t hs = m.height / h->side, ws = m.width / h->side;
      for (uint32_t r0 = 0; r0 < hs; ++r0) {
        for (uint32_t c0 = r0; c0 < hs; ++c0) *square++ = {k, static_cast<uint16_t>(r0), static_cast<uint16_t>(c0)};
        for (uint32_t c0 = 0; c0 < ws; ++c0) *tile++ = {k, static_cast<uint16_t>(r0), static_cast<uint16_t>(c0)};
      }
    }
  }
  return AR_SUCCESS;
}

size_t ar_muon_workspace(const void* plan) {
  const MuonHead* h = static_cast<const MuonHead*>(plan);
  return plan_ok(h) ? h->workspace : 0;
}

ar_status_t ar_muon_step(const void* plan, void* device_plan, void* workspace, const ar_muon_step_t* s,
                         hipStream_t stream) {
  const MuonHead* h = static_cast<const MuonHead*>(plan);
  if (!plan_ok(h) || device_plan == nullptr || !aligned(device_plan, 256) || s == nullptr)
    return AR_ERROR_INVALID_ARGUMENT;
  const double all[] = {s->lr, s->momentum, s->eps, s->weight_decay, s->grad_scale, s->match_rms};
  for (double x : all)
    if (!std::isfinite(x)) return AR_ERROR_INVALID_ARGUMENT;
  if (s->lr < 0 || s->momentum < 0 || s->momentum >= 1 || s->eps < 0 || s->weight_decay < 0 || s->match_rms < 0 ||
      s->ns_steps < 1 || s->ns_steps > ar::kMuonMaxSteps)
    return AR_ERROR_INVALID_ARGUMENT;
  if (h->matrices == 0) return AR_SUCCESS;
  if (workspace == nullptr || !aligned(workspace, 256)) return AR_ERROR_INVALID_ARGUMENT;

  ar::MuonStepArgs a;
  a.plan = static_cast<char*>(device_plan);
  a.workspace = static_cast<char*>(workspace);
  a.matrices_at = h->matrices_at;
  a.chunks_at = h->chunks_at;
  a.squares_at = h->squares_at;
  a.tiles_at = h->tiles_at;
  a.norms_at = h->norms_at;
  a.sums_at = h->sums_at;
  a.momentum = static_cast<float>(s->momentum);
  a.grad_scale = static_cast<float>(s->grad_scale);
  a.lr = static_cast<float>(s->lr);
  a.lr_wd = static_cast<float>(s->lr * s->weight_decay);
  a.eps = s->eps;
  a.rms = static_cast<float>(s->match_rms);
  a.nesterov = s->nesterov != 0;
  a.last = 0;
  a.from = 0;
  const ar_dtype_t pd = static_cast<ar_dtype_t>(h->param_dtype), gd = static_cast<ar_dtype_t>(h->grad_dtype);
  hipError_t err = ar::enqueue([&] { return ar::launch_muon_momentum(a, h->chunks, gd, stream); });
  if (err == hipSuccess)
    err = ar::enqueue([&] { return ar::launch_muon_start(a, h->tiles, h->side, gd, stream); });
  for (int i = 0; i < s->ns_steps && err == hipSuccess; ++i) {
    a.last = i + 1 == s->ns_steps;
    a.from = i & 1;
    err = ar::enqueue([&] { return ar::launch_muon_gram(a, h->squares, h->side, stream); });
    if (err == hipSuccess) err = ar::enqueue([&] { return ar::launch_muon_poly(a, h->squares, h->side, stream); });
    if (err == hipSuccess)
      err = ar::enqueue([&] { return ar::launch_muon_apply(a, h->tiles, h->side, pd, h->has_copy != 0, stream); });
  }
  return ar::launch_status(err);
}

}  // extern "C"
