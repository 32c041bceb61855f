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

// Tiles are 128 wide from so many of X, and of X X^T, on: fewer leave CUs idle (one
// of 2,048 x 2,048, 136 squares: 866 us in 64, 924 in 128; four of 1,024 x 1,024 with
// two of 4,096 x 1,024, 216 squares: 1,170 and 1,050).
constexpr uint64_t kWideTiles = 256, kWideSquares = 160;

// Where every matrix has at most so many rows and columns, each goes a block in
// one launch: one of 100 x 61 24 us instead of 69 in tiles, of 128 x 128 65 instead
// of 82, 4,096 of them 1,275 instead of 2,695.
constexpr uint64_t kWhole = 128;

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

// Tiles of one matrix that lie together, in their order.
struct Group {
  uint32_t matrix, begin, end;
  uint32_t steps, parts;
};

// A matrix's tiles in an order in which neighbours share rows and columns: eight
// rows of tiles at a time, column by column.  `upper`: of a square, those on or
// above the diagonal.
constexpr uint32_t kBand = 8;
template <class F> void in_order(uint32_t height, uint32_t width, bool upper, F&& each) {
  for (uint32_t r0 = 0; r0 < height; r0 += kBand)
    for (uint32_t c = upper ? r0 : 0; c < width; ++c)
      for (uint32_t r = r0; r < std::min(height, r0 + kBand) && (!upper || r <= c); ++r) each(r, c);
}

struct Table {
  std::vector<MuonTile> tiles;
  uint32_t slots = 0, counters = 0;      // of the tiles in parts
  bool fits = true;
};

struct Layout {
  uint64_t matrices = 0, chunks = 0;
  uint32_t side = 0, square_side = 0;
  uint16_t longest = 0, shortest = 0;
  Table squares, polys, tiles;
  uint64_t matrices_at = 0, chunks_at = 0, squares_at = 0, polys_at = 0, tiles_at = 0, norms_at = 0, sums_at = 0,
           arrived_at = 0;
  uint64_t bytes = 0, workspace = 0, parts_at = 0;
  bool fits = true;
};

struct Counts {
  uint64_t matrices = 0, chunks = 0, squares = 0, tiles = 0;
  bool fits = true;
};

// Numbers of tiles of `side`.
Counts count_with(const ar_muon_tensor_t* t, int n, uint64_t side) {
  Counts l;
  for (int i = 0; i < n && l.fits; ++i) {
    if (empty(t[i])) continue;
    const uint64_t count = t[i].count, rows = t[i].rows, cols = t[i].cols;
    const uint64_t h = up(std::min(rows, cols), side) / side, w = up(std::max(rows, cols), side) / side;
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
    l.fits = l.chunks <= ar::kMuonMaxTiles && l.squares <= ar::kMuonMaxTiles && l.tiles <= ar::kMuonMaxTiles;
  }
  return l;
}

enum class Kind { kSquares, kPolys, kTiles };

// Blocks that run at a time, two on a CU.
constexpr uint64_t kPlaces = 512;

// A tile's k is split into at most so many parts (one block adds all of them up),
// none of less than kLeast steps: joining them takes as long as about ten.  One of
// 4,096 x 4,096: 4,063 us, 4,372 without parts, whose 528 squares would be two
// rounds; 16 of 256 x 4,096 561 and 609.  With parts of 8 steps 64 of 512 x 512 took
// 1,092 us instead of 907.
constexpr uint32_t kMostParts = 8, kLeast = 32;

// The parts of the tiles that are left when all places have had the same number
// of whole ones: as many as find a place, so that none of them idles while
// others have whole tiles left.  `left` of the tiles of `steps` each.
struct Rest {
  uint32_t steps;
  uint64_t left;
};
uint32_t parts_of(uint32_t steps, uint32_t each) {
  return std::min({kMostParts, (steps + each - 1) / each, std::max(1u, steps / kLeast)});
}
uint32_t steps_each(const std::vector<Rest>& rest, uint64_t room) {
  uint32_t each = kLeast;
  for (;; each += 1 + each / 8) {
    uint64_t parts = 0;
    bool whole = true;
    for (const Rest& r : rest) {
      parts += r.left * parts_of(r.steps, each);
      whole = whole && parts_of(r.steps, each) == 1;
    }
    if (parts <= room || whole) return each;
  }
}

// The table of a product: the tiles with most steps first, neighbours together,
// each group to the XCD that has least so far; entry i is XCD (i mod 8)'s, so
// lists of unequal lengths leave entries of no matrix.
Table deal(const ar_muon_tensor_t* t, int n, uint32_t pad, uint32_t side, Kind kind) {
  const bool upper = kind != Kind::kTiles;
  // each tensor's tiles in order
  std::vector<std::vector<MuonTile>> order;
  std::vector<uint32_t> steps_of, shape_of;        // of a tensor; of a matrix
  for (int i = 0; i < n; ++i) {
    if (empty(t[i])) continue;
    const uint64_t height = up(std::min(t[i].rows, t[i].cols), pad), width = up(std::max(t[i].rows, t[i].cols), pad);
    const uint32_t h = static_cast<uint32_t>(height / side), w = static_cast<uint32_t>(width / side);
    order.emplace_back();
    in_order(h, upper ? h : w, upper, [&](uint32_t r, uint32_t c) {
      MuonTile tile = {};
      tile.m = static_cast<uint16_t>(r);
      tile.n = static_cast<uint16_t>(c);
      order.back().push_back(tile);
    });
    steps_of.push_back(static_cast<uint32_t>((kind == Kind::kSquares ? width : height) / ar::kMuonStep));
    shape_of.insert(shape_of.end(), t[i].count, static_cast<uint32_t>(order.size() - 1));
  }
  std::vector<uint32_t> matrices(shape_of.size());
  for (uint32_t k = 0; k < matrices.size(); ++k) matrices[k] = k;
  std::stable_sort(matrices.begin(), matrices.end(),
                   [&](uint32_t a, uint32_t b) { return steps_of[shape_of[a]] > steps_of[shape_of[b]]; });

  // whole tiles up to a multiple of the places, parts of the others
  uint64_t total = 0, seen = 0;
  for (uint32_t shape : shape_of) total += order[shape].size();
  uint64_t whole = total - total % kPlaces;
  std::vector<Rest> rest;
  for (uint32_t k : matrices) {
    const uint64_t tiles = order[shape_of[k]].size();
    if (seen + tiles > whole) rest.push_back({steps_of[shape_of[k]], seen + tiles - std::max(seen, whole)});
    seen += tiles;
  }
  const uint32_t each = steps_each(rest, kPlaces);
  // groups small enough for the XCDs' loads to come out even
  const uint32_t most = static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>(32, total / (4 * ar::kMuonXcds))));
  std::vector<Group> groups;
  for (uint32_t k : matrices) {
    const uint32_t tiles = static_cast<uint32_t>(order[shape_of[k]].size()), steps = steps_of[shape_of[k]];
    const uint32_t kept = static_cast<uint32_t>(std::min<uint64_t>(whole, tiles));
    whole -= kept;
    for (uint32_t b = 0; b < kept; b += most) groups.push_back({k, b, std::min(kept, b + most), steps, 1});
    for (uint32_t b = kept; b < tiles; b += most)
      groups.push_back({k, b, std::min(tiles, b + most), steps, parts_of(steps, each)});
  }
  std::stable_sort(groups.begin(), groups.end(),
                   [](const Group& a, const Group& b) { return a.steps / a.parts > b.steps / b.parts; });

  Table table;
  std::vector<MuonTile> of[ar::kMuonXcds];
  uint64_t load[ar::kMuonXcds] = {};
  for (const Group& g : groups)
    for (uint32_t part = 0; part < g.parts; ++part) {
      // the same steps of neighbouring tiles have operands in common
      const size_t x = std::min_element(load, load + ar::kMuonXcds) - load;
      for (uint32_t j = g.begin; j < g.end; ++j) {
        MuonTile tile = order[shape_of[g.matrix]][j];
        tile.matrix = g.matrix;
        tile.first = static_cast<uint32_t>(static_cast<uint64_t>(g.steps) * part / g.parts);
        tile.steps = static_cast<uint32_t>(static_cast<uint64_t>(g.steps) * (part + 1) / g.parts) - tile.first;
        tile.part = part;
        tile.parts = g.parts;
        if (g.parts > 1) {
          tile.slot = table.slots + (j - g.begin) * g.parts;
          tile.counter = table.counters + (j - g.begin);
        }
        load[x] += tile.steps;
        of[x].push_back(tile);
      }
      if (g.parts > 1 && part + 1 == g.parts) {
        table.slots += (g.end - g.begin) * g.parts;
        table.counters += g.end - g.begin;
      }
    }
  size_t longest = 0;
  for (const auto& list : of) longest = std::max(longest, list.size());
  MuonTile none = {};
  none.matrix = ar::kMuonNoMatrix;
  table.tiles.assign(longest * ar::kMuonXcds, none);
  for (uint32_t x = 0; x < ar::kMuonXcds; ++x)
    for (size_t j = 0; j < of[x].size(); ++j) table.tiles[j * ar::kMuonXcds + x] = of[x][j];
  table.fits = table.tiles.size() <= ar::kMuonMaxTiles;
  return table;
}

Layout layout_of(const ar_muon_tensor_t* t, int n) {
  Layout l;
  const Counts wide = count_with(t, n, 128), narrow = count_with(t, n, 64);
  l.side = (wide.fits && wide.tiles >= kWideTiles) || !narrow.fits ? 128 : 64;
  l.square_side = l.side == 128 && (wide.squares >= kWideSquares || !narrow.fits) ? 128 : 64;
  const Counts& at = l.side == 128 ? wide : narrow;
  l.fits = at.fits;
  if (!l.fits) return l;
  l.matrices = at.matrices;
  l.chunks = at.chunks;
  l.squares = deal(t, n, l.side, l.square_side, Kind::kSquares);
  l.polys = deal(t, n, l.side, l.square_side, Kind::kPolys);
  l.tiles = deal(t, n, l.side, l.side, Kind::kTiles);
  l.fits = l.tiles.fits && l.squares.fits && l.polys.fits;
  for (int i = 0; i < n; ++i) {
    if (empty(t[i])) continue;
    const uint64_t height = up(std::min(t[i].rows, t[i].cols), l.side), width = up(std::max(t[i].rows, t[i].cols), l.side);
    l.workspace += t[i].count * (2 * up(height * width * 4, 256) + 2 * up(height * height * 4, 256));
  }
  uint64_t longest = 0, shortest = 0;
  for (int i = 0; i < n; ++i) {
    if (empty(t[i])) continue;
    longest = std::max<uint64_t>({longest, t[i].rows, t[i].cols});
    shortest = std::max<uint64_t>(shortest, std::min(t[i].rows, t[i].cols));
  }
  if (longest <= kWhole) {
    l.longest = longest > 64 ? 128 : 64;
    l.shortest = shortest > 64 ? 128 : 64;
  }
  l.parts_at = l.workspace;
  l.workspace += std::max({static_cast<uint64_t>(l.squares.slots) * l.square_side * l.square_side,
                           static_cast<uint64_t>(l.polys.slots) * l.square_side * l.square_side,
                           static_cast<uint64_t>(l.tiles.slots) * l.side * l.side}) *
                 sizeof(float);
  l.matrices_at = up(sizeof(MuonHead), 256);
  l.chunks_at = up(l.matrices_at + l.matrices * sizeof(MuonMatrix), 256);
  l.squares_at = up(l.chunks_at + l.chunks * sizeof(MuonChunk), 256);
  l.polys_at = up(l.squares_at + l.squares.tiles.size() * sizeof(MuonTile), 256);
  l.tiles_at = up(l.polys_at + l.polys.tiles.size() * sizeof(MuonTile), 256);
  l.norms_at = up(l.tiles_at + l.tiles.tiles.size() * sizeof(MuonTile), 256);
  l.sums_at = up(l.norms_at + l.matrices * sizeof(MuonNorm), 256);
  l.arrived_at = up(l.sums_at + l.chunks * sizeof(double), 256);
  l.bytes = up(l.arrived_at + std::max({l.squares.counters, l.polys.counters, l.tiles.counters}) * sizeof(uint32_t), 256);
  return l;
}

// No exception leaves a C entry: the host running out of memory is reported as a
// request that cannot be served.
ar_status_t layout_noexcept(const ar_muon_tensor_t* t, int n, ar_dtype_t pd, ar_dtype_t gd, Layout* l) {
  try {
    const ar_status_t st = check(t, n, pd, gd);
    if (st != AR_SUCCESS) return st;
    *l = layout_of(t, n);
    return l->fits ? AR_SUCCESS : AR_ERROR_UNSUPPORTED;
  } catch (const std::bad_alloc&) {
    return AR_ERROR_UNSUPPORTED;
  }
}

bool plan_ok(const MuonHead* h) { return h != nullptr && aligned(h, 8) && h->magic == ar::kMuonMagic; }

}  // namespace

extern "C" {

size_t ar_muon_plan_bytes(const ar_muon_tensor_t* tensors, int ntensors, ar_dtype_t param_dtype,
                          ar_dtype_t grad_dtype) {
  Layout l;
  return layout_noexcept(tensors, ntensors, param_dtype, grad_dtype, &l) == AR_SUCCESS ? l.bytes : 0;
}

ar_status_t ar_muon_plan(const ar_muon_tensor_t* tensors, int ntensors, ar_dtype_t param_dtype,
                         ar_dtype_t grad_dtype, void* plan, size_t bytes) {
  Layout l;
  const ar_status_t st = layout_noexcept(tensors, ntensors, param_dtype, grad_dtype, &l);
  if (st != AR_SUCCESS) return st;
  if (plan == nullptr || bytes < l.bytes || !aligned(plan, 8)) return AR_ERROR_INVALID_ARGUMENT;

  char* base = static_cast<char*>(plan);
  std::memset(base, 0, l.bytes);
  MuonHead* h = reinterpret_cast<MuonHead*>(base);
  h->magic = ar::kMuonMagic;
  h->matrices = static_cast<uint32_t>(l.matrices);
  h->chunks = static_cast<uint32_t>(l.chunks);
  h->squares = static_cast<uint32_t>(l.squares.tiles.size());
  h->polys = static_cast<uint32_t>(l.polys.tiles.size());
  h->tiles = static_cast<uint32_t>(l.tiles.tiles.size());
  h->side = l.side;
  h->square_side = l.square_side;
  h->longest = l.longest;
  h->shortest = l.shortest;
  h->param_dtype = param_dtype;
  h->grad_dtype = grad_dtype;
  h->bytes = l.bytes;
  h->workspace = l.workspace;
  h->matrices_at = l.matrices_at;
  h->chunks_at = l.chunks_at;
  h->squares_at = l.squares_at;
  h->polys_at = l.polys_at;
  h->tiles_at = l.tiles_at;
  h->norms_at = l.norms_at;
  h->sums_at = l.sums_at;
  h->arrived_at = l.arrived_at;
  h->parts_at = l.parts_at;
  MuonMatrix* matrix = reinterpret_cast<MuonMatrix*>(base + l.matrices_at);
  MuonChunk* chunk = reinterpret_cast<MuonChunk*>(base + l.chunks_at);
  std::copy(l.squares.tiles.begin(), l.squares.tiles.end(), reinterpret_cast<MuonTile*>(base + l.squares_at));
  std::copy(l.polys.tiles.begin(), l.polys.tiles.end(), reinterpret_cast<MuonTile*>(base + l.polys_at));
  std::copy(l.tiles.tiles.begin(), l.tiles.tiles.end(), reinterpret_cast<MuonTile*>(base + l.tiles_at));
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
      m.flat = aligned(m.g, 4 * size_of(grad_dtype)) && aligned(m.m, 16);
      m.vec = m.flat && x.cols % 4 == 0 && aligned(m.p, 4 * size_of(param_dtype)) && aligned(m.copy, 8);
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
    }
  }
  return AR_SUCCESS;
}

size_t ar_muon_workspace(const void* plan) {
  const MuonHead* h = static_cast<const MuonHead*>(plan);
  return plan_ok(h) ? h->workspace : 0;
}

size_t ar_muon_workspace_used(const void* plan) {
  const MuonHead* h = static_cast<const MuonHead*>(plan);
  return plan_ok(h) && h->longest == 0 ? h->workspace : 0;
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
  a.polys_at = h->polys_at;
  a.tiles_at = h->tiles_at;
  a.norms_at = h->norms_at;
  a.sums_at = h->sums_at;
  a.arrived_at = h->arrived_at;
  a.parts_at = h->parts_at;
  a.momentum = static_cast<float>(s->momentum);
  a.grad_scale = static_cast<float>(s->grad_scale);
  a.lr = static_cast<float>(s->lr);
  a.lr_wd = static_cast<float>(s->lr * s->weight_decay);
  a.eps = s->eps;
  // (0 is none, so what float32 cannot hold becomes the smallest that it can)
  a.rms = s->match_rms > 0
              ? std::max(static_cast<float>(s->match_rms), std::numeric_limits<float>::denorm_min())
              : 0.0f;
  a.nesterov = s->nesterov != 0;
  a.last = 0;
  a.from = 0;
  a.steps = s->ns_steps;
  const ar_dtype_t pd = static_cast<ar_dtype_t>(h->param_dtype), gd = static_cast<ar_dtype_t>(h->grad_dtype);
  if (h->longest != 0)
    return ar::launch_status(ar::enqueue([&] {
      return ar::launch_muon_whole(a, h->matrices, h->longest, h->shortest, pd, gd, h->has_copy != 0, stream);
    }));
  hipError_t err = ar::enqueue([&] { return ar::launch_muon_momentum(a, h->chunks, gd, stream); });
  if (err == hipSuccess)
    err = ar::enqueue([&] { return ar::launch_muon_start(a, h->tiles, h->side, gd, stream); });
  for (int i = 0; i < s->ns_steps && err == hipSuccess; ++i) {
    a.last = i + 1 == s->ns_steps;
    a.from = i & 1;
    err = ar::enqueue([&] { return ar::launch_muon_gram(a, h->squares, h->square_side, stream); });
    if (err == hipSuccess) err = ar::enqueue([&] { return ar::launch_muon_poly(a, h->polys, h->square_side, stream); });
    if (err == hipSuccess)
      err = ar::enqueue([&] { return ar::launch_muon_apply(a, h->tiles, h->side, pd, h->has_copy != 0, stream); });
  }
  return ar::launch_status(err);
}

}  // extern "C"
