// Matrix products grouped by expert, and the gradient of the experts' weights
// (gfx950).
#include "train/experts.hpp"

#include <algorithm>

#include "train/tile.hpp"
#include "train/wave.hpp"

namespace ar {
namespace {

// Eight elements of 16 bits, four of 32, at any element's address.
struct __attribute__((packed, aligned(2))) Chunk {
  u32x4 v;
};
struct __attribute__((packed, aligned(4))) Four {
  f32x4 v;
};

__device__ __forceinline__ uint32_t clamped(int32_t x, uint32_t lo, uint32_t hi) {
  return min(max(static_cast<uint32_t>(max(x, 0)), lo), hi);
}

// The pairs of expert e in order; of expert `experts` those that have none.
__device__ __forceinline__ void rows_of(const int32_t* offsets, int experts, int e, uint32_t pairs, uint32_t* lo,
                                        uint32_t* hi) {
  *lo = clamped(offsets[e], 0, pairs);
  *hi = e < experts ? clamped(offsets[e + 1], *lo, pairs) : pairs;
}

// Up to 8 elements of 16 bits at any element's address, zeros for the others.
__device__ __forceinline__ u32x4 read_elements(const uint16_t* p, int n) {
  u32x4 r = {0, 0, 0, 0};
  if (n >= 8) return reinterpret_cast<const Chunk*>(p)->v;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) r[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i % 2));
  return r;
}

// The chunk of elements e to e + 7 of a line of `length`, in two steps, so that
// many loads can be under way without a branch between them: a chunk over the
// line's end is read from its last 8 elements, and shifted into place when the
// values have come.  Lines of less than 8 are read element by element.
__device__ __forceinline__ u32x4 fetch(const uint16_t* line, uint32_t e, uint32_t length) {
  if (length < 8) return read_elements(line + e, e < length ? static_cast<int>(length - e) : 0);
  return reinterpret_cast<const Chunk*>(line + min(e, length - 8))->v;
}
// `ends`: whether a chunk of the step may lie over its line's end.
__device__ __forceinline__ u32x4 in_place(u32x4 v, bool valid, bool ends, uint32_t e, uint32_t length) {
  if (ends && length >= 8) {
    const uint32_t over = e + 8 > length ? min(e + 8 - length, 8u) : 0;      // elements past the end
    uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32, hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
    if (over & 4) {
      lo = hi;
      hi = 0;
    }
    const uint32_t bits = over % 4 * 16;
    if (bits != 0) {
      lo = lo >> bits | hi << (64 - bits);
      hi >>= bits;
    }
    if (over == 8) lo = hi = 0;
    v = u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
              static_cast<uint32_t>(hi >> 32)};
  }
  return valid ? v : u32x4{0, 0, 0, 0};
}

__device__ __forceinline__ uint32_t two_bf16(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) __bf16 two;
  two t = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, t);
}

// Rows and columns of a block's tile, its waves along each, the k of a step, the
// waves on a SIMD and the steps in LDS.
template <int M_, int N_, int WAVES_M, int WAVES_N, int STEP_, int PER_SIMD, int STAGES_> struct Tile {
  static constexpr int M = M_, N = N_, STEP = STEP_, kPerSimd = PER_SIMD, STAGES = STAGES_;
  static constexpr int kThreads = WAVES_M * WAVES_N * kWave;
  static constexpr int kPartM = M / WAVES_M, kPartN = N / WAVES_N;      // of a wave
  static constexpr int kM = kPartM / 16, kN = kPartN / 16;
  static __device__ __forceinline__ int row0(int wave) { return wave / WAVES_N * kPartM; }
  static __device__ __forceinline__ int column0(int wave) { return wave % WAVES_N * kPartN; }
};
// Two blocks of eight waves on a CU.  131,072 x 1,024 by k = 2,048: 1,099 TFLOP/s;
// 128 x 128 976; 256 x 256 1,120, but an expert's last rows fill 128 more often.
// Weights come from HBM, each expert's for a few tiles only, so products keep two
// steps under way: 131,072 pairs of 128 experts 695 us instead of 712, 8,192 of 64
// 75 instead of 79.
using Large = Tile<128, 256, 2, 4, 32, 4, 3>;
// One block of 256 x 256 moves less through L2 and LDS, which tells where rows
// fill it and the weights' columns are read along k: 131,072 pairs of 128 experts
// 723 us instead of 764, of 8 experts 548 instead of 620.  (With rows of k 672
// against 675 and 490 against 508, but 159 against 148 for k = 1,024.)
using Huge = Tile<256, 256, 2, 4, 64, 2, 2>;
using LargeGrad = Tile<128, 256, 2, 4, 32, 4, 2>;
// Two steps under way for the rows of many experts, of which few come from L2: 131,072
// pairs of 128 experts, 2,048 x 1,024, 785 us instead of 826.  Where an expert has fewer
// rows or a smaller matrix they cost 2 % (32 and 64 experts, 32,768 pairs, 1,024 x 2,048,
// 202 instead of 199 and 228 instead of 222), for 16 experts 9 % (16,384 pairs, 2,048 x
// 2,048, 202 instead of 185).
using DeepGrad = Tile<128, 256, 2, 4, 32, 4, 3>;
using Middle = Tile<128, 128, 2, 2, 64, 2, 2>;
// The weights' gradient of odd sizes: its blocks wait for loads and stores, so many
// small ones.  4,084 pairs of 61 experts, 515 x 1,030, 36 us, 46 in Middle; 16,336
// pairs 76 and 99.
using OddGrad = Tile<64, 128, 2, 2, 32, 4, 2>;
using Small = Tile<64, 128, 2, 2, 64, 3, 2>;

__device__ __forceinline__ uint32_t token_of(const TokenOf& t, uint32_t pair) {
  if (t.top_k == 1) return pair;
  return t.reciprocal != 0 ? __umulhi(pair, t.reciprocal) : pair / t.top_k;
}

// What lies at an address that is the same in all lanes, by a scalar load.
__device__ __forceinline__ uint32_t scalar(const int32_t* p) {
  typedef const __attribute__((address_space(4))) int32_t* Constant;
  const uint64_t at = reinterpret_cast<uintptr_t>(p);
  // (the builtin gives an int, whose sign must not reach the upper half)
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32));
  const uint64_t uniform = static_cast<uint64_t>(hi) << 32 | lo;
  return static_cast<uint32_t>(*reinterpret_cast<Constant>(uniform));
}

constexpr uint32_t kXcds = 8;

// Blocks come to the XCDs in turn; of `n` tiles in order each XCD gets
// neighbours, which share operands in its L2.
__device__ __forceinline__ uint32_t near_tile(uint32_t block, uint32_t n) {
  const uint32_t x = block % kXcds;
  return x * (n / kXcds) + min(x, n % kXcds) + block / kXcds;
}

// --- products ----------------------------------------------------------------------

// A block's part: rows [m0, hi) of expert e, columns from n0.
struct Part {
  int e;
  uint32_t m0, hi, n0;
};

// Cuts the experts' pairs (and those without one, as a last group) into tiles of
// M rows and gives the block its one; false for blocks past the last.  Every
// lane counts some neighbouring groups.
template <int M, int N> __device__ __forceinline__ bool part_of(const ProductArgs& a, Part* part) {
  const int lane = threadIdx.x % kWave, groups = a.experts + 1, each = (groups + kWave - 1) / kWave;
  const auto tiles = [&](int e) {
    uint32_t lo, hi;
    rows_of(a.offsets, a.experts, e, a.pairs, &lo, &hi);
    return (hi - lo + M - 1) / M;
  };
  uint32_t mine = 0;
  for (int i = 0; i < each; ++i)
    if (lane * each + i < groups) mine += tiles(lane * each + i);
  uint32_t upto = mine;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint32_t up = __shfl_up(upto, d);
    if (lane >= d) upto += up;
  }
  const uint64_t total = static_cast<uint64_t>(__shfl(upto, kWave - 1)) * a.tiles_n;
  if (blockIdx.x >= total) return false;
  const uint32_t tile = near_tile(blockIdx.x, static_cast<uint32_t>(total)), unit = tile / a.tiles_n;
  const int owner = __popcll(__ballot(upto <= unit));
  uint32_t rest = unit - __shfl(upto - mine, owner);
  int e = owner * each;
  for (uint32_t n; rest >= (n = tiles(e)); ++e) rest -= n;
  uint32_t lo, hi;
  rows_of(a.offsets, a.experts, e, a.pairs, &lo, &hi);
  part->e = __builtin_amdgcn_readfirstlane(e);
  part->m0 = __builtin_amdgcn_readfirstlane(lo + rest * M);
  part->hi = __builtin_amdgcn_readfirstlane(hi);
  part->n0 = tile % a.tiles_n * N;
  return true;
}

// Up to 16 bytes of a row from column n on (of `size`), PAST the caches or not.
template <bool PAST>
__device__ __forceinline__ void write_values(uint16_t* row, uint32_t n, uint32_t size, f32x4 lo, f32x4 hi) {
  const u32x4 r = {two_bf16(lo[0], lo[1]), two_bf16(lo[2], lo[3]), two_bf16(hi[0], hi[1]), two_bf16(hi[2], hi[3])};
  if (n + 8 <= size) {
    if (PAST)
      __builtin_nontemporal_store(r, &reinterpret_cast<Chunk*>(row + n)->v);
    else
      reinterpret_cast<Chunk*>(row + n)->v = r;
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (n + q < size) row[n + q] = static_cast<uint16_t>(r[q / 2] >> (16 * (q % 2)));
  }
}
template <bool PAST>
__device__ __forceinline__ void write_values(float* row, uint32_t n, uint32_t size, f32x4 v) {
  if (n + 4 <= size) {
    if (PAST)
      __builtin_nontemporal_store(v, &reinterpret_cast<Four*>(row + n)->v);
    else
      reinterpret_cast<Four*>(row + n)->v = v;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < size) row[n + q] = v[q];
  }
}

// Stores a wave's part, kM x kN fragments from row m0 and column n0 on, of a
// matrix of `rows` x `size`.  Each 16 rows go through LDS (the wave's own
// kTurnBytes), so that neighbouring lanes store neighbouring pieces: whole cache
// lines at a time, which the caches need not hold (PAST).  The weights' gradient
// of 8,192 pairs of 64 experts, 1,024 x 2,048: 205 us with each lane storing what
// it has, 150 so, 124 past the caches.
constexpr int kTurnPitch = 64 + 4;
constexpr int kTurnBytes = 16 * kTurnPitch * sizeof(float);

template <bool PAST, int TM, int TN, class OUT>
__device__ __forceinline__ void write_part(const f32x4 (&acc)[TM][TN], float* turn, OUT* to, uint32_t m0, uint32_t rows,
                                           uint32_t n0, uint32_t size, int lane) {
  constexpr int kEach = 16 / sizeof(OUT), kLanes = 64 / kEach;      // values a lane, lanes a row
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int group = 0; group < TN / 4; ++group) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4*>(turn + lane % 16 * kTurnPitch + column(j, lane / 16)) = acc[i][4 * group + j];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int r0 = 0; r0 < 16; r0 += kWave / kLanes) {
        const int r = r0 + lane / kLanes, c = lane % kLanes * kEach;
        const uint32_t m = m0 + 16 * i + r, n = n0 + 64 * group + c;
        const f32x4* v = reinterpret_cast<const f32x4*>(turn + r * kTurnPitch + c);
        if (m < rows && n < size) {
          OUT* row = to + static_cast<uint64_t>(m) * size;
          if constexpr (sizeof(OUT) == 2)
            write_values<PAST>(row, n, size, v[0], v[1]);
          else
            write_values<PAST>(row, n, size, v[0]);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// A thread's chunks of the steps of a product: where they come from in x and in
// the expert's matrix, and how much of each lies in them.  Chunk j of thread t is
// slot j * T::kThreads + t of the step.
template <class T, class SA, class SB, bool BR> struct Operands {
  static constexpr int kA = SA::kChunks / T::kThreads, kB = SB::kChunks / T::kThreads;
  uint32_t row[kA], at[kA];       // kNowhere for no row; first k of a step
  uint32_t line[kB], first[kB];   // line of a step, first element along it
  uint32_t n0;

  __device__ __forceinline__ Operands(const ProductArgs& a, const Part& p, int thread) : n0(p.n0) {
#pragma unroll
    for (int j = 0; j < kA; ++j) {
      const int slot = j * T::kThreads + thread, l = slot / SA::kPerLine;
      const uint32_t r = p.m0 + l;
      row[j] = kNowhere;
      at[j] = SA::place(l, slot % SA::kPerLine) * 8;
      if (p.e < a.experts && r < p.hi) {
        const uint32_t t = a.order == nullptr ? r : token_of(a.token, static_cast<uint32_t>(a.order[r]));
        if (t < a.x_rows) row[j] = t;
      }
    }
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      const int slot = j * T::kThreads + thread;
      line[j] = slot / SB::kPerLine;
      first[j] = SB::place(line[j], slot % SB::kPerLine) * 8;
    }
  }
  // elements of chunk j, from k on, that lie in the operand
  __device__ __forceinline__ int left_a(const ProductArgs& a, int j, uint32_t k) const {
    return row[j] == kNowhere || k + at[j] >= a.in ? 0 : static_cast<int>(min(a.in - k - at[j], 8u));
  }
  __device__ __forceinline__ int left_b(const ProductArgs& a, int j, uint32_t k) const {
    const uint32_t kk = k + (BR ? line[j] : first[j]), n = n0 + (BR ? first[j] : line[j]);
    if (kk >= a.in || n >= a.out) return 0;
    return static_cast<int>(min(BR ? a.out - n : a.in - kk, 8u));
  }
  // straight to LDS: `to` is the wave's first chunk of the step, the waves' chunks
  // of one j follow one another
  __device__ __forceinline__ void issue(const ProductArgs& a, const Source& x, const Source& w, int step,
                                        char* to) const {
    const uint32_t k = step * T::STEP, lds = lds_address(to);
    const uint32_t x_bytes = static_cast<uint32_t>(a.x_stride) * 2, w_bytes = static_cast<uint32_t>(a.w_line) * 2;
#pragma unroll
    for (int j = 0; j < kA; ++j)
      load_to_lds(x, left_a(a, j, k) ? row[j] * x_bytes + (k + at[j]) * 2 : kNowhere,
                  __builtin_amdgcn_readfirstlane(lds + j * T::kThreads * 16));
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      const uint32_t at_line = BR ? k + line[j] : n0 + line[j], along = BR ? n0 + first[j] : k + first[j];
      load_to_lds(w, left_b(a, j, k) ? at_line * w_bytes + along * 2 : kNowhere,
                  __builtin_amdgcn_readfirstlane(lds + SA::kBytes + j * T::kThreads * 16));
    }
  }
  // through registers
  struct Held {
    u32x4 a[kA], b[kB];
  };
  __device__ __forceinline__ void load(const ProductArgs& a, const uint16_t* w, int step, Held* h) const {
    const uint32_t k = step * T::STEP;
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
#pragma unroll
    for (int j = 0; j < kA; ++j) h->a[j] = fetch(x + (row[j] == kNowhere ? 0 : row[j]) * a.x_stride, k + at[j], a.in);
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      const uint32_t l = (BR ? k : n0) + line[j], lines = BR ? a.in : a.out;
      h->b[j] = fetch(w + (l < lines ? l : 0) * a.w_line, (BR ? n0 : k) + first[j], BR ? a.out : a.in);
    }
  }
  __device__ __forceinline__ void put(const ProductArgs& a, const Held& h, int step, char* stage, int thread) const {
    const uint32_t k = step * T::STEP;
    const bool end_k = k + T::STEP > a.in, end_n = n0 + T::N > a.out;
#pragma unroll
    for (int j = 0; j < kA; ++j)
      *reinterpret_cast<u32x4*>(stage + (j * T::kThreads + thread) * 16) =
          in_place(h.a[j], row[j] != kNowhere, end_k, k + at[j], a.in);
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      const uint32_t l = (BR ? k : n0) + line[j], lines = BR ? a.in : a.out;
      *reinterpret_cast<u32x4*>(stage + SA::kBytes + (j * T::kThreads + thread) * 16) =
          in_place(h.b[j], l < lines, BR ? end_n : end_k, (BR ? n0 : k) + first[j], BR ? a.out : a.in);
    }
  }
};

// y_i = x_t(i) W_e(i) for the rows of an expert; 0 for rows without one.
//
// A block has T::M rows of one expert and T::N columns.  The grid is cut for any
// distribution of the pairs (the counts stay on the GPU): each block finds its
// tile from the experts' beginnings, and blocks past the last end.  BR: the
// columns of W are contiguous.  DIRECT: all rows are in 16-byte pieces, which go
// straight to LDS; otherwise they go through registers, element by element only
// at their ends.
template <class T, bool BR, bool DIRECT, bool PAST>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void expert_product(ProductArgs a) {
  using SA = Staged<T::M, false, T::STEP, false>;
  using SB = Staged<T::N, BR, T::STEP, true>;
  constexpr int kStage = SA::kBytes + SB::kBytes;
  __shared__ __attribute__((aligned(1024))) char lds[T::STAGES * kStage];
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  Part p;
  if (!part_of<T::M, T::N>(a, &p)) return;
  f32x4 acc[T::kM][T::kN];
  clear(acc);
  const int steps = p.e < a.experts && a.x_rows > 0 ? static_cast<int>((a.in + T::STEP - 1) / T::STEP) : 0;
  const uint16_t* w = static_cast<const uint16_t*>(a.w) + (p.e < a.experts ? p.e * a.w_expert : 0);
  const Operands<T, SA, SB, BR> from(a, p, tid);
  char* const mine = lds + wave * (kWave * 16);
  if (DIRECT) {
    const Source sx(a.x), sw(w);
    constexpr int kAhead = T::STAGES - 1, kLoads = from.kA + from.kB;
    if (steps > 0)
#pragma unroll
      for (int s = 0; s < kAhead; ++s) from.issue(a, sx, sw, s, mine + s * kStage);
    for (int s = 0; s < steps; ++s) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kAhead - 1) * kLoads) : "memory");
      __builtin_amdgcn_s_barrier();
      from.issue(a, sx, sw, s + kAhead, mine + (s + kAhead) % T::STAGES * kStage);
      const char* stage = lds + s % T::STAGES * kStage;
      multiply_step<T::kM, T::kN, bf16x8, 1, T::STEP, SA, SB>(stage, stage + SA::kBytes, T::row0(wave),
                                                              T::column0(wave), lane, acc);
    }
    settled();
  } else {
    typename Operands<T, SA, SB, BR>::Held held;
    if (steps > 0) from.load(a, w, 0, &held);
    for (int s = 0; s < steps; ++s) {
      char* stage = lds + (s & 1) * kStage;
      from.put(a, held, s, stage, tid);
      __syncthreads();
      if (s + 1 < steps) from.load(a, w, s + 1, &held);
      multiply_step<T::kM, T::kN, bf16x8, 1, T::STEP, SA, SB>(stage, stage + SA::kBytes, T::row0(wave),
                                                              T::column0(wave), lane, acc);
    }
  }
  __syncthreads();
  static_assert(T::kThreads / kWave * kTurnBytes <= T::STAGES * kStage);
  write_part<PAST>(acc, reinterpret_cast<float*>(lds + wave * kTurnBytes), static_cast<uint16_t*>(a.y), p.m0 + T::row0(wave),
             p.hi, p.n0 + T::column0(wave), a.out, lane);
}

// The same for few rows: 16 of them and 64 columns a block, whose waves share the
// k out among themselves, each with steps of its own in LDS and no barrier, and
// add up their sums in the waves' order at the end.  What binds is the reading of
// the weights, of which a block has 40 KB under way: 240 MB of a decoded batch's, 58
// experts of 2,048 x 1,024, 39 us.
using Thin = Tile<16, 64, 1, 1, 64, 2, 2>;
constexpr int kThinWaves = 4, kThinThreads = kThinWaves * kWave;

template <bool BR, bool DIRECT>
__global__ __launch_bounds__(kThinThreads, 2) void expert_product_thin(ProductArgs a) {
  using T = Thin;
  using SA = Staged<T::M, false, T::STEP, false>;
  using SB = Staged<T::N, BR, T::STEP, true>;
  constexpr int kStage = SA::kBytes + SB::kBytes;
  constexpr int kLoads = SA::kChunks / kWave + SB::kChunks / kWave;
  __shared__ __attribute__((aligned(1024))) char lds[kThinWaves * 2 * kStage];
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  Part p;
  if (!part_of<T::M, T::N>(a, &p)) return;
  f32x4 acc[1][T::kN];
  clear(acc);
  const int steps = p.e < a.experts && a.x_rows > 0 ? static_cast<int>((a.in + T::STEP - 1) / T::STEP) : 0;
  const uint16_t* w = static_cast<const uint16_t*>(a.w) + (p.e < a.experts ? p.e * a.w_expert : 0);
  const Operands<T, SA, SB, BR> from(a, p, lane);
  char* const mine = lds + wave * (2 * kStage);
  if (DIRECT) {
    const Source sx(a.x), sw(w);
    if (wave < steps) from.issue(a, sx, sw, wave, mine);
    int buffer = 0;
    for (int s = wave; s < steps; s += kThinWaves, buffer ^= 1) {
      // the other buffer's reads are done; this one's loads are the older ones
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (s + kThinWaves < steps) {
        from.issue(a, sx, sw, s + kThinWaves, mine + (buffer ^ 1) * kStage);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
      } else {
        settled();
      }
      const char* stage = mine + buffer * kStage;
      multiply_step<1, T::kN, bf16x8, 1, T::STEP, SA, SB>(stage, stage + SA::kBytes, 0, 0, lane, acc);
    }
  } else {
    typename Operands<T, SA, SB, BR>::Held held;
    if (wave < steps) from.load(a, w, wave, &held);
    for (int s = wave; s < steps; s += kThinWaves) {
      from.put(a, held, s, mine, lane);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (s + kThinWaves < steps) from.load(a, w, s + kThinWaves, &held);
      multiply_step<1, T::kN, bf16x8, 1, T::STEP, SA, SB>(mine, mine + SA::kBytes, 0, 0, lane, acc);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
  // every wave's sums where its steps were: four lanes' worth of columns a row
  f32x4(*sums)[T::kN][kWave] = reinterpret_cast<f32x4(*)[T::kN][kWave]>(lds);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < T::kN; ++j) sums[wave][j][lane] = acc[0][j];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int j = 0; j < T::kN; ++j) {
    acc[0][j] = sums[0][j][lane];
#pragma unroll
    for (int v = 1; v < kThinWaves; ++v) acc[0][j] += sums[v][j][lane];
  }
  write_part<false>(acc, reinterpret_cast<float*>(lds + 2 * kThinWaves * kStage - kTurnBytes), static_cast<uint16_t*>(a.y), p.m0,
             p.hi, p.n0, a.out, lane);
}

// --- the weights' gradient ------------------------------------------------------------

// dW_e = sum over the rows i of expert e of x_t(i)^T dy_i: a block has a tile of
// one expert's matrix and goes over the expert's rows, a step's at a time.  An
// expert without rows gets zeros.  With `parts` the rows are shared among so many
// blocks (blockIdx.y), whose sums, a matrix each, add_parts() joins.
//
// A tile costs what its expert has rows, so every XCD gets a part of each
// expert's tiles (neighbours, of the same rows of dW), or of each second one's where
// there are enough of them to come out even: each XCD of an expert reads its rows
// once (see weight_grad_xcds).  Where the parts are not equal they are dealt in
// turn, by expert; not elsewhere, since it spreads what an XCD writes (64 matrices of
// 1,024 x 2,048 float32 of zeros: 101 us in turn, 88 not; of 64 experts with 64 rows
// each, 2,048 x 1,024, 105 and 90).
template <class T, class OUT, bool DIRECT, bool PAST>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void expert_weight_grad(WeightGradArgs a) {
  using SA = Staged<T::M, true, T::STEP, false>;
  using SB = Staged<T::N, true, T::STEP, true>;
  constexpr int kStage = SA::kBytes + SB::kBytes;
  constexpr int kA = SA::kChunks / T::kThreads, kB = SB::kChunks / T::kThreads;
  __shared__ __attribute__((aligned(1024))) char lds[T::STAGES * kStage];
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const uint32_t turn = blockIdx.x / kXcds, xcd = blockIdx.x % kXcds, round = turn / a.tiles_xcd;
  const uint32_t e = a.xcds == kXcds ? round : round * 2 + xcd / (kXcds / 2);
  const uint32_t part = (xcd + (a.tiles % a.xcds != 0 ? round : 0)) % a.xcds;
  const uint32_t tile = part * a.tiles_xcd + turn % a.tiles_xcd;
  if (tile >= a.tiles || e >= static_cast<uint32_t>(a.experts)) return;
  const uint32_t m0 = tile / a.tiles_n * T::M, n0 = tile % a.tiles_n * T::N;
  uint32_t lo, hi;
  rows_of(a.offsets, a.experts, e, a.pairs, &lo, &hi);
  if (a.parts > 1) {
    const uint32_t all = (hi - lo + T::STEP - 1) / T::STEP;
    const uint32_t begin = all * blockIdx.y / a.parts, end = all * (blockIdx.y + 1) / a.parts;
    hi = min(hi, lo + end * T::STEP);
    lo = min(hi, lo + begin * T::STEP);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  const int steps = a.x_rows > 0 ? static_cast<int>((hi - lo + T::STEP - 1) / T::STEP) : 0;
  f32x4 acc[T::kM][T::kN];
  clear(acc);

  uint32_t line_a[kA], col_a[kA], line_b[kB], col_b[kB];
#pragma unroll
  for (int j = 0; j < kA; ++j) {
    const int slot = j * T::kThreads + tid;
    line_a[j] = slot / SA::kPerLine;
    col_a[j] = m0 + SA::place(line_a[j], slot % SA::kPerLine) * 8;
  }
#pragma unroll
  for (int j = 0; j < kB; ++j) {
    const int slot = j * T::kThreads + tid;
    line_b[j] = slot / SB::kPerLine;
    col_b[j] = n0 + SB::place(line_b[j], slot % SB::kPerLine) * 8;
  }
  const uint16_t* dy = static_cast<const uint16_t*>(a.dy) + lo * a.dy_stride;
  if (DIRECT) {
    const Source sx(a.x), sy(dy);
    const uint32_t base = lds_address(lds) + wave * (kWave * 16);
    const uint32_t x_bytes = static_cast<uint32_t>(a.x_stride) * 2, y_bytes = static_cast<uint32_t>(a.dy_stride) * 2;
    constexpr int kAhead = T::STAGES - 1, kOfWave = kWave / SA::kPerLine;
    // The pairs of a step: a wave's chunks j are of kOfWave lines.  They are read
    // one step before they are used, by scalar loads, which the waits for the
    // steps' loads do not count.
    uint32_t pair[kA][kOfWave];
    const auto find = [&](int step) {
#pragma unroll
      for (int j = 0; j < kA; ++j)
#pragma unroll
        for (int i = 0; i < kOfWave; ++i) {
          const uint32_t r = lo + step * T::STEP + (j * T::kThreads + wave * kWave) / SA::kPerLine + i;
          pair[j][i] = a.order == nullptr ? r : scalar(a.order + min(r, hi - 1));
        }
    };
    const auto issue = [&](int step) {
      const uint32_t to = base + step % T::STAGES * kStage;
#pragma unroll
      for (int j = 0; j < kA; ++j) {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < kOfWave; ++i) {
          const uint32_t of = a.order == nullptr ? pair[j][i] : token_of(a.token, pair[j][i]);
          t = lane / SA::kPerLine == i ? of : t;
        }
        const bool in = lo + step * T::STEP + line_a[j] < hi && col_a[j] < a.in && t < a.x_rows;
        load_to_lds(sx, in ? t * x_bytes + col_a[j] * 2 : kNowhere,
                    __builtin_amdgcn_readfirstlane(to + j * T::kThreads * 16));
      }
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        const uint32_t r = step * T::STEP + line_b[j];
        load_to_lds(sy, lo + r < hi && col_b[j] < a.out ? r * y_bytes + col_b[j] * 2 : kNowhere,
                    __builtin_amdgcn_readfirstlane(to + SA::kBytes + j * T::kThreads * 16));
      }
    };
    if (steps > 0) {
      find(0);
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        issue(s);
        find(s + 1);
      }
    }
    for (int s = 0; s < steps; ++s) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kAhead - 1) * (kA + kB)) : "memory");
      __builtin_amdgcn_s_barrier();
      issue(s + kAhead);
      find(s + kAhead + 1);
      const char* stage = lds + s % T::STAGES * kStage;
      multiply_step<T::kM, T::kN, bf16x8, 1, T::STEP, SA, SB>(stage, stage + SA::kBytes, T::row0(wave),
                                                              T::column0(wave), lane, acc);
    }
    settled();
  } else {
    // the pairs of a step's lines are read one step before they are used, so that
    // the waits for the steps cover these reads too
    uint32_t pair[kA];
    const auto find = [&](int step) {
  #pragma unroll
      for (int j = 0; j < kA; ++j) {
        const uint32_t r = lo + step * T::STEP + line_a[j];
        pair[j] = r >= hi ? kNowhere : a.order == nullptr ? r : static_cast<uint32_t>(a.order[r]);
      }
    };
    const auto row_of_x = [&](int j) {
      if (pair[j] == kNowhere || col_a[j] >= a.in) return kNowhere;
      const uint32_t t = a.order == nullptr ? pair[j] : token_of(a.token, pair[j]);
      return t < a.x_rows ? t : kNowhere;
    };
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    u32x4 ra[kA], rb[kB];
    bool found[kA];
    const bool end_m = m0 + T::M > a.in, end_n = n0 + T::N > a.out;
    const auto load = [&](int step) {
#pragma unroll
      for (int j = 0; j < kA; ++j) {
        const uint32_t r = row_of_x(j);
        found[j] = r != kNowhere;
        ra[j] = fetch(x + (found[j] ? r : 0) * a.x_stride, col_a[j], a.in);
      }
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        const uint32_t r = step * T::STEP + line_b[j];
        rb[j] = fetch(dy + (lo + r < hi ? r : 0) * a.dy_stride, col_b[j], a.out);
      }
    };
    if (steps > 0) {
      find(0);
      load(0);
    }
    if (steps > 1) find(1);
    for (int s = 0; s < steps; ++s) {
      char* stage = lds + (s & 1) * kStage;
#pragma unroll
      for (int j = 0; j < kA; ++j)
        *reinterpret_cast<u32x4*>(stage + (j * T::kThreads + tid) * 16) =
            in_place(ra[j], found[j], end_m, col_a[j], a.in);
#pragma unroll
      for (int j = 0; j < kB; ++j)
        *reinterpret_cast<u32x4*>(stage + SA::kBytes + (j * T::kThreads + tid) * 16) =
            in_place(rb[j], lo + s * T::STEP + line_b[j] < hi, end_n, col_b[j], a.out);
      __syncthreads();
      if (s + 1 < steps) load(s + 1);
      if (s + 2 < steps) find(s + 2);
      multiply_step<T::kM, T::kN, bf16x8, 1, T::STEP, SA, SB>(stage, stage + SA::kBytes, T::row0(wave),
                                                              T::column0(wave), lane, acc);
    }
  }
  __syncthreads();
  static_assert(T::kThreads / kWave * kTurnBytes <= T::STAGES * kStage);
  write_part<PAST>(acc, reinterpret_cast<float*>(lds + wave * kTurnBytes),
             static_cast<OUT*>(a.dw) + (static_cast<uint64_t>(blockIdx.y) * a.experts + e) * a.in * a.out, m0 + T::row0(wave), a.in,
             n0 + T::column0(wave), a.out, lane);
}

// The sum of `parts` arrays of n elements, one behind the other, in their order:
// what they read and write at HBM's rate.
constexpr int kAddThreads = 256;
template <class OUT>
__global__ __launch_bounds__(kAddThreads) void add_parts(const float* from, OUT* to, uint64_t n, uint32_t parts) {
  const uint64_t i = (static_cast<uint64_t>(blockIdx.x) * kAddThreads + threadIdx.x) * 4;
  if (i >= n) return;
  if (i + 4 <= n) {
    f32x4 sum = {0, 0, 0, 0};
    for (uint32_t p = 0; p < parts; ++p) sum += reinterpret_cast<const Four*>(from + p * n + i)->v;
    if constexpr (sizeof(OUT) == 4) {
      reinterpret_cast<Four*>(to + i)->v = sum;
    } else {
      const uint32_t w[2] = {two_bf16(sum[0], sum[1]), two_bf16(sum[2], sum[3])};
#pragma unroll
      for (int q = 0; q < 4; ++q) to[i + q] = static_cast<OUT>(w[q / 2] >> (16 * (q % 2)));
    }
    return;
  }
  for (uint64_t j = i; j < n; ++j) {
    float sum = 0;
    for (uint32_t p = 0; p < parts; ++p) sum += from[p * n + j];
    if constexpr (sizeof(OUT) == 4)
      to[j] = sum;
    else
      to[j] = static_cast<OUT>(two_bf16(sum, 0.0f));
  }
}

template <class T> uint64_t tiles_n(uint64_t out) { return (out + T::N - 1) / T::N; }

// Tiles for any distribution of the pairs: whole ones, and a part of one for
// every group that has pairs.
template <class T> uint64_t product_blocks(uint64_t pairs, int experts, uint64_t out) {
  const uint64_t groups = static_cast<uint64_t>(experts) + 1;
  return (pairs / T::M + (groups < pairs ? groups : pairs)) * tiles_n<T>(out);
}
template <class T> uint64_t weight_grad_tiles(uint64_t in, uint64_t out) {
  return (in + T::M - 1) / T::M * tiles_n<T>(out);
}

// The XCDs that share an expert's tiles of the weights' gradient, half or all, with one
// step under way: 32 experts, 32,768 pairs, 1,024 x 2,048, 199 us and 215 (even rows
// 173 and 187); 64 experts 222 and 243; 131,072 pairs of 256, 1,024 x 512, 240 and 283;
// of 128, 2,048 x 1,024, 826 and 775, but 785 with two steps (see DeepGrad).  Below 32
// experts half is no slower either on a later card (16,384 pairs of 16, 2,048 x 2,048,
// 185 and 186; an earlier one had 185 and 173; 65,536 pairs of 16 327 and 355), so 32 is
// a border on the safe side, not where the two cross.
constexpr int kManyExperts = 32;
uint32_t weight_grad_xcds(int experts) { return experts >= kManyExperts ? kXcds / 2 : kXcds; }
uint64_t weight_grad_blocks(int experts, uint64_t tiles) {
  const uint64_t xcds = weight_grad_xcds(experts), at_once = kXcds / xcds;
  return (experts + at_once - 1) / at_once * ((tiles - 1) / xcds + 1) * kXcds;
}

// So many wide tiles give every CU one.  With fewer, smaller ones are faster: 2,048
// pairs of 8 experts, 1,024 x 1,024, 14 us in 64 x 128 and 21 in 128 x 256, 8,192
// pairs 33 either way.
constexpr uint64_t kFull = 256;

// Which tiles a product has, by the rows of an expert if all have as many (the counts
// stay on the GPU): 4,096 pairs of 256 experts that all go to 16 take 90 us in 16 x 64,
// 25 if only those 16 are there.
enum class Rows { kFew, kSome, kMany, kMost };
Rows rows_of_product(uint64_t pairs, int experts, uint64_t out, bool by_out, bool direct) {
  const uint64_t each = pairs / (static_cast<uint64_t>(experts) < pairs ? experts : pairs);
  if (each <= 16) return Rows::kFew;
  if (each <= (direct ? 64 : 128) || (out <= 128 && direct) || pairs / 128 * ((out + 255) / 256) < kFull)
    return Rows::kSome;
  return each >= 1024 && direct && !by_out ? Rows::kMost : Rows::kMany;
}

// Results of this size and more are stored past the caches, since they would push
// out what the product reads, if their rows are whole cache lines: parts of lines
// have to meet in a cache (61 matrices of 1,000 x 776 float32: 109 us past the
// caches, 73 through them).
constexpr uint64_t kPastBytes = 32ull << 20;
bool past_caches(const void* to, uint64_t rows, uint64_t row_bytes) {
  return rows * row_bytes >= kPastBytes && (reinterpret_cast<uintptr_t>(to) | row_bytes) % 128 == 0;
}

template <class T, bool BR, bool DIRECT> void launch_product(ProductArgs a, hipStream_t stream) {
  a.tiles_n = static_cast<uint32_t>(tiles_n<T>(a.out));
  const dim3 grid(static_cast<uint32_t>(product_blocks<T>(a.pairs, a.experts, a.out)));
  if constexpr (T::M == Thin::M)
    expert_product_thin<BR, DIRECT><<<grid, kThinThreads, 0, stream>>>(a);
  else
    (past_caches(a.y, a.pairs, static_cast<uint64_t>(a.out) * 2) ? expert_product<T, BR, DIRECT, true>
                                                             : expert_product<T, BR, DIRECT, false>)
        <<<grid, T::kThreads, 0, stream>>>(a);
}

template <class T, class OUT, bool DIRECT> void launch_weight_grad(WeightGradArgs a, hipStream_t stream) {
  a.tiles_n = static_cast<uint32_t>(tiles_n<T>(a.out));
  a.tiles = static_cast<uint32_t>(weight_grad_tiles<T>(a.in, a.out));
  a.xcds = weight_grad_xcds(a.experts);
  a.tiles_xcd = (a.tiles - 1) / a.xcds + 1;
  const bool past = a.parts == 1 && past_caches(a.dw, static_cast<uint64_t>(a.experts) * a.in, a.out * sizeof(OUT));
  (past ? expert_weight_grad<T, OUT, DIRECT, true> : expert_weight_grad<T, OUT, DIRECT, false>)
      <<<dim3(static_cast<uint32_t>(weight_grad_blocks(a.experts, a.tiles)), a.parts), T::kThreads, 0, stream>>>(a);
}

}  // namespace

uint64_t expert_product_blocks(uint64_t pairs, int experts, uint64_t out, bool by_out, bool direct) {
  switch (rows_of_product(pairs, experts, out, by_out, direct)) {
    case Rows::kFew: return product_blocks<Thin>(pairs, experts, out);
    case Rows::kSome: return product_blocks<Small>(pairs, experts, out);
    case Rows::kMost: return product_blocks<Huge>(pairs, experts, out);
    default: return direct ? product_blocks<Large>(pairs, experts, out) : product_blocks<Middle>(pairs, experts, out);
  }
}

uint64_t expert_weight_grad_blocks(int experts, uint64_t in, uint64_t out, bool direct) {
  const uint64_t tiles = direct ? weight_grad_tiles<LargeGrad>(in, out) : weight_grad_tiles<OddGrad>(in, out);
  return weight_grad_blocks(experts, tiles);
}

// Where the tiles leave places on the CUs free and have many rows to go over, the
// rows are shared: 16,384 pairs of 4 experts, 256 x 512, 28 us instead of 123; but
// two parts are no faster than one (8,192 pairs of 8 experts, 1,024 x 1,024, 53 us
// against 48).  A part has at least 256 rows if all experts have as many.
uint32_t expert_weight_grad_parts(uint64_t pairs, int experts, uint64_t in, uint64_t out) {
  constexpr uint64_t kPlaces = 512, kMost = 16, kRows = 256;
  const uint64_t tiles = experts * weight_grad_tiles<LargeGrad>(in, out);
  const uint64_t parts = std::min({kMost, kPlaces / tiles, pairs / experts / kRows});
  return parts > 2 ? static_cast<uint32_t>(parts) : 1;
}

hipError_t launch_expert_product(const ProductArgs& a, bool out_contiguous, bool direct, hipStream_t stream) {
  switch (rows_of_product(a.pairs, a.experts, a.out, out_contiguous, direct)) {
    case Rows::kFew:
      if (direct)
        (out_contiguous ? launch_product<Thin, true, true> : launch_product<Thin, false, true>)(a, stream);
      else
        (out_contiguous ? launch_product<Thin, true, false> : launch_product<Thin, false, false>)(a, stream);
      break;
    case Rows::kSome:
      if (direct)
        (out_contiguous ? launch_product<Small, true, true> : launch_product<Small, false, true>)(a, stream);
      else
        (out_contiguous ? launch_product<Small, true, false> : launch_product<Small, false, false>)(a, stream);
      break;
    case Rows::kMany:
      if (direct)
        (out_contiguous ? launch_product<Large, true, true> : launch_product<Large, false, true>)(a, stream);
      else
        (out_contiguous ? launch_product<Middle, true, false> : launch_product<Middle, false, false>)(a, stream);
      break;
    case Rows::kMost:
      launch_product<Huge, false, true>(a, stream);
  }
  return hipGetLastError();
}

hipError_t launch_expert_weight_grad(const WeightGradArgs& a, ar_dtype_t dw_dtype, bool direct, hipStream_t stream) {
  const bool many = a.experts >= kManyExperts;
  if (dw_dtype == AR_FLOAT32)
    (!direct ? launch_weight_grad<OddGrad, float, false>
     : many  ? launch_weight_grad<DeepGrad, float, true>
             : launch_weight_grad<LargeGrad, float, true>)(a, stream);
  else
    (!direct ? launch_weight_grad<OddGrad, uint16_t, false>
     : many  ? launch_weight_grad<DeepGrad, uint16_t, true>
             : launch_weight_grad<LargeGrad, uint16_t, true>)(a, stream);
  return hipGetLastError();
}

hipError_t launch_expert_add_parts(const WeightGradArgs& a, void* dw, ar_dtype_t dw_dtype, hipStream_t stream) {
  const uint64_t n = static_cast<uint64_t>(a.experts) * a.in * a.out;
  const dim3 grid(static_cast<uint32_t>((n + kAddThreads * 4 - 1) / (kAddThreads * 4)));
  const float* from = static_cast<const float*>(a.dw);
  if (dw_dtype == AR_FLOAT32)
    add_parts<float><<<grid, kAddThreads, 0, stream>>>(from, static_cast<float*>(dw), n, a.parts);
  else
    add_parts<uint16_t><<<grid, kAddThreads, 0, stream>>>(from, static_cast<uint16_t*>(dw), n, a.parts);
  return hipGetLastError();
}

}  // namespace ar
