// Expert router kernels (gfx950): the choice of experts with its weights,
// counts and balance loss, and the gradient of the logits.
//
// A token's logits are one row, held by G lanes of a wave (8 up to 256
// experts), V = 4 to 32 values each, so that a wave has 8 rows at a time: a
// row's maximum and sums then take three steps across lanes, shared by 8
// rows, where a wave a row would take six for each.  Rows are read in
// 16-byte accesses whatever their alignment.
//
// Exponentials and reciprocals are single instructions, off by one step of the
// last place each: a weight's error is then a few roundings of float32, most of
// them the exponent's, 3 |x - top| half steps.  A full-precision exponential is
// several instructions more a value, in a kernel that instructions bind.
//
// Times in this file are medians of a kernel trace unless they say otherwise;
// pairs that compare two forms were taken together, back to back, when the one
// was chosen.
#include "device_common.hpp"
#include "train/route.hpp"
#include "train/wave.hpp"

namespace ar {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kWaves = kBlock / kWave;
constexpr int kRouteBlock = 512;                 // threads of the forward kernel
constexpr int kRouteWaves = kRouteBlock / kWave;
constexpr int kNone = INT32_MIN;

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_widen(x); }

// --- lanes of a row ----------------------------------------------------------------

// Lane g of a row's G = 2^LG has C chunks of W consecutive columns, chunk c
// at column (c G + g) W, so that G lanes read one run.
template <class T, int LG, int C> struct Shape {
  static constexpr int G = 1 << LG;
  static constexpr int W = 16 / sizeof(T);
  static constexpr int V = C * W;
  static constexpr int kColumns = G * V;
  static constexpr int kRows = kWave / G;           // of a wave
  static __device__ int lane() { return threadIdx.x & (G - 1); }
  static __device__ int column(int v) { return ((v / W) * G + lane()) * W + v % W; }
};

template <int CTRL> __device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, 0xf, 0xf, false);
}
// The value of the lane across step S of a row: pairs, pairs of pairs, then
// mirrored halves of 8 and 16, and lanes 16 apart.
template <int S> __device__ __forceinline__ int across(int x) {
  if constexpr (S == 0)
    return dpp<0xB1>(x);
  else if constexpr (S == 1)
    return dpp<0x4E>(x);
  else if constexpr (S == 2)
    return dpp<0x141>(x);
  else if constexpr (S == 3)
    return dpp<0x140>(x);
  else
    return __shfl_xor(x, 16);
}
template <int LG, int S = 0> __device__ __forceinline__ int row_max(int x) {
  if constexpr (S < LG)
    return row_max<LG, S + 1>(max(x, across<S>(x)));
  else
    return x;
}
template <int LG, int S = 0> __device__ __forceinline__ float row_sum(float x) {
  if constexpr (S < LG)
    return row_sum<LG, S + 1>(x + __int_as_float(across<S>(__float_as_int(x))));
  else
    return x;
}

// A wave's LDS accesses happen in the order of its program; this keeps the
// compiler from changing that.
__device__ __forceinline__ void wave_in_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A row's chunks as they lie in memory; -infinity beyond its end.
using Chunk = uint32_t __attribute__((ext_vector_type(4)));
template <class T> struct Loose;
template <> struct Loose<float> {
  typedef Chunk type __attribute__((aligned(4)));
};
template <> struct Loose<uint16_t> {
  typedef Chunk type __attribute__((aligned(2)));
};

template <class T> __device__ __forceinline__ Chunk minus_infinity() {
  const uint32_t w = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
  return Chunk{w, w, w, w};
}

// Whether all lanes' parts of chunk c exist.  Launches take the smallest
// arrangement that holds a row, so the lower half of the chunks always do.
template <class S, int C> __device__ __forceinline__ bool whole_chunk(int c, int experts) {
  return c < C / 2 || (c + 1) * S::G * S::W <= experts;
}

template <class S, class T, int C>
__device__ __forceinline__ void load_chunks(const T* row, int experts, Chunk (&raw)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * S::G + S::lane()) * S::W;
    if (whole_chunk<S, C>(c, experts)) {
      raw[c] = *reinterpret_cast<const typename Loose<T>::type*>(row + col);
    } else {
      T e[S::W];
      raw[c] = minus_infinity<T>();
      __builtin_memcpy(e, &raw[c], 16);
#pragma unroll
      for (int w = 0; w < S::W; ++w)
        if (col + w < experts) e[w] = row[col + w];
      __builtin_memcpy(&raw[c], e, 16);
    }
  }
}

template <class T> __device__ __forceinline__ float value_of(const Chunk& raw, int w) {
  if constexpr (sizeof(T) == 4)
    return __uint_as_float(raw[w]);
  else
    return __uint_as_float(w % 2 == 0 ? raw[w / 2] << 16 : raw[w / 2] & 0xffff0000u);
}

// --- the choice ----------------------------------------------------------------------

// A logit as an integer of the same order, 0 for both zeros.  With `bias`, a
// negative one is moved up by that much, so that dropping the low bits keeps
// -infinity apart from the lowest finite number.
__device__ __forceinline__ int order(float x, int bias) {
  const int b = __float_as_int(x);
  return b < 0 ? static_cast<int>(0x80000000u + bias - static_cast<uint32_t>(b)) : b;
}
__device__ __forceinline__ float from_order(int key) {
  return __uint_as_float(key < 0 ? 0x80000000u - static_cast<uint32_t>(key) : static_cast<uint32_t>(key));
}
constexpr int kMinusInfinity = -0x7f800000;         // order(-infinity, 0)

__device__ __forceinline__ void sort2(int& a, int& b) {
  const int hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}

// Batcher's odd-even merge sort (Knuth, The Art of Computer Programming 3,
// 5.2.2), descending.
template <int N> __device__ __forceinline__ void sort(int* x) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k && i + j + k < N; ++i)
          if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) sort2(x[i + j], x[i + j + k]);
}

// Merge of a bitonic list, descending.
template <int N> __device__ __forceinline__ void merge(int* x) {
#pragma unroll
  for (int k = N / 2; k >= 1; k /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & k) == 0) sort2(x[i], x[i + k]);
}

// The N largest of two descending lists of N, into the first: the larger of
// each pair of opposite ends, which is a bitonic list.
template <int N> __device__ __forceinline__ void join(int* x, const int* y) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = max(x[i], y[N - 1 - i]);
  merge<N>(x);
}

// The row's L largest from each lane's N (descending), for every lane.
template <int LG, int L, int N, int S = 0> __device__ __forceinline__ void join_row(int* x) {
  if constexpr (S < LG) {
    if constexpr (N < L) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[2 * N - 1 - i] = across<S>(x[i]);
      merge<2 * N>(x);
      join_row<LG, L, 2 * N, S + 1>(x);
    } else {
      int y[N];
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = across<S>(x[i]);
      join<N>(x, y);
      join_row<LG, L, N, S + 1>(x);
    }
  }
}

// What was chosen for a row: lane k of the row has the k-th column, -1 for
// none, and its logit (where a float32 key has cut it, only the interval).
// `top` is the largest logit, or (within 2^16) the end of its interval
// of keys, at most 8 away: any number near it serves the softmax.
struct Choice {
  int index;
  float value, top;
};

template <class T, int LG, int C> struct Keys {
  static constexpr bool kExact = sizeof(T) == 2;
  static constexpr int kLow = Shape<T, LG, C>::kColumns - 1;
  static constexpr int kBig = 0x47800000;            // 2^16
  // The order of a logit without the low bits; -infinity is by itself.
  static __device__ __forceinline__ int high(float x) { return order(x, kExact ? 0 : kLow) & ~kLow; }
  // In unsigned numbers, which may wrap: high + kBig passes INT_MAX from 6e-5 on.
  static __host__ __device__ constexpr bool big(int high) { return static_cast<uint32_t>(high) + kBig > 2u * kBig; }
};
static_assert(Keys<float, 3, 8>::big(0x7f800000) && Keys<float, 3, 8>::big(-0x7f800000) &&
                  !Keys<float, 3, 8>::big(0x3f800000) && !Keys<float, 3, 8>::big(-0x47800000),
              "infinities are big, 1 and -2^16 are not");

// How far the keys have decided a row.
enum Decided { kDecided, kOrderOpen, kOpen };

// The row's L largest by keys of 32 bits: the order of the logit in the high
// bits, its column (the lowest the largest) in the low ones.  Each lane sorts
// its values in lists of L and joins them, then the lanes join theirs.
// bfloat16 fits the high bits and keys are exact.  Of a float32 log2(columns)
// bits are cut off: where neighbours among the top_k largest agree in what is
// left their order is open (kOrderOpen), where the top_k-th agrees with the
// next one the choice is (kOpen).  So it is where the top is beyond 2^16 or
// not finite; a row of -infinity only is decided.
template <class T, int LG, int C, int L>
__device__ __forceinline__ Decided choose(const float (&x)[Shape<T, LG, C>::V], int top_k, bool token, Choice* out) {
  using S = Shape<T, LG, C>;
  using K = Keys<T, LG, C>;
  constexpr int kLow = K::kLow;                      // of a key: columns - 1 - column
  constexpr int N = L < S::V ? L : S::V;
  const int lane = S::lane();
  int list[L], key[S::V];
#pragma unroll
  for (int v = 0; v < S::V; ++v) {
    const int low = kLow - ((v / S::W) * S::G * S::W + v % S::W);   // of lane 0
    key[v] = K::kExact ? order(x[v], 0) | low : K::high(x[v]) | low;
  }
  int part[S::V];
#pragma unroll
  for (int v = 0; v < S::V; ++v) part[v] = key[v];
#pragma unroll
  for (int v = 0; v < S::V; v += N) {
    sort<N>(part + v);
    if (v > 0) join<N>(part, part + v);
  }
  // the lane's share of the column: its bits are ones so far
#pragma unroll
  for (int i = 0; i < N; ++i) list[i] = part[i] - lane * S::W;
  join_row<LG, L, N>(list);

  const int top = list[0] & ~kLow;
  const bool any = top > kMinusInfinity;
  bool open = any && K::big(top), order_open = false;
  int mine = list[0];
#pragma unroll
  for (int k = 1; k < L; ++k) mine = lane == k ? list[k] : mine;
  if constexpr (!K::kExact) {
    constexpr int kNothing = kMinusInfinity | kLow;   // the largest key of -infinity
    uint32_t apart = UINT32_MAX;                      // least difference of neighbours
    int last = list[0];
#pragma unroll
    for (int k = 1; k < L; ++k) {
      const uint32_t differ = static_cast<uint32_t>(list[k - 1] ^ list[k]);
      apart = min(apart, differ);
      if (k == top_k) open = open || (differ <= kLow && list[k] > kNothing);
      if (k < top_k) last = list[k];
    }
    order_open = apart <= kLow;                       // of what was not chosen too: no matter
    // with top_k = L the next largest is not in the list: no more values than
    // were chosen may reach the last one's interval, none of them a lane's L-th
    if (top_k == L) {
      const bool counts = token && last > kNothing;
      const int floor = counts ? last & ~kLow : INT32_MAX;
      int reach = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) reach += __popcll(__ballot(part[i] >= floor));
      open = open || reach != __popcll(__ballot(counts && lane == 0)) * L ||
             (N < S::V && __any(part[N - 1] >= floor));
    }
  }
  out->top = any ? from_order(top) : 0.0f;
  out->value = from_order(mine & ~kLow);
  out->index = lane < top_k && (mine & ~kLow) > kMinusInfinity ? kLow - (mine & kLow) : -1;
  return open ? kOpen : order_open ? kOrderOpen : kDecided;
}

// Puts the row's chosen (lane k has the k-th, with its whole logit) in order;
// `room` is L pairs of LDS for the row.
template <class S, int L> __device__ __forceinline__ void reorder(Choice* c, int2* room) {
  const int lane = S::lane();
  const int key = c->index >= 0 ? order(c->value, 0) : kNone;
  if (lane < L) room[lane] = make_int2(key, c->index);
  wave_in_order();
  int rank = 0;
#pragma unroll
  for (int k = 0; k < L; ++k) {
    const int2 other = room[k];
    rank += other.x > key || (other.x == key && (c->index < 0 ? k < lane : other.y < c->index)) ? 1 : 0;
  }
  wave_in_order();
  if (lane < L) room[rank] = make_int2(key, c->index);
  wave_in_order();
  if (lane < L) {
    const int2 at = room[lane];
    c->index = at.y;
    c->value = from_order(at.x);
  }
}

// The same for any row, by top_k searches over all values: exact, NaN never
// chosen, about three times the work, and a wave takes it for all its rows if
// one of them is open.  Of normal bfloat16 logits none is.  Of float32 ones
// with eight of 256 chosen one row in 2,600 is; but with two chosen, where the
// list ends with the choice, every row whose two best lie in one lane: 10 to
// 12 % of the rows of 32 to 256 experts and 42 % of 8, which are 57 to 99 % of
// the waves (131,072 rows of 256 take 40.8 us back to back for two chosen, 35.3
// for four).  Within 2^16 its top is the one above, so that a row's results do
// not depend on which of the two its wave took.
template <class T, int LG, int C>
__device__ __forceinline__ Choice choose_slowly(const float (&x)[Shape<T, LG, C>::V], int top_k) {
  using S = Shape<T, LG, C>;
  using K = Keys<T, LG, C>;
  int key[S::V];
#pragma unroll
  for (int v = 0; v < S::V; ++v) {
    float y = x[v];
    asm volatile("" : "+v"(y));                      // keeps this work on this path
    key[v] = y > -__builtin_inff() ? order(y, 0) : kNone;
  }
  Choice out = {-1, 0.0f, 0.0f};
  for (int k = 0; k < top_k; ++k) {
    int best = kNone;
#pragma unroll
    for (int v = 0; v < S::V; ++v) best = max(best, key[v]);
    best = row_max<LG>(best);
    int first = -S::kColumns;                        // minus the lowest column of the best
#pragma unroll
    for (int v = S::V - 1; v >= 0; --v)
      if (key[v] == best) first = -S::column(v);
    const int col = -row_max<LG>(first);
    if (best != kNone) {
      if (k == 0) {
        const int high = K::high(from_order(best));
        out.top = K::big(high) ? from_order(best) : from_order(high);
      }
      if (S::lane() == k) {
        out.index = col;
        out.value = from_order(best);
      }
    }
#pragma unroll
    for (int v = 0; v < S::V; ++v)
      if (S::column(v) == col) key[v] = kNone;
  }
  return out;
}

// a plus what lies 32 (16) lanes across, in the lower half (the even rows of
// 16), and b's in the upper half (the odd rows).
__device__ __forceinline__ float swap32_and_add(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap16_and_add(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// --- forward ----------------------------------------------------------------------------

__device__ __forceinline__ uint64_t pair_of(float s, uint32_t count) {
  return static_cast<uint64_t>(__float_as_uint(s)) << 32 | count;
}
__device__ __forceinline__ float sum_in(uint64_t pair) { return __uint_as_float(static_cast<uint32_t>(pair >> 32)); }
__device__ __forceinline__ uint32_t count_in(uint64_t pair) { return static_cast<uint32_t>(pair); }

// Reads n rows (row, row + stride, ...) of a table, column e, several at a
// time (they come from memory, about a microsecond each if one by one), and
// hands them to take() in order.  `most` is the largest n of the block.
template <int kAtOnce, class Take>
__device__ __forceinline__ void read_rows(const uint64_t* table, int row, int n, int most, int stride, int experts,
                                          int e, const Take& take) {
  for (int i = 0; i < most; i += kAtOnce) {
    uint64_t x[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (i + u < most)
        x[u] = shared_load(&table[static_cast<size_t>(row + max(min(i + u, n - 1), 0) * stride) * experts + e]);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (i + u < most && i + u < n) take(x[u]);
  }
}

// How the last block's threads share the columns: E of them (a power of two)
// at a time, in P slices of rows.
struct Slices {
  int E, P, e, slice;
  __device__ explicit Slices(int experts) {
    E = min(kRouteBlock, 1 << (32 - __clz(max(experts - 1, 1))));
    P = kRouteBlock / E;
    e = threadIdx.x & (E - 1);
    slice = threadIdx.x / E;
  }
};

// E / (K T^2) of T tokens.
__device__ __forceinline__ double unit_of(const RouteShape& a, uint32_t tokens) {
  const double n = tokens;
  return n > 0 ? a.experts / (a.top_k * n * n) : 0.0;
}

// The forward pass.  Its bytes are few (the logits once, eight bytes a choice)
// and its VALUs bind it: a row of 256 bfloat16 takes about 94 instructions of
// a wave, nearly half of them the 8-of-32 lists (a maximum, a minimum or a
// compare takes 4.3 cycles of a SIMD, an addition, product or xor 2.2 and an
// exp 8.2), most of the rest keys and exponentials.  Two waves a SIMD fit (200
// to 240 registers): four of 128 registers spilled and took 46 us where two
// took 32.4, twice the blocks 39.  The rows' exponentials stay where they were
// read and are added up per column in registers; the sums of a block's 8
// waves, of up to 16 blocks and of all are joined by the last to arrive, in
// three short stages (about 6 us).
// Measured, 131,072 rows: 256 bfloat16, 8 chosen 32.7 us (2.1 TB/s read; the
// bytes alone 12; 31 back to back), 256 float32 45.6 us (2.9 TB/s; 23; 42 back
// to back); 32,768 rows of 128 bfloat16, 2 chosen 12 us; one row 3.8 us.
template <class T, int LG, int C, int L, int RANKS>
__global__ __launch_bounds__(kRouteBlock, 2) void route_kernel(RouteArgs<RANKS> a) {
  using S = Shape<T, LG, C>;
  constexpr int V = S::V;
  __shared__ uint32_t hist[S::kColumns];
  __shared__ alignas(16) float rows_lds[sizeof(T) == 4 ? kRouteWaves * kWave * V : 1];
  __shared__ uint32_t tokens[kRouteWaves];
  const int wave = wave_uniform(threadIdx.x / kWave), lane = S::lane();
  const int rank = blockIdx.y;
  const T* logits = static_cast<const T*>(a.logits.p[rank]);
  const uint8_t* masks = static_cast<const uint8_t*>(a.masks.p[rank]);
  for (int i = threadIdx.x; i < S::kColumns; i += kRouteBlock) hist[i] = 0;
  __syncthreads();

  float total[V];
#pragma unroll
  for (int v = 0; v < V; ++v) total[v] = 0.0f;
  uint32_t live_rows = 0;
  const uint32_t begin = blockIdx.x * a.rows_per_block;
  const uint32_t end = min(begin + a.rows_per_block, a.tokens);
  // a wave's rows are neighbours; rows past the end are read as the last one
  const uint32_t sub = wave * S::kRows + threadIdx.x % kWave / S::G;
  Chunk next[C];
  bool next_token = false;
  auto fetch = [&](uint32_t first) {
    const uint32_t i = min(first + sub, end - 1);
    next_token = first + sub < end && (masks == nullptr || masks[i] != 0);
    load_chunks<S>(logits + i * a.row_stride, a.experts, next);
  };
  // A row's results are stored when the next one's work begins, before the
  // reads ahead: memory answers in order, so whoever waits for a read waits for
  // all stores before it, which are then a whole row's work old.
  int done_index = -1;
  float done_weight = 0.0f;
  uint32_t done_first = end;
  auto store_done = [&] {
    if (lane < a.top_k && done_first + sub < end) {
      const uint64_t at = (static_cast<uint64_t>(rank) * a.tokens + done_first + sub) * a.top_k + lane;
      a.indices[at] = done_index;
      a.weights[at] = done_weight;
      if (done_index >= 0) atomicAdd(&hist[done_index], 1u);
    }
  };
  if (begin < end) fetch(begin);
  for (uint32_t first = begin; first < end; first += kRouteWaves * S::kRows) {
    // a wave that is ahead gives way to the one it shares a SIMD with, which
    // would otherwise finish alone, at half the rate (32.4 us without, 30.8 with)
    const uint32_t done = (first - begin) * 4;
    if (done >= (end - begin) * 3)
      __builtin_amdgcn_s_setprio(0);
    else if (done >= (end - begin) * 2)
      __builtin_amdgcn_s_setprio(1);
    else if (done >= end - begin)
      __builtin_amdgcn_s_setprio(2);
    else
      __builtin_amdgcn_s_setprio(3);
    const bool token = next_token;
    Chunk raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) raw[c] = next[c];
    store_done();
    if (first + kRouteWaves * S::kRows < end) fetch(first + kRouteWaves * S::kRows);
    if (__any(!token)) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (!token) raw[c] = minus_infinity<T>();
    }
    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = value_of<T>(raw[v / S::W], v % S::W);

    Choice choice;
    const Decided decided = choose<T, LG, C, L>(x, a.top_k, token, &choice);
    if (__any(token && decided == kOpen)) {
      choice = choose_slowly<T, LG, C>(x, a.top_k);
    } else if constexpr (sizeof(T) == 4) {
      // the whole float32, by way of LDS: reading it again from memory would
      // wait for the rows that are being read ahead
      float* room = rows_lds + sub * S::kColumns;
#pragma unroll
      for (int v = 0; v < V; ++v) room[S::column(v)] = x[v];
      wave_in_order();
      choice.value = room[max(choice.index, 0)];
      wave_in_order();
      if (__any(token && decided == kOrderOpen)) reorder<S, L>(&choice, reinterpret_cast<int2*>(room));
    }
    if (!token) choice = {-1, 0.0f, 0.0f};

    // exp(x - top) = 2^(x log2(e) - top log2(e)): rounding the second product
    // scales a row's values by one factor, which the sum takes out.  Tops
    // beyond 2^20, where that factor could overflow, are subtracted first.
    float top = choice.top;
    const float away = fabsf(top) <= 0x1p20f ? 0.0f : top;
    if (__any(away != 0.0f)) {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] -= away;
      top -= away;
    }
    const float shift = top * kLog2e;
    const float xk = choice.index >= 0 ? choice.value - away : -__builtin_inff();
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = __builtin_amdgcn_exp2f(fmaf(x[v], kLog2e, -shift));
      sum += x[v];
    }
    sum = row_sum<LG>(sum);
    const bool live = sum != 0.0f;          // a NaN lives
    const float inv = live ? __builtin_amdgcn_rcpf(sum) : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) total[v] = fmaf(x[v], inv, total[v]);
    live_rows += static_cast<uint32_t>(__popcll(__ballot(live && lane == 0)));

    const float mine = __builtin_amdgcn_exp2f(fmaf(xk, kLog2e, -shift));
    float weight = mine * inv;
    if (a.renormalize) weight = live ? mine * __builtin_amdgcn_rcpf(row_sum<LG>(mine)) : 0.0f;
    if (sum != sum) weight = sum;
    done_index = choice.index;
    done_weight = weight;
    done_first = first;
  }
  store_done();

  // the wave's rows added up, two registers into one at a step: halves of the
  // wave, then rows of 16 lanes, change places between the two, so that each
  // lane is left with the sums of other columns
  __shared__ float sums[kRouteWaves][S::kColumns];
  if constexpr (S::G == 8) {
#pragma unroll
    for (int v = 0; v < V; ++v) total[v] += __int_as_float(dpp<0x128>(__float_as_int(total[v])));
  }
#pragma unroll
  for (int v = 0; v < V / 2; ++v) total[v] = swap32_and_add(total[v], total[v + V / 2]);
  constexpr int N = S::G <= 16 ? V / 4 : V / 2;
  if constexpr (S::G <= 16) {
#pragma unroll
    for (int v = 0; v < N; ++v) total[v] = swap16_and_add(total[v], total[v + N]);
  }
  const int first_v = (threadIdx.x & 32 ? V / 2 : 0) + (S::G <= 16 && (threadIdx.x & 16) ? V / 4 : 0);
#pragma unroll
  for (int v = 0; v < N; ++v)
    if (S::G > 8 || (threadIdx.x & 8) == 0) sums[wave][S::column(first_v + v)] = total[v];
  if (threadIdx.x % kWave == 0) tokens[wave] = live_rows;
  __syncthreads();

  RouteSums* ws = a.sums;
  const uint32_t groups_of_rank = (gridDim.x - 1) / a.group + 1, groups = groups_of_rank * gridDim.y;
  const uint32_t my_group = rank * groups_of_rank + blockIdx.x / a.group;
  const uint32_t in_group = min(a.group, gridDim.x - blockIdx.x / a.group * a.group);
  const uint32_t block = rank * gridDim.x + blockIdx.x, block0 = block - blockIdx.x % a.group;
  uint32_t n = 0;
#pragma unroll
  for (int w = 0; w < kRouteWaves; ++w) n += tokens[w];
  auto of_waves = [&](int e) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) s += sums[w][e];
    return s;
  };

  if (groups == 1 && in_group == 1) {         // the only block
    const double unit = unit_of(a, n);
    double loss = 0.0;
    for (int e = threadIdx.x; e < a.experts; e += kRouteBlock) {
      const float share = static_cast<float>(unit * hist[e]);
      a.counts[e] = static_cast<int32_t>(hist[e]);
      a.share[e] = share;
      loss += static_cast<double>(of_waves(e)) * share;
    }
    loss = block_sum<kRouteBlock>(loss);
    if (threadIdx.x == 0) *a.loss = static_cast<float>(loss);
    return;
  }

  // a group's sums onto the totals
  auto add = [&](int e, double s, uint32_t count) {
    if (s >= 0.0) {
      const uint64_t fixed = static_cast<uint64_t>(s * 4294967296.0 + 0.5);
      if (fixed != 0) shared_add(&ws->share[e], fixed);
    } else {
      shared_store(&ws->not_finite, 1u);
    }
    if (count != 0) shared_add(&ws->counts[rank * a.experts + e], count);
  };
  if (in_group > 1) {
    __shared__ double part_s[kRouteBlock];
    __shared__ uint32_t part_c[kRouteBlock];
    for (int e = threadIdx.x; e < a.experts; e += kRouteBlock)
      shared_store(&ws->of_block[static_cast<size_t>(block) * a.experts + e], pair_of(of_waves(e), hist[e]));
    if (threadIdx.x == 0) shared_store(&ws->tokens_of_block[block], n);
    if (!last_to_arrive(&ws->arrived[my_group].count, in_group)) return;
    n = threadIdx.x < in_group ? shared_load(&ws->tokens_of_block[block0 + threadIdx.x]) : 0u;
    const Slices t(a.experts);
    for (int e0 = 0; e0 < a.experts; e0 += t.E) {
      const int e = min(e0 + t.e, a.experts - 1);
      double s = 0.0;
      uint32_t c = 0;
      const int rows = (static_cast<int>(in_group) - t.slice + t.P - 1) / t.P;
      read_rows<16>(ws->of_block, block0 + t.slice, rows, (in_group + t.P - 1) / t.P, t.P, a.experts, e,
                    [&](uint64_t x) {
                      s += sum_in(x);
                      c += count_in(x);
                    });
      if (t.P > 1) {
        part_s[threadIdx.x] = s;
        part_c[threadIdx.x] = c;
        __syncthreads();
        if (t.slice == 0)
          for (int i = 1; i < min(t.P, static_cast<int>(in_group)); ++i) {
            s += part_s[i * t.E + t.e];
            c += part_c[i * t.E + t.e];
          }
      }
      if (t.slice == 0 && e0 + t.e < a.experts) add(e, s, c);
    }
    n = wave_sum(n);                       // at most 16 blocks: the first wave has them all
    if (threadIdx.x == 0) ws->arrived[my_group].count = 0;
  } else {
    for (int e = threadIdx.x; e < a.experts; e += kRouteBlock) add(e, of_waves(e), hist[e]);
  }
  if (threadIdx.x == 0) shared_add(&ws->tokens, n);
  if (!last_to_arrive(&ws->groups_arrived.count, groups)) return;

  // the last block: counts, shares and loss, and the totals 0 again
  const uint32_t live = shared_load(&ws->tokens), bad = shared_load(&ws->not_finite);
  for (int e = threadIdx.x; e < a.experts; e += kRouteBlock) hist[e] = 0;
  __syncthreads();
  const int all = a.nranks * a.experts;
  constexpr int kAtOnce = 8;
  for (int i0 = threadIdx.x; i0 < all; i0 += kAtOnce * kRouteBlock) {
    uint32_t c[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (i0 + u * kRouteBlock < all) c[u] = shared_load(&ws->counts[i0 + u * kRouteBlock]);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kRouteBlock;
      if (i < all) {
        a.counts[i] = static_cast<int32_t>(c[u]);
        ws->counts[i] = 0;
        if (c[u] != 0) atomicAdd(&hist[i % a.experts], c[u]);
      }
    }
  }
  __syncthreads();
  const double unit = unit_of(a, live);
  double loss = 0.0;
  for (int e = threadIdx.x; e < a.experts; e += kRouteBlock) {
    const double s = static_cast<double>(shared_load(&ws->share[e])) / 4294967296.0;
    ws->share[e] = 0;
    const float share = static_cast<float>(unit * hist[e]);
    a.share[e] = share;
    loss += s * share;
  }
  loss = block_sum<kRouteBlock>(loss);
  if (threadIdx.x == 0) {
    *a.loss = bad ? __builtin_nanf("") : static_cast<float>(loss);
    ws->tokens = ws->not_finite = ws->groups_arrived.count = 0;
  }
}

// --- gradient ----------------------------------------------------------------------------

// The gradient.  A row is read again and its softmax taken again, which costs
// less than keeping it would (8 bytes a row of statistics save two of the
// reductions, and memory is what binds this kernel); with p and the
// coefficients c_e = dloss E C_e / (K T^2), per row
//   dx = p (c - sum p c) + w (dw - sum w dw) at the chosen    (renormalized)
//   dx = p (d - sum p d), d = c + dw at the chosen            (otherwise)
// What belongs to the chosen columns alone takes a detour through LDS, one
// write a choice, instead of a compare of every column with every choice.
// Measured, 131,072 rows of 256 float32: 42.9 us, 6.3 TB/s of the 268 MB read
// and written; of 256 bfloat16 24 us back to back (5.6 TB/s); 32,768 rows of
// 128 bfloat16, renormalized: 5.8 us.
template <class T, int LG, int C, bool RENORMALIZE, int RANKS>
__global__ __launch_bounds__(kBlock, 4) void route_grad_kernel(RouteGradArgs<RANKS> a) {
  using S = Shape<T, LG, C>;
  constexpr int V = S::V, W = S::W;
  // what the chosen experts' weights add, a row of columns for each row of
  // logits; zero but for the entries in use.  The pad keeps two rows' same
  // columns out of each other's banks.
  constexpr int kPitch = S::kColumns + 32;
  __shared__ alignas(16) float spread[kWaves * S::kRows * kPitch];
  __shared__ alignas(16) float coef[S::kColumns];    // of every row: dloss times the expert's share
  const int wave = wave_uniform(threadIdx.x / kWave), lane = S::lane();
  const int rank = blockIdx.y;
  const uint32_t sub = wave * S::kRows + threadIdx.x % kWave / S::G;
  float* at = spread + sub * kPitch;
  const T* logits = static_cast<const T*>(a.logits.p[rank]);
  const uint8_t* masks = static_cast<const uint8_t*>(a.masks.p[rank]);
  const float* dweights = static_cast<const float*>(a.dweights.p[rank]);
  const float dloss = a.dloss != nullptr ? *a.dloss : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) at[S::column(v)] = 0.0f;
  for (int e = threadIdx.x; e < S::kColumns; e += kBlock) coef[e] = e < a.experts ? dloss * a.share[e] : 0.0f;
  __syncthreads();
  const uint32_t begin = blockIdx.x * a.rows_per_block;
  const uint32_t end = min(begin + a.rows_per_block, a.tokens);
  for (uint32_t first = begin; first < end; first += kWaves * S::kRows) {
    const uint32_t i = min(first + sub, end - 1);
    const uint64_t token = static_cast<uint64_t>(rank) * a.tokens + i;
    const T* row = logits + i * a.row_stride;
    const bool counts = masks == nullptr || masks[i] != 0;
    int index = -1;
    float dw = 0.0f;
    if (dweights != nullptr && lane < a.top_k) {
      index = a.indices[token * a.top_k + lane];
      if (static_cast<uint32_t>(index) >= static_cast<uint32_t>(a.experts)) index = -1;
      if (index >= 0) dw = dweights[static_cast<uint64_t>(i) * a.top_k + lane];
    }
    Chunk raw[C];
    load_chunks<S>(row, a.experts, raw);
    if (__any(!counts)) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (!counts) raw[c] = minus_infinity<T>();
    }
    float p[V], top = -__builtin_inff();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = value_of<T>(raw[v / W], v % W);
      top = fmaxf(top, p[v]);
    }
    const int top_key = row_max<LG>(order(top, 0));
    top = top_key > kMinusInfinity ? from_order(top_key) : 0.0f;
    const float away = fabsf(top) <= 0x1p20f ? 0.0f : top;
    if (__any(away != 0.0f)) {
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] -= away;
      top -= away;
    }
    const float shift = top * kLog2e;
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = __builtin_amdgcn_exp2f(fmaf(p[v], kLog2e, -shift));
      sum += p[v];
    }
    sum = row_sum<LG>(sum);
    const bool live = sum != 0.0f;
    const float inv = live ? __builtin_amdgcn_rcpf(sum) : 0.0f;

    float add = dw;                // to dp of its expert, or (renormalized) to dx
    if constexpr (RENORMALIZE) {
      const float x = index >= 0 && live ? widen(row[index]) - away : -__builtin_inff();
      const float e = __builtin_amdgcn_exp2f(fmaf(x, kLog2e, -shift));
      const float all = row_sum<LG>(e);
      const float w = all > 0.0f ? e * __builtin_amdgcn_rcpf(all) : 0.0f;
      add = w * (dw - row_sum<LG>(w * dw));
    }
    if (index >= 0) at[index] = add;
    wave_in_order();
    // the part of dx (renormalized) or of dp that is given, dp's from the loss
    float dot = 0.0f, here[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      here[v] = at[S::column(v)];
      if (!RENORMALIZE) here[v] += coef[S::column(v)];
      p[v] *= inv;
      dot = fmaf(p[v], RENORMALIZE ? coef[S::column(v)] : here[v], dot);
    }
    wave_in_order();
    if (index >= 0) at[index] = 0.0f;
    dot = row_sum<LG>(dot);
    if (first + sub >= end) continue;
    T* out = static_cast<T*>(a.dlogits) + token * a.experts;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float dx[W];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int v = c * W + w;
        dx[w] = RENORMALIZE ? fmaf(p[v], coef[S::column(v)] - dot, here[v]) : p[v] * (here[v] - dot);
      }
      const int col = (c * S::G + lane) * W;
      Chunk o;
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int w = 0; w < 4; ++w) o[w] = __float_as_uint(dx[w]);
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) o[w] = bf16x2_round(dx[2 * w], dx[2 * w + 1]);
      }
      if (__any(!live) && !live) o = Chunk{0, 0, 0, 0};
      if (whole_chunk<S, C>(c, a.experts)) {
        // past the caches, which then still hold logits of the forward pass:
        // 42 us against 48 for 131,072 rows of 256 float32
        __builtin_nontemporal_store(o, reinterpret_cast<typename Loose<T>::type*>(out + col));
      } else {
        T e[W];
        __builtin_memcpy(e, &o, 16);
#pragma unroll
        for (int w = 0; w < W; ++w)
          if (col + w < a.experts) out[col + w] = e[w];
      }
    }
  }
}

// --- launches -----------------------------------------------------------------------------

// One block of a rank takes rows_per_block tokens, a whole number of the
// rows that its waves hold at a time; at most `most` blocks in all (or one a
// rank).  The gradient has 1,024 (four a CU): 512 took 52 us for the 42 of
// 131,072 rows of 256 float32, 2,048 the same.
dim3 grid_of(RouteShape* a, uint32_t rows, uint32_t most) {
  const uint32_t wanted = std::max(1u, (a->tokens + rows - 1) / rows);
  const uint32_t blocks = std::min(wanted, std::max<uint32_t>(1, most / a->nranks));
  const uint32_t each = (wanted + blocks - 1) / blocks;
  a->rows_per_block = each * rows;
  return dim3((wanted + each - 1) / each, a->nranks);
}

hipError_t launch_rows(const void* kernel, dim3 grid, int threads, void* a, hipStream_t stream) {
  void* args[] = {a};
  return hipLaunchKernel(kernel, grid, dim3(threads), args, 0, stream);
}

template <class T, int LG, int C, int RANKS> hipError_t route_as(RouteArgs<RANKS> a, hipStream_t stream) {
  const dim3 grid = grid_of(&a, kRouteWaves * Shape<T, LG, C>::kRows, kRouteBlocks);
  // few blocks are all joined by the last one
  a.group = grid.x * grid.y <= kRouteGroups ? 1 : 16;
  const void* fn = a.top_k <= 2   ? reinterpret_cast<const void*>(&route_kernel<T, LG, C, 2, RANKS>)
                   : a.top_k <= 4 ? reinterpret_cast<const void*>(&route_kernel<T, LG, C, 4, RANKS>)
                                  : reinterpret_cast<const void*>(&route_kernel<T, LG, C, 8, RANKS>);
  return launch_rows(fn, grid, kRouteBlock, &a, stream);
}

template <class T, int LG, int C, int RANKS> hipError_t route_grad_as(RouteGradArgs<RANKS> a, hipStream_t stream) {
  const dim3 grid = grid_of(&a, kWaves * Shape<T, LG, C>::kRows, 1024);
  const void* fn = a.renormalize ? reinterpret_cast<const void*>(&route_grad_kernel<T, LG, C, true, RANKS>)
                                 : reinterpret_cast<const void*>(&route_grad_kernel<T, LG, C, false, RANKS>);
  return launch_rows(fn, grid, kBlock, &a, stream);
}

// The smallest arrangement that holds a row: 8 lanes of 1 to 8 chunks, then
// 16 and 32 lanes.
#define AR_BY_EXPERTS(call, e, a, dtype, stream)                                          \
  if (dtype == AR_FLOAT32)                                                                \
    return e <= 32    ? call<float, 3, 1, N>(a, stream)                                      \
           : e <= 64  ? call<float, 3, 2, N>(a, stream)                                      \
           : e <= 128 ? call<float, 3, 4, N>(a, stream)                                      \
           : e <= 256 ? call<float, 3, 8, N>(a, stream)                                      \
           : e <= 512 ? call<float, 4, 8, N>(a, stream)                                      \
                      : call<float, 5, 8, N>(a, stream);                                     \
  return e <= 64    ? call<uint16_t, 3, 1, N>(a, stream)                                     \
         : e <= 128 ? call<uint16_t, 3, 2, N>(a, stream)                                     \
         : e <= 256 ? call<uint16_t, 3, 4, N>(a, stream)                                     \
         : e <= 512 ? call<uint16_t, 4, 4, N>(a, stream)                                     \
                    : call<uint16_t, 5, 4, N>(a, stream)

}  // namespace

template <int N> hipError_t launch_route(const RouteArgs<N>& a, ar_dtype_t dtype, hipStream_t stream) {
  AR_BY_EXPERTS(route_as, a.experts, a, dtype, stream);
}
template <int N> hipError_t launch_route_grad(const RouteGradArgs<N>& a, ar_dtype_t dtype, hipStream_t stream) {
  AR_BY_EXPERTS(route_grad_as, a.experts, a, dtype, stream);
}

template hipError_t launch_route(const RouteArgs<kFewRanks>&, ar_dtype_t, hipStream_t);
template hipError_t launch_route(const RouteArgs<AR_MAX_RANKS>&, ar_dtype_t, hipStream_t);
template hipError_t launch_route_grad(const RouteGradArgs<kFewRanks>&, ar_dtype_t, hipStream_t);
template hipError_t launch_route_grad(const RouteGradArgs<AR_MAX_RANKS>&, ar_dtype_t, hipStream_t);

}  // namespace ar
