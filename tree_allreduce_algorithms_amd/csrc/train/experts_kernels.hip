// The order of (token, choice) pairs by expert, and the sums over a token's
// pairs with their gradient (gfx950).
#include "train/experts.hpp"

#include "train/wave.hpp"

namespace ar {
namespace {

constexpr int kOrderThreads = kOrderWaves * kWave;
constexpr uint32_t kNone = 0xffffffffu;

// The expert of a pair, kNone for what is no expert's number.
__device__ __forceinline__ uint32_t expert_of(const OrderArgs& a, uint32_t p) {
  const uint32_t e = static_cast<uint32_t>(a.indices[p]);
  return e < static_cast<uint32_t>(a.experts) ? e : kNone;
}

// The wave's part of the block's pairs.
__device__ __forceinline__ void span_of(const OrderArgs& a, uint32_t wave, uint32_t* begin, uint32_t* end) {
  const uint32_t first = blockIdx.x * a.block_pairs;
  const uint32_t last = a.pairs - first < a.block_pairs ? a.pairs : first + a.block_pairs;
  const uint32_t each = a.block_pairs / kOrderWaves;
  *begin = min(first + wave * each, last);
  *end = min(*begin + each, last);
}

__device__ __forceinline__ void count_pairs(const OrderArgs& a, uint32_t* mine, uint32_t begin, uint32_t end) {
  const uint32_t lane = threadIdx.x % kWave;
  for (uint32_t p = begin + lane; p < end; p += kWave) {
    const uint32_t e = expert_of(a, p);
    if (e != kNone) atomicAdd(mine + e, 1u);
  }
}

// A block's pairs of each expert, for long lists.
__global__ __launch_bounds__(kOrderThreads) void order_count(OrderArgs a) {
  extern __shared__ uint32_t counts[];
  for (int e = threadIdx.x; e < a.experts; e += kOrderThreads) counts[e] = 0;
  __syncthreads();
  uint32_t begin, end;
  span_of(a, threadIdx.x / kWave, &begin, &end);
  count_pairs(a, counts, begin, end);
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kOrderThreads)
    a.counts[static_cast<size_t>(blockIdx.x) * a.experts + e] = counts[e];
}

// A stable counting sort.  Every wave takes its pairs in their order, 64 at a
// time; a pair's row is its expert's beginning, plus the expert's pairs of the
// blocks and waves before, plus those of the wave's lower lanes (found by
// comparing the number's bits across the lanes).  A chain of dependent steps binds it,
// not what it moves: 192 pairs of 64 experts 3.3 us, 131,072 of 128 4.9 and 9.7 us.
__global__ __launch_bounds__(kOrderThreads) void order_place(OrderArgs a) {
  extern __shared__ uint32_t next[];       // [waves][experts]; of pairs of other blocks, before and behind
  __shared__ uint32_t part[kOrderWaves];
  const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int experts = a.experts;
  const bool once = a.counts == nullptr;
  uint32_t *const lower_blocks = next + kOrderWaves * experts, *const upper_blocks = lower_blocks + experts;
  for (int i = threadIdx.x; i < experts * static_cast<int>(kOrderWaves + (once ? 2 : 0)); i += kOrderThreads) next[i] = 0;
  __syncthreads();
  uint32_t begin, end;
  span_of(a, wave, &begin, &end);
  uint32_t* mine = next + wave * experts;
  if (once) {
    // (a wave has 64 pairs)
    const uint32_t first = blockIdx.x * kOrderThreads;
    for (uint32_t p0 = threadIdx.x; p0 < a.pairs; p0 += 4 * kOrderThreads) {
      uint32_t key[4];
#pragma unroll
      for (uint32_t q = 0; q < 4; ++q) {
        const uint32_t p = p0 + q * kOrderThreads;
        key[q] = p < a.pairs ? expert_of(a, p) : kNone;
      }
#pragma unroll
      for (uint32_t q = 0; q < 4; ++q) {
        const uint32_t p = p0 - threadIdx.x + q * kOrderThreads;      // a whole block's or none
        if (key[q] != kNone)
          atomicAdd((p < first ? lower_blocks : p > first ? upper_blocks : mine) + key[q], 1u);
      }
    }
  } else {
    count_pairs(a, mine, begin, end);
  }
  __syncthreads();

  // thread e has expert e (at most 1,024 of both): its pairs in all blocks, and
  // in those before this one
  const int e = threadIdx.x;
  uint32_t all = 0, before = 0;
  if (e < experts) {
    if (once) {
      before = lower_blocks[e];
      all = before + upper_blocks[e];
      for (uint32_t w = 0; w < kOrderWaves; ++w) all += next[w * experts + e];
    } else {
      for (uint32_t b = 0; b < a.blocks; b += 8) {
        uint32_t n[8];
#pragma unroll
        for (uint32_t q = 0; q < 8; ++q)
          n[q] = b + q < a.blocks ? a.counts[static_cast<size_t>(b + q) * experts + e] : 0;
#pragma unroll
        for (uint32_t q = 0; q < 8; ++q) {
          all += n[q];
          before += b + q < blockIdx.x ? n[q] : 0;
        }
      }
    }
  }
  // where each expert begins: a scan over the threads
  uint32_t sum = all;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint32_t up = __shfl_up(sum, d);
    if (static_cast<int>(lane) >= d) sum += up;
  }
  if (lane == kWave - 1) part[wave] = sum;
  __syncthreads();
  uint32_t live = 0, lower = 0;
  for (uint32_t w = 0; w < kOrderWaves; ++w) {
    lower += w < wave ? part[w] : 0;
    live += part[w];
  }
  sum += lower;
  if (e < experts) {
    uint32_t at = sum - all + before;
    for (uint32_t w = 0; w < kOrderWaves; ++w) {
      const uint32_t n = next[w * experts + e];
      next[w * experts + e] = at;
      at += n;
    }
    if (blockIdx.x == 0) {
      a.offsets[e + 1] = static_cast<int32_t>(sum);
      if (e == 0) a.offsets[0] = 0;
    }
  }
  __syncthreads();

  for (uint32_t p0 = begin; p0 < end; p0 += kWave) {
    const uint32_t p = p0 + lane;
    const uint32_t key = p < end ? expert_of(a, p) : kNone;
    uint64_t same = __ballot(key != kNone);
#pragma unroll
    for (int bit = 0; bit < 10; ++bit) {
      const uint64_t ones = __ballot((key >> bit) & 1);
      same &= (key >> bit) & 1 ? ones : ~ones;
    }
    if (p < end) {
      int32_t row = -1;
      if (key != kNone) {
        const uint32_t rank = __popcll(same & ((1ull << lane) - 1));
        row = static_cast<int32_t>(mine[key] + rank);
        a.order[row] = static_cast<int32_t>(p);
      }
      a.position[p] = row;
    }
    // every lane has read before the first of each group counts on, and reads
    // what was counted in the next round
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (key != kNone && (same & ((1ull << lane) - 1)) == 0) mine[key] += __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  // behind the last pair that has an expert
  for (uint32_t i = live + blockIdx.x * kOrderThreads + threadIdx.x; i < a.pairs; i += a.blocks * kOrderThreads)
    a.order[i] = -1;
}

// --- sums over a token's pairs ------------------------------------------------------

// Eight bfloat16 at any element's address.
union Eight {
  typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t Words;
  uint16_t v[8];
  Words words;
};

__device__ __forceinline__ float to_float(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

// Round to nearest, ties to even; NaN stays NaN.
__device__ __forceinline__ uint16_t to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>(u >> 16 | 0x40);
  return static_cast<uint16_t>((u + 0x7fffu + (u >> 16 & 1)) >> 16);
}

// The `n` (up to 8) elements at p, zeros behind them.  PAST: past the caches.
template <bool PAST> __device__ __forceinline__ Eight read(const uint16_t* p, uint32_t n) {
  Eight r = {};
  if (n == 8) {
    const Eight::Words* from = reinterpret_cast<const Eight::Words*>(p);
    r.words = PAST ? __builtin_nontemporal_load(from) : *from;
    return r;
  }
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i)
    if (i < n) r.v[i] = p[i];
  return r;
}
template <bool PAST> __device__ __forceinline__ void write(uint16_t* p, const Eight& x, uint32_t n) {
  if (n == 8) {
    Eight::Words* to = reinterpret_cast<Eight::Words*>(p);
    if (PAST)
      __builtin_nontemporal_store(x.words, to);
    else
      *to = x.words;
    return;
  }
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i)
    if (i < n) p[i] = x.v[i];
}

// A row's part of eight from `part` on; over the row's end its last eight, some of
// them the part before's too.
__device__ __forceinline__ uint32_t first_of(uint32_t part, uint32_t size) {
  return part + 8 <= size || size < 8 ? part : size - 8;
}

constexpr int kSumThreads = 256;
constexpr uint32_t kLine = 64;        // elements of a cache line

// out_t = sum over the choices k that have an expert of w_tk y_row(t,k), added
// up in float32 in the order of k.  A thread has eight columns of a token; a
// block has `lanes` of a token's threads, so whole tokens where they are short.
// 131,072 rows of 1,024: 55 us with the rows read past the caches, 70 through them;
// what it moves at 6.2 TB/s takes 49.  The rows of WAY choices are under way at
// a time: 8,192 pairs, two a token, 5.4 us with two, 6.6 with four; 131,072, eight a
// token, 58 with two, 55 with four, 54 with eight, which cost tokens of four a
// microsecond.
template <int WAY, bool PAST>
__global__ __launch_bounds__(kSumThreads) void combine(CombineArgs a, uint32_t lanes) {
  const uint32_t per_block = kSumThreads / lanes, in_block = threadIdx.x / lanes;
  const uint64_t part = (static_cast<uint64_t>(blockIdx.y) * lanes + threadIdx.x % lanes) * 8;
  if (in_block >= per_block || part >= a.size) return;
  const uint32_t c = first_of(static_cast<uint32_t>(part), a.size), n = min(8u, a.size);
  const uint16_t* y = static_cast<const uint16_t*>(a.y) + c;
  uint16_t* out = static_cast<uint16_t*>(a.out) + c;
  for (uint64_t t = static_cast<uint64_t>(blockIdx.x) * per_block + in_block; t < a.tokens;
       t += static_cast<uint64_t>(gridDim.x) * per_block) {
    const uint64_t first = t * a.top_k;
    float sum[8] = {};
    for (int k = 0; k < a.top_k; k += WAY) {
      uint32_t row[WAY];
      float w[WAY];
      Eight r[WAY];
#pragma unroll
      for (int q = 0; q < WAY; ++q) {
        row[q] = k + q < a.top_k ? static_cast<uint32_t>(a.position[first + k + q]) : kNone;
        w[q] = a.weights == nullptr || k + q >= a.top_k ? 1.0f : a.weights[first + k + q];
      }
#pragma unroll
      for (int q = 0; q < WAY; ++q) r[q] = read<PAST>(y + row[q] * a.y_stride, row[q] < a.pairs ? n : 0);
#pragma unroll
      for (int q = 0; q < WAY; ++q)
        if (row[q] < a.pairs)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[q], to_float(r[q].v[i]), sum[i]);
    }
    Eight o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = to_bf16(sum[i]);
    write<false>(out + t * a.size, o, n);
  }
}

// dy_i = w_p dout_t and dw_p = dout_t . y_i, i the row of pair p of token t; a
// wave has a pair, a block neighbours, whose token is mostly the same.  Rows that
// belong to no pair become 0.  131,072 rows of 1,024: 94 us with y's and dy's rows
// past the caches, 184 through them; what it moves at 6.2 TB/s takes 92.
// ENDS: rows are not in whole parts of eight.
template <bool ENDS, bool PAST>
__global__ __launch_bounds__(kSumThreads) void combine_grad(CombineArgs a) {
  constexpr uint32_t kWaves = kSumThreads / kWave, kRound = kWave * 8;
  const uint32_t lane = threadIdx.x % kWave;
  const uint32_t id = blockIdx.x * kWaves + threadIdx.x / kWave, waves = gridDim.x * kWaves;
  uint16_t* dy = static_cast<uint16_t*>(a.out);
  const uint32_t pairs = a.tokens * a.top_k;
  for (uint32_t p = id; p < pairs; p += waves) {
    const uint32_t row = static_cast<uint32_t>(a.position[p]);
    float dot = 0.0f;
    if (row < a.pairs) {
      const uint16_t* dout = static_cast<const uint16_t*>(a.dout) + p / a.top_k * a.dout_stride;
      const uint16_t* y = static_cast<const uint16_t*>(a.y) + row * a.y_stride;
      uint16_t* to = dy + static_cast<uint64_t>(row) * a.size;
      const float w = a.weights[p];
      for (uint32_t c = lane * 8; c < a.size; c += 2 * kRound) {
        const uint32_t part[2] = {c, c + kRound};
        uint32_t at[2], n[2];
        Eight d[2], r[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          at[h] = ENDS ? first_of(part[h], a.size) : part[h];
          n[h] = part[h] < a.size ? ENDS ? min(8u, a.size) : 8 : 0;
          d[h] = read<false>(dout + at[h], n[h]);
          r[h] = read<PAST>(y + at[h], n[h]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t counted = part[h] - at[h];      // by the part before
          Eight o;
#pragma unroll
          for (uint32_t i = 0; i < 8; ++i) {
            const float x = to_float(d[h].v[i]), sum = __builtin_fmaf(x, to_float(r[h].v[i]), dot);
            dot = ENDS && i < counted ? dot : sum;
            o.v[i] = to_bf16(w * x);
          }
          if (PAST && a.size % kLine == 0)
            write<true>(to + at[h], o, n[h]);
          else
            write<false>(to + at[h], o, n[h]);
        }
      }
      dot = wave_sum(dot);
    }
    if (lane == 0) a.dweights[p] = dot;
  }
  const uint32_t live = min(static_cast<uint32_t>(max(a.offsets[a.experts], 0)), a.pairs);
  const Eight zero = {};
  for (uint32_t row = live + id; row < a.pairs; row += waves)
    for (uint32_t c = lane * 8; c < a.size; c += kRound)
      write<false>(dy + static_cast<uint64_t>(row) * a.size + c, zero, min(8u, a.size - c));
}

}  // namespace

// Rows of this size and more are read and written past the caches, if they are
// whole cache lines: parts of lines are better met there, 131,072 rows of 1,000 in
// 52 us instead of 61.  The gradient, which has twice as much under way, reads
// those too past the caches from four times the size on (108 us instead of 118;
// 72,000 rows of 515 54 instead of 44), but writes them through (115 so).
constexpr uint64_t kPastBytes = 32ull << 20;
static bool past_caches(const CombineArgs& a, bool gradient) {
  const uint64_t bytes = static_cast<uint64_t>(a.pairs) * a.size * 2;
  return bytes >= kPastBytes && (a.size % kLine == 0 || (gradient && bytes >= 4 * kPastBytes));
}

hipError_t launch_expert_order_count(const OrderArgs& a, hipStream_t stream) {
  order_count<<<a.blocks, kOrderThreads, static_cast<size_t>(a.experts) * sizeof(uint32_t), stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_expert_order_place(const OrderArgs& a, hipStream_t stream) {
  order_place<<<a.blocks, kOrderThreads, static_cast<size_t>(a.experts) * (kOrderWaves + (a.counts == nullptr ? 2 : 0)) * sizeof(uint32_t), stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_expert_combine(const CombineArgs& a, hipStream_t stream) {
  const uint32_t per = (a.size - 1) / 8 + 1, lanes = per < kSumThreads ? per : kSumThreads;
  const uint32_t tokens = kSumThreads / lanes, blocks = (a.tokens - 1) / tokens + 1;
  const dim3 grid(blocks < 65536 ? blocks : 65536, (per - 1) / lanes + 1);
  const auto kernel = a.top_k <= 2 ? (past_caches(a, false) ? combine<2, true> : combine<2, false>)
                                   : (past_caches(a, false) ? combine<4, true> : combine<4, false>);
  kernel<<<grid, kSumThreads, 0, stream>>>(a, lanes);
  return hipGetLastError();
}

hipError_t launch_expert_combine_grad(const CombineArgs& a, hipStream_t stream) {
  const uint32_t per = kSumThreads / kWave;
  const uint32_t pairs = a.tokens * static_cast<uint32_t>(a.top_k), rows = pairs > a.pairs ? pairs : a.pairs;
  const uint32_t blocks = (rows - 1) / per + 1;
  const auto kernel = a.size % 8 != 0 ? (past_caches(a, true) ? combine_grad<true, true> : combine_grad<true, false>)
                                      : (past_caches(a, true) ? combine_grad<false, true> : combine_grad<false, false>);
  kernel<<<blocks < 65536 ? blocks : 65536, kSumThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace ar
