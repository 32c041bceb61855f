// Matrix products grouped by expert, and the gradient of the experts' weights
// (gfx950).
#include "train/experts.hpp"

#include "train/tile.hpp"
#include "train/wave.hpp"

namespace ar {
namespace {

struct __attribute__((packed, aligned(2))) Chunk {
  u32x4 v;
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

__device__ __forceinline__ uint32_t two_bf16(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) __bf16 two;
  two t = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, t);
}

constexpr int kTileM = 128, kTileN = 128, kWavesM = 2, kWavesN = 2;
constexpr int kThreads = kWavesM * kWavesN * kWave;
constexpr int kPartM = kTileM / kWavesM / 16, kPartN = kTileN / kWavesN / 16;

// Blocks come to the XCDs in turn; of `n` tiles in order each XCD gets
// neighbours, which share operands in its L2.
__device__ __forceinline__ uint32_t near_tile(uint32_t block, uint32_t n) {
  constexpr uint32_t kXcds = 8;
  const uint32_t x = block % kXcds;
  return x * (n / kXcds) + min(x, n % kXcds) + block / kXcds;
}

// --- products ----------------------------------------------------------------------

// The expert and the row tile of unit `id`, when the experts' pairs (and those
// without one, as a last group) are cut into tiles of kTileM rows; `total` of
// them.  Every lane has some neighbouring groups.
struct Unit {
  int expert;
  uint32_t lo, hi;      // rows of the tile
};

__device__ __forceinline__ uint32_t tiles_of(const ProductArgs& a, int e) {
  uint32_t lo, hi;
  rows_of(a.offsets, a.experts, e, a.pairs, &lo, &hi);
  return (hi - lo + kTileM - 1) / kTileM;
}

// y_i = x_t(i) W_e(i) for the rows of an expert; 0 for rows without one.
//
// A block has kTileM rows of one expert and kTileN columns.  The grid is cut
// for any distribution of the pairs (the counts stay on the GPU): each block
// finds its tile from the experts' beginnings, and blocks past the last end.
template <bool BR, bool DIRECT>
__global__ __launch_bounds__(kThreads, 2) void expert_product(ProductArgs a) {
  using SA = Staged<kTileM, false>;
  using SB = Staged<kTileN, BR>;
  constexpr int kStage = SA::kBytes + SB::kBytes;
  constexpr int kLoadsA = SA::kChunks / kThreads, kLoadsB = SB::kChunks / kThreads;
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);

  // the tile
  const int groups = a.experts + 1, each = (groups + kWave - 1) / kWave;
  uint32_t mine = 0;
  for (int i = 0; i < each; ++i)
    if (lane * each + i < groups) mine += tiles_of(a, lane * each + i);
  uint32_t upto = mine;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint32_t up = __shfl_up(upto, d);
    if (lane >= d) upto += up;
  }
  const uint64_t total = static_cast<uint64_t>(__shfl(upto, kWave - 1)) * a.tiles_n;
  if (blockIdx.x >= total) return;
  const uint32_t tile = near_tile(blockIdx.x, static_cast<uint32_t>(total));
  const uint32_t unit = tile / a.tiles_n, n0 = tile % a.tiles_n * kTileN;
  const int owner = __popcll(__ballot(upto <= unit));
  uint32_t rest = unit - __shfl(upto - mine, owner);
  int e = owner * each;
  for (uint32_t n; rest >= (n = tiles_of(a, e)); ++e) rest -= n;
  e = __builtin_amdgcn_readfirstlane(e);
  uint32_t lo, hi;
  rows_of(a.offsets, a.experts, e, a.pairs, &lo, &hi);
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lo + rest * kTileM);
  hi = __builtin_amdgcn_readfirstlane(hi);

  f32x4 acc[kPartM][kPartN];
#pragma unroll
  for (auto& row : acc)
#pragma unroll
    for (auto& x : row) x = f32x4{0, 0, 0, 0};

  const int steps = e < a.experts ? static_cast<int>((a.in + kStep - 1) / kStep) : 0;
  const int wave_m = wave / kWavesN * (kTileM / kWavesM), wave_n = wave % kWavesN * (kTileN / kWavesN);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  const uint16_t* w = static_cast<const uint16_t*>(a.w) + (e < a.experts ? e * a.w_expert : 0);

  // the thread's chunks of a step: the rows of x that they come from, kNowhere for none
  uint32_t row[kLoadsA], at[kLoadsA], col[kLoadsB], line[kLoadsB];
#pragma unroll
  for (int j = 0; j < kLoadsA; ++j) {
    const int slot = j * kThreads + tid, l = slot / SA::kPerLine;
    const uint32_t r = m0 + l;
    row[j] = kNowhere;
    at[j] = SA::place(l, slot % SA::kPerLine) * 8;
    if (steps > 0 && r < hi) {
      uint32_t t = r;
      if (a.order != nullptr) t = static_cast<uint32_t>(a.order[r]) / static_cast<uint32_t>(a.top_k);
      if (t < a.x_rows) row[j] = t;
    }
  }
#pragma unroll
  for (int j = 0; j < kLoadsB; ++j) {
    const int slot = j * kThreads + tid, l = slot / SB::kPerLine;
    line[j] = l;
    col[j] = SB::place(l, slot % SB::kPerLine) * 8;
  }
  // elements of a chunk that lie in the operands
  const auto left_a = [&](int j, uint32_t k) {
    return row[j] == kNowhere || k + at[j] >= a.in ? 0 : static_cast<int>(min(a.in - k - at[j], 8u));
  };
  const auto left_b = [&](int j, uint32_t k) {
    const uint32_t kk = BR ? k + line[j] : k + col[j], n = BR ? n0 + col[j] : n0 + line[j];
    if (kk >= a.in || n >= a.out) return 0;
    return static_cast<int>(min(BR ? a.out - n : a.in - kk, 8u));
  };

  if (DIRECT) {
    const Source from_x(x), from_w(w);
    const uint32_t base = lds_address(lds) + wave * (kWave * 16);
    const uint32_t x_bytes = static_cast<uint32_t>(a.x_stride) * 2, w_bytes = static_cast<uint32_t>(a.w_line) * 2;
    const auto issue = [&](int step) {
      const uint32_t to = base + (step & 1) * kStage, k = step * kStep;
#pragma unroll
      for (int j = 0; j < kLoadsA; ++j)
        load_to_lds(from_x, left_a(j, k) ? row[j] * x_bytes + (k + at[j]) * 2 : kNowhere,
                    __builtin_amdgcn_readfirstlane(to + j * kThreads * 16));
#pragma unroll
      for (int j = 0; j < kLoadsB; ++j)
        load_to_lds(from_w,
                    left_b(j, k) ? (BR ? (k + line[j]) * w_bytes + (n0 + col[j]) * 2
                                       : (n0 + line[j]) * w_bytes + (k + col[j]) * 2)
                                 : kNowhere,
                    __builtin_amdgcn_readfirstlane(to + SA::kBytes + j * kThreads * 16));
    };
    if (steps > 0) issue(0);
    for (int s = 0; s < steps; ++s) {
      settled();
      __builtin_amdgcn_s_barrier();
      if (s + 1 < steps) issue(s + 1);
      const char* stage = lds + (s & 1) * kStage;
      multiply_step<kPartM, kPartN, bf16x8, 1, SA, SB>(stage, stage + SA::kBytes, wave_m, wave_n, lane, acc);
    }
  } else {
    u32x4 ra[kLoadsA], rb[kLoadsB];
    const auto load = [&](int step) {
      const uint32_t k = step * kStep;
#pragma unroll
      for (int j = 0; j < kLoadsA; ++j) ra[j] = read_elements(x + row[j] * a.x_stride + k + at[j], left_a(j, k));
#pragma unroll
      for (int j = 0; j < kLoadsB; ++j)
        rb[j] = read_elements(BR ? w + (k + line[j]) * a.w_line + n0 + col[j] : w + (n0 + line[j]) * a.w_line + k + col[j],
                              left_b(j, k));
    };
    if (steps > 0) load(0);
    for (int s = 0; s < steps; ++s) {
      char* stage = lds + (s & 1) * kStage;
#pragma unroll
      for (int j = 0; j < kLoadsA; ++j) *reinterpret_cast<u32x4*>(stage + (j * kThreads + tid) * 16) = ra[j];
#pragma unroll
      for (int j = 0; j < kLoadsB; ++j)
        *reinterpret_cast<u32x4*>(stage + SA::kBytes + (j * kThreads + tid) * 16) = rb[j];
      __syncthreads();
      if (s + 1 < steps) load(s + 1);
      multiply_step<kPartM, kPartN, bf16x8, 1, SA, SB>(stage, stage + SA::kBytes, wave_m, wave_n, lane, acc);
    }
  }

#pragma unroll
  for (int i = 0; i < kPartM; ++i) {
    const uint32_t r = m0 + wave_m + 16 * i + lane % 16;
    if (r >= hi) continue;
    uint16_t* y = static_cast<uint16_t*>(a.y) + static_cast<uint64_t>(r) * a.out;
#pragma unroll
    for (int j = 0; j < kPartN; ++j) {
      const uint32_t n = n0 + wave_n + 16 * j + 4 * (lane / 16);
      if (n >= a.out) continue;
      const uint2 v = {two_bf16(acc[i][j][0], acc[i][j][1]), two_bf16(acc[i][j][2], acc[i][j][3])};
      if (a.vec) {
        *reinterpret_cast<uint2*>(y + n) = v;
      } else {
        const uint32_t part[4] = {v.x & 0xffff, v.x >> 16, v.y & 0xffff, v.y >> 16};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n + q < a.out) y[n + q] = static_cast<uint16_t>(part[q]);
      }
    }
  }
}

// --- the weights' gradient ------------------------------------------------------------

// dW_e = sum over the rows i of expert e of x_t(i)^T dy_i: a block has a tile of
// one expert's matrix and goes over the expert's rows, 64 at a time.  An expert
// without rows gets zeros.
template <bool WIDE, bool DIRECT>
__global__ __launch_bounds__(kThreads, 2) void expert_weight_grad(WeightGradArgs a) {
  using SA = Staged<kTileM, true>;
  using SB = Staged<kTileN, true>;
  constexpr int kStage = SA::kBytes + SB::kBytes;
  constexpr int kLoadsA = SA::kChunks / kThreads, kLoadsB = SB::kChunks / kThreads;
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const uint32_t tile = near_tile(blockIdx.x, gridDim.x), of_expert = a.tiles_m * a.tiles_n;
  const int e = tile / of_expert;
  const uint32_t m0 = tile % of_expert / a.tiles_n * kTileM, n0 = tile % a.tiles_n * kTileN;
  uint32_t lo, hi;
  rows_of(a.offsets, a.experts, e, a.pairs, &lo, &hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  const int steps = static_cast<int>((hi - lo + kStep - 1) / kStep);

  f32x4 acc[kPartM][kPartN];
#pragma unroll
  for (auto& row : acc)
#pragma unroll
    for (auto& x : row) x = f32x4{0, 0, 0, 0};

  const int wave_m = wave / kWavesN * (kTileM / kWavesM), wave_n = wave % kWavesN * (kTileN / kWavesN);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  const uint16_t* dy = static_cast<const uint16_t*>(a.dy);
  uint32_t line_a[kLoadsA], col_a[kLoadsA], line_b[kLoadsB], col_b[kLoadsB], token[kLoadsA];
#pragma unroll
  for (int j = 0; j < kLoadsA; ++j) {
    const int slot = j * kThreads + tid;
    line_a[j] = slot / SA::kPerLine;
    col_a[j] = m0 + SA::place(line_a[j], slot % SA::kPerLine) * 8;
  }
#pragma unroll
  for (int j = 0; j < kLoadsB; ++j) {
    const int slot = j * kThreads + tid;
    line_b[j] = slot / SB::kPerLine;
    col_b[j] = n0 + SB::place(line_b[j], slot % SB::kPerLine) * 8;
  }
  // the rows of x of a step's lines, found one step before their loads are issued
  const auto find = [&](int step) {
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j) {
      const uint32_t r = lo + step * kStep + line_a[j];
      token[j] = kNowhere;
      if (r < hi) {
        uint32_t t = r;
        if (a.order != nullptr) t = static_cast<uint32_t>(a.order[r]) / static_cast<uint32_t>(a.top_k);
        if (t < a.x_rows) token[j] = t;
      }
    }
  };
  const auto left_a = [&](int j) {
    return token[j] == kNowhere || col_a[j] >= a.in ? 0 : static_cast<int>(min(a.in - col_a[j], 8u));
  };
  const auto left_b = [&](int j, uint32_t r) {
    return r >= hi || col_b[j] >= a.out ? 0 : static_cast<int>(min(a.out - col_b[j], 8u));
  };

  if (steps > 0) find(0);
  if (DIRECT) {
    const Source from_x(x), from_y(dy + lo * a.dy_stride);
    const uint32_t base = lds_address(lds) + wave * (kWave * 16);
    const uint32_t x_bytes = static_cast<uint32_t>(a.x_stride) * 2, y_bytes = static_cast<uint32_t>(a.dy_stride) * 2;
    const auto issue = [&](int step) {
      const uint32_t to = base + (step & 1) * kStage;
#pragma unroll
      for (int j = 0; j < kLoadsA; ++j)
        load_to_lds(from_x, left_a(j) ? token[j] * x_bytes + col_a[j] * 2 : kNowhere,
                    __builtin_amdgcn_readfirstlane(to + j * kThreads * 16));
#pragma unroll
      for (int j = 0; j < kLoadsB; ++j) {
        const uint32_t r = step * kStep + line_b[j];
        load_to_lds(from_y, left_b(j, lo + r) ? r * y_bytes + col_b[j] * 2 : kNowhere,
                    __builtin_amdgcn_readfirstlane(to + SA::kBytes + j * kThreads * 16));
      }
    };
    if (steps > 0) issue(0);
    if (steps > 1) find(1);
    for (int s = 0; s < steps; ++s) {
      settled();
      __builtin_amdgcn_s_barrier();
      if (s + 1 < steps) issue(s + 1);
      if (s + 2 < steps) find(s + 2);
      const char* stage = lds + (s & 1) * kStage;
      multiply_step<kPartM, kPartN, bf16x8, 1, SA, SB>(stage, stage + SA::kBytes, wave_m, wave_n, lane, acc);
    }
  } else {
    u32x4 ra[kLoadsA], rb[kLoadsB];
    const auto load = [&](int step) {
#pragma unroll
      for (int j = 0; j < kLoadsA; ++j) ra[j] = read_elements(x + token[j] * a.x_stride + col_a[j], left_a(j));
#pragma unroll
      for (int j = 0; j < kLoadsB; ++j) {
        const uint32_t r = lo + step * kStep + line_b[j];
        rb[j] = read_elements(dy + r * a.dy_stride + col_b[j], left_b(j, r));
      }
    };
    if (steps > 0) load(0);
    if (steps > 1) find(1);
    for (int s = 0; s < steps; ++s) {
      char* stage = lds + (s & 1) * kStage;
#pragma unroll
      for (int j = 0; j < kLoadsA; ++j) *reinterpret_cast<u32x4*>(stage + (j * kThreads + tid) * 16) = ra[j];
#pragma unroll
      for (int j = 0; j < kLoadsB; ++j)
        *reinterpret_cast<u32x4*>(stage + SA::kBytes + (j * kThreads + tid) * 16) = rb[j];
      __syncthreads();
      if (s + 1 < steps) load(s + 1);
      if (s + 2 < steps) find(s + 2);
      multiply_step<kPartM, kPartN, bf16x8, 1, SA, SB>(stage, stage + SA::kBytes, wave_m, wave_n, lane, acc);
    }
  }

#pragma unroll
  for (int i = 0; i < kPartM; ++i) {
    const uint32_t m = m0 + wave_m + 16 * i + lane % 16;
    if (m >= a.in) continue;
    const uint64_t first = (static_cast<uint64_t>(e) * a.in + m) * a.out;
#pragma unroll
    for (int j = 0; j < kPartN; ++j) {
      const uint32_t n = n0 + wave_n + 16 * j + 4 * (lane / 16);
      if (n >= a.out) continue;
      if (WIDE) {
        float* to = static_cast<float*>(a.dw) + first + n;
        if (a.vec) {
          *reinterpret_cast<f32x4*>(to) = acc[i][j];
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < a.out) to[q] = acc[i][j][q];
        }
      } else {
        uint16_t* to = static_cast<uint16_t*>(a.dw) + first + n;
        const uint2 v = {two_bf16(acc[i][j][0], acc[i][j][1]), two_bf16(acc[i][j][2], acc[i][j][3])};
        if (a.vec) {
          *reinterpret_cast<uint2*>(to) = v;
        } else {
          const uint32_t part[4] = {v.x & 0xffff, v.x >> 16, v.y & 0xffff, v.y >> 16};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + q < a.out) to[q] = static_cast<uint16_t>(part[q]);
        }
      }
    }
  }
}

}  // namespace

// Tiles for any distribution of the pairs: whole ones, and a part of one for
// every group that has pairs.
uint64_t expert_product_blocks(uint64_t pairs, int experts, uint64_t out) {
  const uint64_t groups = static_cast<uint64_t>(experts) + 1;
  return (pairs / kTileM + (groups < pairs ? groups : pairs)) * ((out + kTileN - 1) / kTileN);
}

uint64_t expert_weight_grad_blocks(int experts, uint64_t in, uint64_t out) {
  return experts * ((in + kTileM - 1) / kTileM) * ((out + kTileN - 1) / kTileN);
}

hipError_t launch_expert_product(const ProductArgs& args, bool out_contiguous, bool direct, hipStream_t stream) {
  ProductArgs a = args;
  a.tiles_n = (a.out + kTileN - 1) / kTileN;
  const dim3 grid(static_cast<uint32_t>(expert_product_blocks(a.pairs, a.experts, a.out)));
  if (out_contiguous)
    (direct ? expert_product<true, true> : expert_product<true, false>)<<<grid, kThreads, 0, stream>>>(a);
  else
    (direct ? expert_product<false, true> : expert_product<false, false>)<<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_expert_weight_grad(const WeightGradArgs& args, ar_dtype_t dw_dtype, bool direct,
                                     hipStream_t stream) {
  WeightGradArgs a = args;
  a.tiles_m = (a.in + kTileM - 1) / kTileM;
  a.tiles_n = (a.out + kTileN - 1) / kTileN;
  const dim3 grid(static_cast<uint32_t>(expert_weight_grad_blocks(a.experts, a.in, a.out)));
  if (dw_dtype == AR_FLOAT32)
    (direct ? expert_weight_grad<true, true> : expert_weight_grad<true, false>)<<<grid, kThreads, 0, stream>>>(a);
  else
    (direct ? expert_weight_grad<false, true> : expert_weight_grad<false, false>)<<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace ar
