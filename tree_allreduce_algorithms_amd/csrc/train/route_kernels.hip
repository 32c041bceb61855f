// Expert router kernels (gfx950): the choice of experts with its weights,
// counts and balance loss, and the gradient of the logits.
//
// A token's logits are one row.  A wave takes a row at a time, lane l the
// columns l, l + 64, ...; the row is read once and stays in registers.
#include "device_common.hpp"
#include "train/route.hpp"
#include "train/wave.hpp"

namespace ar {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kWaves = kBlock / kWave;

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_widen(x); }
template <class T> __device__ __forceinline__ T narrow(float x) {
  if constexpr (sizeof(T) == 4)
    return x;
  else
    return bf16_round(x);
}

// exp(x - top): 0 for x = -infinity, NaN for a NaN.
__device__ __forceinline__ float exp_from(float x, float top) {
  return __builtin_amdgcn_exp2f((x - top) * kLog2e);
}

// Order-preserving bits of a logit; 0 for -infinity and NaN, which are never
// chosen.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);   // -0 and 0 are equal
  const uint32_t key = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return x > -__builtin_inff() ? key : 0u;
}
__device__ __forceinline__ float from_key(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// The tokens [begin, end) of a block.
struct Rows {
  uint32_t begin, end;
  template <class A> __device__ explicit Rows(const A& a) {
    begin = blockIdx.x * a.rows_per_block;
    end = min(begin + a.rows_per_block, a.tokens);
  }
};

template <class T, int V>
__device__ __forceinline__ void load_row(const T* row, int experts, bool live, float* x) {
  const int lane = threadIdx.x % kWave;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int col = lane + v * kWave;
    x[v] = live && col < experts ? widen(row[col]) : -__builtin_inff();
  }
}

template <class T, int V> __global__ __launch_bounds__(kBlock) void route_kernel(RouteArgs a) {
  __shared__ uint32_t hist[V * kWave];
  __shared__ float sums[kWaves][V * kWave];
  __shared__ uint32_t tokens[kWaves];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int rank = blockIdx.y;
  for (int i = threadIdx.x; i < V * kWave; i += kBlock) hist[i] = 0;
  __syncthreads();

  float total[V];
#pragma unroll
  for (int v = 0; v < V; ++v) total[v] = 0.0f;
  uint32_t live_rows = 0;
  const Rows rows(a);
  for (uint32_t i = rows.begin + wave; i < rows.end; i += kWaves) {
    const uint8_t* mask = static_cast<const uint8_t*>(a.masks.p[rank]);
    const bool masked = mask != nullptr && mask[i] == 0;
    float x[V];
    load_row<T, V>(static_cast<const T*>(a.logits.p[rank]) + i * a.row_stride, a.experts, !masked, x);
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = order_key(x[v]);

    // the largest key, then its lowest column, top_k times; lane k keeps the k-th
    int index = -1;
    float value = 0.0f, top = 0.0f;
    for (int k = 0; k < a.top_k; ++k) {
      uint32_t best = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) best = max(best, key[v]);
      best = wave_max(best);
      if (best == 0) break;
      uint32_t first = 0;       // counted from the end: the largest is the lowest column
#pragma unroll
      for (int v = V - 1; v >= 0; --v)
        if (key[v] == best) first = AR_MAX_EXPERTS - (lane + v * kWave);
      const int col = AR_MAX_EXPERTS - static_cast<int>(wave_max(first));
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (col == lane + v * kWave) key[v] = 0;
      if (k == 0) top = from_key(best);
      if (lane == k) {
        index = col;
        value = from_key(best);
      }
    }

    float e[V], sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      e[v] = exp_from(x[v], top);
      sum += e[v];
    }
    sum = wave_sum(sum);
    const bool live = sum != 0.0f;          // a NaN lives
    const float inv = live ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) total[v] = fmaf(e[v], inv, total[v]);
    live_rows += live ? 1 : 0;

    const float mine = index >= 0 ? exp_from(value, top) : 0.0f;
    float weight = mine * inv;
    if (a.renormalize) weight = live ? mine / wave_sum(mine) : 0.0f;
    if (sum != sum) weight = sum;
    if (lane < a.top_k) {
      const uint64_t at = (static_cast<uint64_t>(rank) * a.tokens + i) * a.top_k + lane;
      a.indices[at] = index;
      a.weights[at] = weight;
      if (index >= 0) atomicAdd(&hist[index], 1u);
    }
  }

  // the block's sums into the call's
#pragma unroll
  for (int v = 0; v < V; ++v) sums[wave][lane + v * kWave] = total[v];
  if (lane == 0) tokens[wave] = live_rows;
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kBlock) {
    float s = sums[0][e];
    for (int w = 1; w < kWaves; ++w) s += sums[w][e];
    if (s >= 0.0f) {
      const uint64_t fixed = static_cast<uint64_t>(static_cast<double>(s) * 4294967296.0 + 0.5);
      if (fixed != 0)
        shared_add(&a.sums->share[e], fixed);
    } else {
      shared_store(&a.sums->not_finite, 1u);
    }
    if (hist[e] != 0)
      shared_add(&a.sums->counts[rank * a.experts + e], hist[e]);
  }
  if (threadIdx.x == 0) {
    uint32_t n = 0;
    for (int w = 0; w < kWaves; ++w) n += tokens[w];
    shared_add(&a.sums->tokens, n);
  }
  if (!last_to_arrive(&a.sums->arrived, gridDim.x * gridDim.y)) return;

  // the last block: counts, shares and loss, and the workspace zero again
  RouteSums* ws = a.sums;
  const double n = shared_load(&ws->tokens);
  const bool bad = shared_load(&ws->not_finite) != 0;
  const double unit = n > 0 ? a.experts / (a.top_k * n * n) : 0.0;
  double loss = 0.0;
  for (int e = threadIdx.x; e < a.experts; e += kBlock) {
    uint64_t chosen = 0;
    for (int r = 0; r < a.nranks; ++r) {
      const int at = r * a.experts + e;
      const uint32_t c = shared_load(&ws->counts[at]);
      ws->counts[at] = 0;
      a.counts[at] = static_cast<int32_t>(c);
      chosen += c;
    }
    const uint64_t fixed = shared_load(&ws->share[e]);
    ws->share[e] = 0;
    const double share = unit * static_cast<double>(chosen);
    a.share[e] = static_cast<float>(share);
    loss += share * (static_cast<double>(fixed) / 4294967296.0);
  }
  loss = block_sum<kBlock>(loss);      // its barriers come after every thread's reads above
  if (threadIdx.x == 0) {
    *a.loss = bad ? __builtin_nanf("") : static_cast<float>(loss);
    ws->tokens = ws->not_finite = ws->arrived = 0;
  }
}

template <class T, int V> __global__ __launch_bounds__(kBlock) void route_grad_kernel(RouteGradArgs a) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int rank = blockIdx.y;
  const float dloss = a.dloss != nullptr ? *a.dloss : 0.0f;
  float coef[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int col = lane + v * kWave;
    coef[v] = col < a.experts ? dloss * a.share[col] : 0.0f;
  }
  const Rows rows(a);
  for (uint32_t i = rows.begin + wave; i < rows.end; i += kWaves) {
    const uint8_t* mask = static_cast<const uint8_t*>(a.masks.p[rank]);
    const bool masked = mask != nullptr && mask[i] == 0;
    const T* row = static_cast<const T*>(a.logits.p[rank]) + i * a.row_stride;
    float x[V], top = -__builtin_inff();
    load_row<T, V>(row, a.experts, !masked, x);
#pragma unroll
    for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
    const uint32_t top_key = wave_max(order_key(top));
    top = top_key != 0 ? from_key(top_key) : 0.0f;
    float p[V], sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = exp_from(x[v], top);
      sum += p[v];
    }
    sum = wave_sum(sum);
    const bool live = sum != 0.0f;
    const float inv = live ? 1.0f / sum : 0.0f;

    // lane k has the k-th chosen expert's part
    int index = -1;
    float dw = 0.0f;
    const uint64_t token = static_cast<uint64_t>(rank) * a.tokens + i;
    if (lane < a.top_k && a.dweights.p[0] != nullptr && live) {
      index = a.indices[token * a.top_k + lane];
      if (static_cast<uint32_t>(index) >= static_cast<uint32_t>(a.experts)) index = -1;
      if (index >= 0)
        dw = static_cast<const float*>(a.dweights.p[rank])[static_cast<uint64_t>(i) * a.top_k + lane];
    }
    float add = dw;                // to dp of its expert, or (renormalized) to dx
    if (a.renormalize) {
      const float e = index >= 0 ? exp_from(widen(row[index]), top) : 0.0f;
      const float all = wave_sum(e);
      const float w = all > 0.0f ? e / all : 0.0f;
      add = w * (dw - wave_sum(w * dw));
    }
    float at[V];
#pragma unroll
    for (int v = 0; v < V; ++v) at[v] = 0.0f;
    for (int k = 0; k < a.top_k; ++k) {
      const int col = __shfl(index, k);
      const float y = __shfl(add, k);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (col == lane + v * kWave) at[v] = y;
    }
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] *= inv;
      dot = fmaf(p[v], a.renormalize ? coef[v] : coef[v] + at[v], dot);
    }
    dot = wave_sum(dot);
    T* out = static_cast<T*>(a.dlogits) + token * a.experts;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = lane + v * kWave;
      const float dx = a.renormalize ? fmaf(p[v], coef[v] - dot, at[v]) : p[v] * (coef[v] + at[v] - dot);
      if (col < a.experts) out[col] = narrow<T>(live ? dx : 0.0f);
    }
  }
}

// Enough blocks to fill the chip, each with rows for all its waves.
template <class A> dim3 grid_of(A* a) {
  const uint32_t most = std::max<uint32_t>(1, 2048 / a->nranks);
  const uint32_t blocks = std::max<uint32_t>(1, std::min((a->tokens + kWaves - 1) / kWaves, most));
  a->rows_per_block = (a->tokens + blocks - 1) / blocks;
  return dim3(a->tokens == 0 ? 1 : (a->tokens + a->rows_per_block - 1) / a->rows_per_block, a->nranks);
}

template <class A>
hipError_t launch_rows(const void* kernel, dim3 grid, A* a, hipStream_t stream) {
  void* args[] = {a};
  return hipLaunchKernel(kernel, grid, dim3(kBlock), args, 0, stream);
}

#define AR_BY_EXPERTS(kernel, T, e)                                              \
  ((e) <= 64    ? reinterpret_cast<const void*>(&kernel<T, 1>)                   \
   : (e) <= 128 ? reinterpret_cast<const void*>(&kernel<T, 2>)                   \
   : (e) <= 256 ? reinterpret_cast<const void*>(&kernel<T, 4>)                   \
   : (e) <= 512 ? reinterpret_cast<const void*>(&kernel<T, 8>)                   \
                : reinterpret_cast<const void*>(&kernel<T, 16>))

}  // namespace

hipError_t launch_route(RouteArgs a, ar_dtype_t dtype, hipStream_t stream) {
  const void* fn = dtype == AR_FLOAT32 ? AR_BY_EXPERTS(route_kernel, float, a.experts)
                                       : AR_BY_EXPERTS(route_kernel, uint16_t, a.experts);
  const dim3 grid = grid_of(&a);
  return launch_rows(fn, grid, &a, stream);
}

hipError_t launch_route_grad(RouteGradArgs a, ar_dtype_t dtype, hipStream_t stream) {
  const void* fn = dtype == AR_FLOAT32 ? AR_BY_EXPERTS(route_grad_kernel, float, a.experts)
                                       : AR_BY_EXPERTS(route_grad_kernel, uint16_t, a.experts);
  const dim3 grid = grid_of(&a);
  return launch_rows(fn, grid, &a, stream);
}

}  // namespace ar
