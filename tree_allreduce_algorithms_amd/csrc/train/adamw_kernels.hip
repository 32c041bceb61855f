// AdamW kernels (gfx950): the gradient norm, the step, the decoding of 8-bit
// states.
//
// All three are streams: each element's values are read once and written
// once, by one lane, so HBM bandwidth is what bounds them.  Work is cut into
// tiles of one tensor (the plan's table), a tile into steps of 1,024
// elements, 256 for each of the block's four waves: a wave's 256 elements are
// one block of an 8-bit state, whose maxima therefore need one reduction
// across its lanes and no LDS.
#include "device_common.hpp"
#include "train/adamw.hpp"
#include "train/wave.hpp"

namespace ar {
namespace {

constexpr int kQuad = 4;                                  // elements a lane holds of each step
static_assert(kWave * kQuad == AR_ADAMW_BLOCK, "a wave's step is a block of an 8-bit state");
static_assert(kBlock * kQuad == kAdamwStep, "a block's step");

// --- accesses ------------------------------------------------------------------

// Four consecutive elements in one access, past the caches where it is 16
// bytes (nothing here is used twice).
template <class T> struct Quad {
  T e[kQuad];
};

template <class T> __device__ __forceinline__ Quad<T> load_quad(const T* p) {
  using Raw = uint32_t __attribute__((ext_vector_type(sizeof(T))));   // sizeof(T) words
  if constexpr (sizeof(T) == 1) {
    return __builtin_bit_cast(Quad<T>, __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p)));
  } else {
    return __builtin_bit_cast(Quad<T>, __builtin_nontemporal_load(reinterpret_cast<const Raw*>(p)));
  }
}
template <class T> __device__ __forceinline__ void store_quad(T* p, const Quad<T>& v) {
  using Raw = uint32_t __attribute__((ext_vector_type(sizeof(T))));
  if constexpr (sizeof(T) == 1) {
    __builtin_nontemporal_store(__builtin_bit_cast(uint32_t, v), reinterpret_cast<uint32_t*>(p));
  } else {
    __builtin_nontemporal_store(__builtin_bit_cast(Raw, v), reinterpret_cast<Raw*>(p));
  }
}

// The lane's four elements of a wave's 256: neighbours where the tensor is
// aligned and the 256 are whole, else 64 apart, each only if it exists.
struct Lanes {
  uint64_t base;      // the wave's first element
  uint32_t live;      // how many of the 256 exist
  bool quad;
  __device__ uint32_t at(int j) const {
    const uint32_t lane = threadIdx.x % kWave;
    return quad ? lane * kQuad + j : j * kWave + lane;
  }
  template <class T> __device__ Quad<T> load(const void* p) const {
    const T* q = static_cast<const T*>(p) + base;
    if (quad) return load_quad<T>(q + threadIdx.x % kWave * kQuad);
    Quad<T> v;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) v.e[j] = at(j) < live ? q[at(j)] : T(0);
    return v;
  }
  template <class T> __device__ void store(void* p, const Quad<T>& v) const {
    T* q = static_cast<T*>(p) + base;
    if (quad) {
      store_quad<T>(q + threadIdx.x % kWave * kQuad, v);
    } else {
#pragma unroll
      for (int j = 0; j < kQuad; ++j)
        if (at(j) < live) q[at(j)] = v.e[j];
    }
  }
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_widen(x); }

template <class T> __device__ __forceinline__ Quad<T> narrow(const Quad<float>& x) {
  if constexpr (sizeof(T) == 4) {
    return x;
  } else {
    const Words<2> w = {{bf16x2_round(x.e[0], x.e[1]), bf16x2_round(x.e[2], x.e[3])}};
    return __builtin_bit_cast(Quad<T>, w);
  }
}

// The wave's part of step `s` of a tile; false where nothing of it exists.
__device__ __forceinline__ bool lanes_of(const AdamwTensor& t, uint64_t tile_begin, uint32_t s, Lanes* l) {
  l->base = tile_begin + s * kAdamwStep + threadIdx.x / kWave * AR_ADAMW_BLOCK;
  if (l->base >= t.count) return false;
  const uint64_t left = t.count - l->base;
  l->live = left < AR_ADAMW_BLOCK ? static_cast<uint32_t>(left) : AR_ADAMW_BLOCK;
  l->quad = t.vec != 0 && l->live == AR_ADAMW_BLOCK;
  return true;
}

// --- the norm --------------------------------------------------------------------

// The squares are exact in 64 bits and are added up in 64 bits: the clipping
// factor must be the float32 nearest to max_norm / norm, because 8-bit codes
// are decided on what it scales.  Every block leaves a partial sum; the one
// that arrives last adds them up in their order and sets the factor, so a
// norm is one launch and its bits do not depend on which block that is.
template <class G> __global__ __launch_bounds__(kBlock) void adamw_norm_kernel(AdamwNormArgs a) {
  const AdamwTensor* tensors = reinterpret_cast<const AdamwTensor*>(a.plan + a.tensors_at);
  const AdamwTile* tiles = reinterpret_cast<const AdamwTile*>(a.plan + a.tiles_at);
  double* partials = reinterpret_cast<double*>(a.plan + a.partials_at);
  AdamwHead* head = reinterpret_cast<AdamwHead*>(a.plan);

  double sum = 0.0;
  for (uint32_t i = blockIdx.x; i < a.tiles; i += gridDim.x) {
    const AdamwTile tile = tiles[i];
    const AdamwTensor& t = tensors[tile.tensor];
    const uint64_t begin = static_cast<uint64_t>(tile.index) * a.tile_elements;
    for (uint32_t s = 0; s < a.tile_elements / kAdamwStep; ++s) {
      Lanes l;
      if (!lanes_of(t, begin, s, &l)) break;
      const Quad<G> g = l.load<G>(t.g);
#pragma unroll
      for (int j = 0; j < kQuad; ++j) {
        const double x = widen(g.e[j]);
        sum = fma(x, x, sum);
      }
    }
  }
  sum = block_sum<kBlock>(sum);
  if (threadIdx.x == 0)
    __hip_atomic_store(&partials[blockIdx.x], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (!last_to_arrive(&head->arrived, gridDim.x)) return;

  double all = 0.0;
  for (uint32_t i = threadIdx.x; i < gridDim.x; i += kBlock)
    all += __hip_atomic_load(&partials[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  all = block_sum<kBlock>(all);
  if (threadIdx.x == 0) {
    const double norm = fabs(a.grad_scale) * sqrt(all);
    const float c = norm > a.max_norm ? static_cast<float>(a.max_norm / norm) : 1.0f;
    head->factor = static_cast<float>(c * a.grad_scale);
    head->arrived = 0;
    if (a.norm != nullptr) *a.norm = static_cast<float>(norm);
  }
}

// --- 8-bit states ------------------------------------------------------------------

// Largest of the wave's doubles, none of them negative; a NaN counts as
// larger than all.  Such numbers are ordered as their bits are: first the
// high words, then the low words of the lanes that have the highest.
__device__ __forceinline__ double wave_max(double x) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, x);
  const uint32_t hi = static_cast<uint32_t>(bits >> 32), lo = static_cast<uint32_t>(bits);
  const uint32_t top = wave_max(hi);
  const uint32_t low = wave_max(hi == top ? lo : 0u);
  return __builtin_bit_cast(double, static_cast<uint64_t>(top) << 32 | low);
}

__device__ __forceinline__ double larger(double x, double y) {
  const uint64_t a = __builtin_bit_cast(uint64_t, x), b = __builtin_bit_cast(uint64_t, y);
  return __builtin_bit_cast(double, a > b ? a : b);
}

// Values between the codes j and j + 1 round to j up to the middle between
// their squares, j^2 + j + 1/2 = (j + 1/2)^2 + 1/4 (in units of the scale).
// y = sqrt(t - 1/4) in float32 is off by far less than 1/2, so the only
// border that can be wrong is that between j and j + 1 with j = floor(y); it
// is decided in float64, where scale * border is exact.
__device__ __forceinline__ float border_below(float t, float most) {
  return fminf(floorf(__builtin_amdgcn_sqrtf(fmaxf(t - 0.25f, 0.0f))), most);
}

struct ScaleM {
  double a, inv;
  bool ok;
  // `top`: the block's largest |m|
  __device__ explicit ScaleM(double top, float* scale) {
    const float s = static_cast<float>(top / 16129.0);
    ok = s > 0.0f && s < __builtin_inff();
    *scale = s < __builtin_inff() ? s : __builtin_nanf("");
    a = s;
    inv = 1.0 / a;
  }
  __device__ int8_t code(double m) const {
    const double x = fabs(m);
    const float j = border_below(static_cast<float>(x * inv), 126.0f);
    const float border = fmaf(j, j, j) + 0.5f;
    const int q = static_cast<int>(j) + (x > a * static_cast<double>(border) ? 1 : 0);
    return static_cast<int8_t>(ok ? (m < 0.0 ? -q : q) : 0);
  }
};

struct ScaleV {
  double r, inv2;
  bool ok;
  // `top`: the block's largest v
  __device__ explicit ScaleV(double top, float* scale) {
    const float s = static_cast<float>(sqrt(top) / 65025.0);
    ok = s > 0.0f && s < __builtin_inff();
    *scale = s < __builtin_inff() ? s : __builtin_nanf("");
    r = s;
    inv2 = 1.0 / (r * r);
  }
  __device__ uint8_t code(double v) const {
    const float t = __builtin_amdgcn_sqrtf(static_cast<float>(v * inv2));
    const float j = border_below(t, 254.0f);
    const double border = r * static_cast<double>(fmaf(j, j, j) + 0.5f);
    int u = static_cast<int>(j) + (v > border * border ? 1 : 0);
    if (u == 0 && v > 0.0) u = 1;
    return static_cast<uint8_t>(ok ? u : 0);
  }
};

__device__ __forceinline__ double value_m(int8_t code, double a) {
  const int q = code;
  return static_cast<double>(q * (q < 0 ? -q : q)) * a;
}
__device__ __forceinline__ double value_v(uint8_t code, double r) {
  const uint32_t u = code;
  const double s = static_cast<double>(u * u) * r;
  return s * s;
}

// --- the step ------------------------------------------------------------------------

__device__ __forceinline__ float updated(float p, float m, float v, const AdamwStepArgs& a) {
  const float u = (m / a.bc1) / (sqrtf(v / a.bc2) + a.eps);
  return p - fmaf(a.lr_wd, p, a.lr * u);
}

template <class P, class G, bool COPY, int BITS>
__global__ __launch_bounds__(kBlock) void adamw_step_kernel(AdamwStepArgs a) {
  const AdamwTensor* tensors = reinterpret_cast<const AdamwTensor*>(a.plan + a.tensors_at);
  const AdamwTile tile = reinterpret_cast<const AdamwTile*>(a.plan + a.tiles_at)[blockIdx.x];
  const AdamwTensor& t = tensors[tile.tensor];
  const float c = a.clip ? reinterpret_cast<const AdamwHead*>(a.plan)->factor : a.factor;
  const uint64_t begin = static_cast<uint64_t>(tile.index) * a.tile_elements;

  for (uint32_t s = 0; s < a.tile_elements / kAdamwStep; ++s) {
    Lanes l;
    if (!lanes_of(t, begin, s, &l)) break;
    const Quad<P> p = l.load<P>(t.p);
    const Quad<G> g = l.load<G>(t.g);
    Quad<float> out;
    if constexpr (BITS == 32) {
      Quad<float> m = l.load<float>(t.m), v = l.load<float>(t.v);
      const float b1 = static_cast<float>(a.b1), one_b1 = static_cast<float>(a.one_b1);
      const float b2 = static_cast<float>(a.b2), one_b2 = static_cast<float>(a.one_b2);
#pragma unroll
      for (int j = 0; j < kQuad; ++j) {
        const float x = widen(g.e[j]) * c;
        m.e[j] = fmaf(b1, m.e[j], one_b1 * x);
        v.e[j] = fmaf(b2, v.e[j], one_b2 * x * x);
        out.e[j] = updated(widen(p.e[j]), m.e[j], v.e[j], a);
      }
      l.store<float>(t.m, m);
      l.store<float>(t.v, v);
    } else {
      const uint64_t block = l.base / AR_ADAMW_BLOCK;
      const Quad<int8_t> qm = l.load<int8_t>(t.m);
      const Quad<uint8_t> qv = l.load<uint8_t>(t.v);
      const double am = t.ms[block], rv = t.vs[block];
      double m[kQuad], v[kQuad], top_m = 0.0, top_v = 0.0;
      // m and v in float64: a code changes where a value crosses a border
#pragma unroll
      for (int j = 0; j < kQuad; ++j) {
        const double x = static_cast<double>(widen(g.e[j])) * static_cast<double>(c);
        m[j] = a.b1 * value_m(qm.e[j], am) + a.one_b1 * x;
        v[j] = a.b2 * value_v(qv.e[j], rv) + a.one_b2 * x * x;
        if (!l.quad && l.at(j) >= l.live) m[j] = v[j] = 0.0;
        top_m = larger(top_m, fabs(m[j]));
        top_v = larger(top_v, v[j]);
        out.e[j] = updated(widen(p.e[j]), static_cast<float>(m[j]), static_cast<float>(v[j]), a);
      }
      // every lane stores the same scale to the same place
      const ScaleM sm(wave_max(top_m), &t.ms[block]);
      const ScaleV sv(wave_max(top_v), &t.vs[block]);
      Quad<int8_t> nm;
      Quad<uint8_t> nv;
#pragma unroll
      for (int j = 0; j < kQuad; ++j) {
        nm.e[j] = sm.code(m[j]);
        nv.e[j] = sv.code(v[j]);
      }
      l.store<int8_t>(t.m, nm);
      l.store<uint8_t>(t.v, nv);
    }
    l.store<P>(t.p, narrow<P>(out));
    if constexpr (COPY) l.store<uint16_t>(t.copy, narrow<uint16_t>(out));
  }
}

// --- decoding ---------------------------------------------------------------------------

// One rounding per value: the products are taken in float64 (m's is exact
// there) and rounded to float32.
template <bool SIGNED>
__global__ __launch_bounds__(kBlock) void adamw_dequantize_kernel(const void* codes, const float* scales,
                                                                  uint64_t count, int quads, float* out) {
  using C = typename std::conditional<SIGNED, int8_t, uint8_t>::type;
  const uint64_t blocks = (count - 1) / AR_ADAMW_BLOCK + 1;
  const uint64_t stride = static_cast<uint64_t>(gridDim.x) * (kBlock / kWave);
  for (uint64_t b = static_cast<uint64_t>(blockIdx.x) * (kBlock / kWave) + threadIdx.x / kWave;
       b < blocks; b += stride) {
    Lanes l;
    l.base = b * AR_ADAMW_BLOCK;
    const uint64_t left = count - l.base;
    l.live = left < AR_ADAMW_BLOCK ? static_cast<uint32_t>(left) : AR_ADAMW_BLOCK;
    l.quad = quads != 0 && l.live == AR_ADAMW_BLOCK;
    const double scale = scales[b];
    const Quad<C> q = l.load<C>(codes);
    Quad<float> x;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
      if constexpr (SIGNED)
        x.e[j] = static_cast<float>(value_m(q.e[j], scale));
      else
        x.e[j] = static_cast<float>(value_v(q.e[j], scale));
    }
    l.store<float>(out, x);
  }
}

template <class A> hipError_t launch1(void (*kernel)(A), uint64_t blocks, const A& a, hipStream_t stream) {
  A copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(static_cast<uint32_t>(blocks)),
                         dim3(kBlock), args, 0, stream);
}

template <int BITS>
void (*step_kernel_for(bool p32, bool g32, bool copy))(AdamwStepArgs) {
  if (!p32) return g32 ? adamw_step_kernel<uint16_t, float, false, BITS> : adamw_step_kernel<uint16_t, uint16_t, false, BITS>;
  if (copy) return g32 ? adamw_step_kernel<float, float, true, BITS> : adamw_step_kernel<float, uint16_t, true, BITS>;
  return g32 ? adamw_step_kernel<float, float, false, BITS> : adamw_step_kernel<float, uint16_t, false, BITS>;
}

}  // namespace

hipError_t launch_adamw_norm(const AdamwNormArgs& a, ar_dtype_t grad_dtype, hipStream_t stream) {
  const uint32_t blocks = std::max(1u, std::min(a.tiles, kMaxNormBlocks));
  return launch1(grad_dtype == AR_FLOAT32 ? adamw_norm_kernel<float> : adamw_norm_kernel<uint16_t>,
                 blocks, a, stream);
}

hipError_t launch_adamw_step(const AdamwStepArgs& a, uint32_t tiles, ar_dtype_t param_dtype,
                             ar_dtype_t grad_dtype, int state_bits, bool copy, hipStream_t stream) {
  const bool p32 = param_dtype == AR_FLOAT32, g32 = grad_dtype == AR_FLOAT32;
  return launch1(state_bits == 32 ? step_kernel_for<32>(p32, g32, copy) : step_kernel_for<8>(p32, g32, copy),
                 tiles, a, stream);
}

hipError_t launch_adamw_dequantize(const void* codes, const float* scales, uint64_t count,
                                   bool is_signed, float* out, hipStream_t stream) {
  const uint64_t blocks = ((count - 1) / AR_ADAMW_BLOCK) / (kBlock / kWave) + 1;
  const uint32_t grid = static_cast<uint32_t>(std::min<uint64_t>(blocks, 1u << 20));
  int quads = reinterpret_cast<uintptr_t>(codes) % 4 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
  void* args[] = {&codes, &scales, &count, &quads, &out};
  const void* fn = is_signed ? reinterpret_cast<const void*>(&adamw_dequantize_kernel<true>)
                             : reinterpret_cast<const void*>(&adamw_dequantize_kernel<false>);
  return hipLaunchKernel(fn, dim3(grid), dim3(kBlock), args, 0, stream);
}

}  // namespace ar
