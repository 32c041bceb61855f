// AdamW kernels (gfx950): the gradient norm, the step, the decoding of 8-bit
// states.
//
// All three are streams: each element's values are read once and written
// once, by one lane, so HBM bandwidth is what should bound them.  Work is cut
// into tiles of kAdamwTile elements of one tensor (the plan's table), one
// quarter for each of the block's four waves, sixteen elements a lane.
//
// Times in this file are medians of a kernel trace unless they say otherwise;
// pairs that compare two forms were taken together, on one card, when the one
// was chosen.
#include <type_traits>

#include "device_common.hpp"
#include "train/adamw.hpp"
#include "train/wave.hpp"

namespace ar {
namespace {

constexpr int kWaveElements = kAdamwTile / (kBlock / kWave);
constexpr int kQuads = kWaveElements / kWave / 4;          // of a lane
static_assert(kWaveElements == 4 * AR_ADAMW_BLOCK && kQuads == 4, "a wave's part is four blocks of an 8-bit state");

// --- accesses ------------------------------------------------------------------

// Four consecutive elements, one access where they are aligned and all exist.
template <class T> struct Quad {
  T e[4];
};

// Four bytes of codes are a quarter of what a lane group touches of a line at
// a time, so they go through the caches; wider ones stream past (nothing here
// is used twice).
template <class T> struct Raw {
  using type = uint32_t __attribute__((ext_vector_type(sizeof(T))));
};
template <> struct Raw<int8_t> {
  using type = uint32_t;
};
template <> struct Raw<uint8_t> {
  using type = uint32_t;
};

// A pointer out of the plan's table is to global memory, which the compiler
// cannot see; an access that might be to LDS as well (flat) costs more.
#define AR_GLOBAL __attribute__((address_space(1)))

// Which elements of a tensor a lane has: kQuads runs of four, `step` apart.
// WHOLE: all of the wave's elements exist, and the tensor's pointers allow
// quads.  Only the last wave of a tensor goes element by element, or all of
// them where one of its arrays is aligned to its elements only: 300M in eight
// shards of an odd count take 1.4 to 1.5 times as long (norm of float32, 32-bit
// steps) to 2.2 times (norm of bfloat16, 8-bit steps).
template <bool WHOLE> struct Lanes {
  uint64_t first, count;
  uint32_t step;
  __device__ uint64_t at(int q) const { return first + q * step; }
  template <class T> __device__ __forceinline__ Quad<T> load(const void* p, int q) const {
    using R = typename Raw<T>::type;
    if constexpr (WHOLE) {
      const AR_GLOBAL T* x = (const AR_GLOBAL T*)p + at(q);
      if constexpr (sizeof(T) == 1)
        return __builtin_bit_cast(Quad<T>, *(const AR_GLOBAL R*)x);
      else
        return __builtin_bit_cast(Quad<T>, __builtin_nontemporal_load((const AR_GLOBAL R*)x));
    }
    // past the end the last element again, so that no access waits for a branch
    Quad<T> v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.e[i] = ((const AR_GLOBAL T*)p)[at(q) + i < count ? at(q) + i : count - 1];
    return v;
  }
  template <class T> __device__ __forceinline__ void store(void* p, int q, const Quad<T>& v) const {
    using R = typename Raw<T>::type;
    AR_GLOBAL T* x = (AR_GLOBAL T*)p + at(q);
    if constexpr (WHOLE) {
      if constexpr (sizeof(T) == 1)
        *(AR_GLOBAL R*)x = __builtin_bit_cast(R, v);
      else
        __builtin_nontemporal_store(__builtin_bit_cast(R, v), (AR_GLOBAL R*)x);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at(q) + i < count) x[i] = v.e[i];
    }
  }
};

// The wave's first element of a tile.
__device__ __forceinline__ uint64_t wave_begin(const AdamwTile& tile) {
  return static_cast<uint64_t>(tile.index) * kAdamwTile + wave_uniform(threadIdx.x / kWave) * kWaveElements;
}

__device__ __forceinline__ bool whole(uint64_t begin, uint64_t count, bool vec) {
  return vec && begin + kWaveElements <= count;
}

// A wave's elements spread so that each of its accesses is one run.
template <bool WHOLE> __device__ __forceinline__ Lanes<WHOLE> runs_of(uint64_t begin, uint64_t count) {
  return {begin + threadIdx.x % kWave * 4, count, 4 * kWave};
}

// The same elements, each row of 16 lanes with one block of 256: an access is
// four runs of 16 quads, and a block's maximum needs the row only.
template <bool WHOLE> __device__ __forceinline__ Lanes<WHOLE> rows_of(uint64_t begin, uint64_t count) {
  const uint32_t lane = threadIdx.x % kWave;
  return {begin + lane / 16 * AR_ADAMW_BLOCK + lane % 16 * 4, count, 64};
}

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

// --- the norm --------------------------------------------------------------------

template <bool WHOLE, class G>
__device__ __forceinline__ void add_squares(const AdamwTensor& t, uint64_t begin, double* sum) {
  const Lanes<WHOLE> l = runs_of<WHOLE>(begin, t.count);
  Quad<G> g[kQuads];
#pragma unroll
  for (int q = 0; q < kQuads; ++q) g[q] = l.template load<G>(t.g, q);
#pragma unroll
  for (int q = 0; q < kQuads; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double x = WHOLE || l.at(q) + i < t.count ? widen(g[q].e[i]) : 0.0f;
      sum[i] = fma(x, x, sum[i]);
    }
}

// The squares are exact in 64 bits and are added up in 64 bits: the clipping
// factor must be the float32 nearest to max_norm / norm, because 8-bit codes
// are decided on what it scales.  Every block leaves a partial sum; the last
// block of each group adds up the group's, the last group the groups', each
// in their order, so a norm is one launch and its bits do not depend on which
// block comes last.  300M float32 take 170 to 176 us (6.8-7.1 TB/s), 300M
// bfloat16 94 us (6.4 TB/s).  Of 1,024 blocks in groups of 32, 2,048 in groups
// of 64 and 512 in groups of 16 the first were best for both together: 175
// and 87 us back to back, against 175 and 97, and 167 and 130.
template <class G> __global__ __launch_bounds__(kBlock) void adamw_norm_kernel(AdamwNormArgs a) {
  const AdamwTensor* tensors = reinterpret_cast<const AdamwTensor*>(a.plan + a.tensors_at);
  const AdamwTile* tiles = reinterpret_cast<const AdamwTile*>(a.plan + a.tiles_at);
  AdamwSums* sums = reinterpret_cast<AdamwSums*>(a.plan + a.sums_at);

  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  for (uint32_t i = blockIdx.x; i < a.tiles; i += gridDim.x) {
    const AdamwTile tile = tiles[i];
    const AdamwTensor& t = tensors[tile.tensor];
    const uint64_t begin = wave_begin(tile);
    if (begin >= t.count) continue;
    if (whole(begin, t.count, t.vec != 0))
      add_squares<true, G>(t, begin, sum);
    else
      add_squares<false, G>(t, begin, sum);
  }
  double all = block_sum<kBlock>((sum[0] + sum[1]) + (sum[2] + sum[3]));

  const uint32_t group = blockIdx.x / kNormGroup, groups = (gridDim.x - 1) / kNormGroup + 1;
  const uint32_t first = group * kNormGroup, members = min(kNormGroup, gridDim.x - first);
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) shared_store(&sums->of_block[blockIdx.x], all);
    if (!last_to_arrive(&sums->arrived[group].count, members)) return;
    all = block_sum<kBlock>(threadIdx.x < members ? shared_load(&sums->of_block[first + threadIdx.x]) : 0.0);
    if (threadIdx.x == 0) sums->arrived[group].count = 0;
    if (groups > 1) {
      if (threadIdx.x == 0) shared_store(&sums->of_group[group], all);
      if (!last_to_arrive(&sums->groups_arrived.count, groups)) return;
      all = block_sum<kBlock>(threadIdx.x < groups ? shared_load(&sums->of_group[threadIdx.x]) : 0.0);
      if (threadIdx.x == 0) sums->groups_arrived.count = 0;
    }
  }
  if (threadIdx.x == 0) {
    const double norm = fabs(a.grad_scale) * sqrt(all);
    const float c = norm > a.max_norm ? static_cast<float>(a.max_norm / norm) : 1.0f;
    sums->factor = static_cast<float>(c * a.grad_scale);
    if (a.norm != nullptr) *a.norm = static_cast<float>(norm);
  }
}

// --- 8-bit states ------------------------------------------------------------------

// Maximum over each row of 16 lanes, by rotations: every lane gets it.
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
#define AR_DPP_MAX(ctrl) \
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), ctrl, 0xf, 0xf, false)))
  AR_DPP_MAX(0x121);
  AR_DPP_MAX(0x122);
  AR_DPP_MAX(0x124);
  AR_DPP_MAX(0x128);
#undef AR_DPP_MAX
  return x;
}

// Largest of a row's doubles, none of them negative; a NaN counts as larger
// than all.  Such numbers are ordered as their bits are: first the high
// words, then the low words of the lanes that have the highest.
__device__ __forceinline__ double row_max(double x) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, x);
  const uint32_t hi = static_cast<uint32_t>(bits >> 32), lo = static_cast<uint32_t>(bits);
  const uint32_t top = row_max(hi);
  const uint32_t low = row_max(hi == top ? lo : 0u);
  return __builtin_bit_cast(double, static_cast<uint64_t>(top) << 32 | low);
}

// Values between the codes j and j + 1 round to j up to the middle between
// their squares, j^2 + j + 1/2 (in units of the scale).  A float32 root of
// the value in those units is off by far less than 1/2, and the border lies
// between (j + 1/2)^2 and (j + 3/4)^2, so the only border in doubt is that
// above j = floor(root); it is decided in float64, where scale * border is
// exact.  An 8-bit step thus rounds as the definition in 64 bits does, at the
// price of a few float64 instructions a value.
//
// Scales are one per block and therefore the same in a row's lanes, which
// share the cost of computing them over sixteen elements each.
__device__ __forceinline__ uint32_t floor_root(float t) {
  return static_cast<uint32_t>(__builtin_amdgcn_sqrtf(t));
}
__device__ __forceinline__ double below_border(uint32_t j) {       // j^2 + j
  return static_cast<double>(__umul24(j, j) + j);
}

// The float32 nearest to x / d: one correction step makes the quotient as
// good as a division's.
__device__ __forceinline__ float quotient(double x, double d, double inv_d) {
  const double q = x * inv_d;
  return static_cast<float>(fma(fma(-q, d, x), inv_d, q));
}

// The roots' arguments come from float32 numbers that the step has anyway,
// |m| and sqrt(v).  Where a scale is `tiny`, they could be subnormal (which
// root and reciprocal take as 0) or the scale's reciprocal infinite, and where
// it is `huge` v could be beyond float32's range: there the arguments are
// taken in float64 instead.
constexpr double kHugeV = 0x1p127;
struct ScaleM {
  double a, half;
  float stored, inv;
  bool tiny;
  // `top`: the block's largest |m|
  __device__ explicit ScaleM(double top) {
    const float s = quotient(top, 16129.0, 1.0 / 16129.0);
    const bool ok = s > 0.0f && s < __builtin_inff();
    stored = s < __builtin_inff() ? s : __builtin_nanf("");
    a = ok ? s : __builtin_inf();                 // no value is above its borders
    half = a * 0.5;
    inv = ok ? __builtin_amdgcn_rcpf(s) : 0.0f;
    tiny = ok && s < 1e-30f;
  }
  template <bool FAR> __device__ __forceinline__ uint32_t code(double m, float m32) const {
    const double x = fabs(m);
    const float t = FAR ? static_cast<float>(tiny ? x * __builtin_amdgcn_rcp(a) : x * inv) : fabsf(m32) * inv;
    const uint32_t j = floor_root(t);
    uint32_t q = j + (x > fma(a, below_border(j), half) ? 1u : 0u);
    if (FAR) q = min(q, 127u);                   // a subnormal scale may be half of what it should be
    const uint32_t sign = static_cast<uint32_t>(static_cast<int>(__builtin_bit_cast(uint64_t, m) >> 32) >> 31);
    return (q ^ sign) - sign;
  }
};

struct ScaleV {
  double r, half, zero;
  float stored, inv;
  bool tiny, huge;
  // `top`: the block's largest v
  __device__ explicit ScaleV(double top) {
    const float s = quotient(sqrt(top), 65025.0, 1.0 / 65025.0);
    const bool ok = s > 0.0f && s < __builtin_inff();
    stored = s < __builtin_inff() ? s : __builtin_nanf("");
    r = ok ? s : __builtin_inf();
    half = r * 0.5;
    zero = ok ? 0.0 : __builtin_inf();
    inv = ok ? __builtin_amdgcn_rcpf(s) : 0.0f;
    tiny = ok && s < 1e-18f;
    huge = !(top < kHugeV);
  }
  template <bool FAR> __device__ __forceinline__ uint32_t code(double v, float root) const {
    const float t = FAR ? static_cast<float>(__builtin_amdgcn_sqrt(v) * (tiny ? __builtin_amdgcn_rcp(r) : inv)) : root * inv;
    const uint32_t j = floor_root(t);
    const double border = fma(r, below_border(j), half);
    uint32_t u = j + (v > border * border ? 1u : 0u);
    if (FAR) u = min(u, 255u);
    return max(u, v > zero ? 1u : 0u);
  }
};

// Four codes as a word; the upper bytes of each are dropped.
__device__ __forceinline__ uint32_t pack(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
  return lo | hi;
}

// What a code stands for in units of its scale (m) or its scale's root (v).
__device__ __forceinline__ double units(int8_t code) {
  const float q = static_cast<float>(code);
  return q * fabsf(q);
}
__device__ __forceinline__ double units(uint8_t code) {
  const float u = static_cast<float>(code);
  return u * u;
}

// --- the step ------------------------------------------------------------------------

// u = (m / bc1) / (sqrt(v / bc2) + eps), with the two corrections moved to
// the factor in front and to eps.  The root and the reciprocal are single
// instructions, off by one step of the last place each; the root takes a
// subnormal v (a root below 1.1e-19) as 0, which shows only beside an eps that
// is hardly larger: see wide_eps().
__device__ __forceinline__ float updated(float p, float m, float root_v, const AdamwStepArgs& a) {
  const float u = m * __builtin_amdgcn_rcpf(root_v + a.eps);
  return p - fmaf(a.lr_wd, p, a.lr * u);
}

// The same from m and v in float64, for a v beyond float32's range and for a
// wide_eps().
__device__ __forceinline__ float updated_far(float p, double m, double v, const AdamwStepArgs& a) {
  const float u = static_cast<float>(m / (sqrt(v) + a.eps64));
  return p - fmaf(a.lr_wd, p, a.lr * u);
}

// Four elements of the 32-bit step.
template <class P, class G>
__device__ __forceinline__ Quad<float> step_quad(const AdamwStepArgs& a, const Quad<P>& p, const Quad<G>& g, float c,
                                                 Quad<float>& m, Quad<float>& v) {
  const float b1 = static_cast<float>(a.b1), one_b1 = static_cast<float>(a.one_b1);
  const float b2 = static_cast<float>(a.b2), one_b2 = static_cast<float>(a.one_b2);
  Quad<float> out;
  if (a.far) {                                   // m' and v' before they are rounded
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double x = static_cast<double>(widen(g.e[i])) * c;
      out.e[i] = updated_far(widen(p.e[i]), fma(a.one_b1, x, a.b1 * m.e[i]),
                             fma(a.one_b2 * x, x, a.b2 * v.e[i]), a);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = widen(g.e[i]) * c;
    m.e[i] = fmaf(b1, m.e[i], one_b1 * x);
    v.e[i] = fmaf(b2, v.e[i], one_b2 * x * x);
    if (!a.far) out.e[i] = updated(widen(p.e[i]), m.e[i], __builtin_amdgcn_sqrtf(v.e[i]), a);
  }
  return out;
}

// One array's kPiece elements between memory and LDS, by one wave, sixteen
// bytes an access.  The plan lets an array begin at any four elements, so in
// memory a bfloat16 access is aligned to eight bytes only (the hardware takes
// it as one access all the same).
constexpr int kPiece = kBlock * 4;
template <class T> struct Staged {
  using type = Raw16;
};
template <> struct Staged<uint16_t> {
  typedef Raw16 type __attribute__((aligned(8)));
};
template <class T, bool KEEP> __device__ __forceinline__ void stage(const void* from, uint64_t begin, Raw16* to) {
  using R = typename Staged<T>::type;
  const AR_GLOBAL R* x = (const AR_GLOBAL R*)((const AR_GLOBAL T*)from + begin) + threadIdx.x % kWave;
  constexpr int N = kPiece * sizeof(T) / 16 / kWave;
  Raw16 r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (KEEP)
      r[i] = x[i * kWave];
    else
      r[i] = __builtin_nontemporal_load(x + i * kWave);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) to[threadIdx.x % kWave + i * kWave] = r[i];
}
template <class T> __device__ __forceinline__ void unstage(const Raw16* from, void* to, uint64_t begin) {
  using R = typename Staged<T>::type;
  AR_GLOBAL R* x = (AR_GLOBAL R*)((AR_GLOBAL T*)to + begin) + threadIdx.x % kWave;
  constexpr int N = kPiece * sizeof(T) / 16 / kWave;
#pragma unroll
  for (int i = 0; i < N; ++i)
    __builtin_nontemporal_store(from[threadIdx.x % kWave + i * kWave], x + i * kWave);
}

// The 32-bit step of kPiece elements by a block, through LDS: wave w reads
// and writes the w-th of the arrays only.  Memory binds it; the detour keeps
// each wave's accesses to one array at a time, in runs of 4 KiB.  Measured,
// with float32 gradients and copies (30 bytes an element): 300M elements
// 1,555 to 1,575 us (5.7-5.8 TB/s), 9M in 250 tensors with bfloat16 gradients
// 40.8 us.  When it was chosen: 1,560 us against 1,585 with all arrays in one
// lane's registers, 1,640 with pieces twice as long and 1,650 with write-back
// stores; 38.9 us against 46.8 in registers.
template <class P, class G, bool COPY, bool KEEP>
__device__ __forceinline__ void step32_staged(const AdamwStepArgs& a, const AdamwTensor& t, uint64_t begin, float c) {
  __shared__ Raw16 lds[4][kPiece / 4];
  const int wave = wave_uniform(threadIdx.x / kWave);
  if (wave == 0) stage<P, KEEP>(t.p, begin, lds[0]);
  else if (wave == 1) stage<G, KEEP>(t.g, begin, lds[1]);
  else if (wave == 2) stage<float, KEEP>(t.m, begin, lds[2]);
  else stage<float, KEEP>(t.v, begin, lds[3]);
  __syncthreads();
  Quad<P>* p = reinterpret_cast<Quad<P>*>(lds[0]) + threadIdx.x;
  Quad<G>* g = reinterpret_cast<Quad<G>*>(lds[1]) + threadIdx.x;
  Quad<float>* m = reinterpret_cast<Quad<float>*>(lds[2]) + threadIdx.x;
  Quad<float>* v = reinterpret_cast<Quad<float>*>(lds[3]) + threadIdx.x;
  Quad<float> nm = *m, nv = *v;
  const Quad<float> out = step_quad<P, G>(a, *p, *g, c, nm, nv);
  *m = nm;
  *v = nv;
  *p = narrow<P>(out);
  if constexpr (COPY && sizeof(G) == 4) __syncthreads();          // the copy takes the gradient's place
  if constexpr (COPY) reinterpret_cast<Quad<uint16_t>*>(lds[1])[threadIdx.x] = narrow<uint16_t>(out);
  __syncthreads();
  if (wave == 0) unstage<P>(lds[0], t.p, begin);
  else if (wave == 1) { if constexpr (COPY) unstage<uint16_t>(lds[1], t.copy, begin); }
  else if (wave == 2) unstage<float>(lds[2], t.m, begin);
  else unstage<float>(lds[3], t.v, begin);
}

// The same without LDS, where not all of the elements exist or the arrays are
// aligned to their elements only.
template <class P, class G, bool COPY>
__device__ __forceinline__ void step32_loose(const AdamwStepArgs& a, const AdamwTensor& t, uint64_t begin, float c) {
  const Lanes<false> l = {begin + threadIdx.x * 4, t.count, 0};
  Quad<float> m = l.template load<float>(t.m, 0), v = l.template load<float>(t.v, 0);
  const Quad<float> out = step_quad<P, G>(a, l.template load<P>(t.p, 0), l.template load<G>(t.g, 0), c, m, v);
  l.template store<float>(t.m, 0, m);
  l.template store<float>(t.v, 0, v);
  l.template store<P>(t.p, 0, narrow<P>(out));
  if constexpr (COPY) l.template store<uint16_t>(t.copy, 0, narrow<uint16_t>(out));
}

template <class P, class G, bool COPY, bool KEEP>
__global__ __launch_bounds__(kBlock) void adamw_step_kernel(AdamwStepArgs a) {
  constexpr uint32_t kPieces = kAdamwTile / kPiece;
  const AdamwTile tile = reinterpret_cast<const AdamwTile*>(a.plan + a.tiles_at)[blockIdx.x / kPieces];
  const AdamwTensor t = reinterpret_cast<const AdamwTensor*>(a.plan + a.tensors_at)[tile.tensor];
  const float c = a.clip ? reinterpret_cast<const AdamwSums*>(a.plan + a.sums_at)->factor : a.factor;
  const uint64_t begin = static_cast<uint64_t>(tile.index) * kAdamwTile + blockIdx.x % kPieces * kPiece;
  if (begin >= t.count) return;
  if (t.vec != 0 && begin + kPiece <= t.count)
    step32_staged<P, G, COPY, KEEP>(a, t, begin, c);
  else
    step32_loose<P, G, COPY>(a, t, begin, c);
}

// The update from m and v, and their codes.  The 8-bit step's arithmetic
// (about 60 instructions an element, a third of them in float64) and its bytes
// take about as long: 300M elements with bfloat16 gradients and copies (16.03
// bytes each) 776 us, 6.2 TB/s; 6.5M with float32 gradients 22.6 us.  A block
// of a state per 16 lanes shares the scales' arithmetic over 16 elements a
// lane; one per wave, four elements a lane, took 2,140 us.
// FAR: a block of the wave is tiny or huge, or ends early, or eps is wide.
// What an element gets does not depend on which of the two forms its wave
// takes.
template <bool FAR, class P, bool COPY, class L>
__device__ __forceinline__ void finish8(const AdamwStepArgs& a, const AdamwTensor& t, const L& l,
                                        const Quad<P> (&p)[kQuads], const double (&m)[kQuads][4],
                                        const double (&v)[kQuads][4], const ScaleM& sm, const ScaleV& sv) {
#pragma unroll
  for (int q = 0; q < kQuads; ++q) {
    Quad<float> out;
    uint32_t nm[4], nv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m32 = static_cast<float>(m[q][i]);
      const float root = __builtin_amdgcn_sqrtf(static_cast<float>(v[q][i]));
      if (FAR && (a.far || v[q][i] >= kHugeV))
        out.e[i] = updated_far(widen(p[q].e[i]), m[q][i], v[q][i], a);
      else
        out.e[i] = updated(widen(p[q].e[i]), m32, root, a);
      nm[i] = sm.template code<FAR>(m[q][i], m32);
      nv[i] = sv.template code<FAR>(v[q][i], root);
    }
    l.template store<P>(t.p, q, narrow<P>(out));
    if constexpr (COPY) l.template store<uint16_t>(t.copy, q, narrow<uint16_t>(out));
    l.template store<int8_t>(t.m, q, __builtin_bit_cast(Quad<int8_t>, pack(nm[0], nm[1], nm[2], nm[3])));
    l.template store<uint8_t>(t.v, q, __builtin_bit_cast(Quad<uint8_t>, pack(nv[0], nv[1], nv[2], nv[3])));
  }
}

template <bool WHOLE, class P, class G, bool COPY>
__device__ __forceinline__ void step8(const AdamwStepArgs& a, const AdamwTensor& t, uint64_t begin, double c) {
  const Lanes<WHOLE> l = rows_of<WHOLE>(begin, t.count);
  const uint64_t block = begin / AR_ADAMW_BLOCK + threadIdx.x % kWave / 16;
  const bool exists = WHOLE || block * AR_ADAMW_BLOCK < t.count;
  // what a lane has past the tensor's end is its last element, in the block
  // of that element too, and stays out of memory
  const uint64_t held = exists ? block : (t.count - 1) / AR_ADAMW_BLOCK;
  AR_GLOBAL float* ms = (AR_GLOBAL float*)t.ms + held;
  AR_GLOBAL float* vs = (AR_GLOBAL float*)t.vs + held;
  const double am = *ms, rv = *vs;

  // m and v in float64 (a code changes where a value crosses a border), the
  // factors of a block's sixteen elements a lane taken together first
  const double old_m = a.b1 * am, old_v = a.root_b2 * rv;
  const double new_m = a.one_b1 * c, new_v = a.root_one_b2 * c;
  Quad<P> p[kQuads];
  double m[kQuads][4], v[kQuads][4], top_m = 0.0, top_v = 0.0, sum_v = 0.0;
#pragma unroll
  for (int q = 0; q < kQuads; ++q) {
    p[q] = l.template load<P>(t.p, q);
    const Quad<G> g = l.template load<G>(t.g, q);
    const Quad<int8_t> qm = l.template load<int8_t>(t.m, q);
    const Quad<uint8_t> qv = l.template load<uint8_t>(t.v, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double x = widen(g.e[i]), old = units(qv.e[i]) * old_v, now = x * new_v;
      m[q][i] = fma(new_m, x, units(qm.e[i]) * old_m);
      v[q][i] = fma(now, now, old * old);
      top_m = fmax(top_m, fabs(m[q][i]));
      top_v = fmax(top_v, v[q][i]);
      sum_v += v[q][i];
    }
  }
  // a maximum leaves a NaN out; a NaN is in v where the gradient or v's scale
  // is one, and in m where the gradient or m's scale is
  if (sum_v != sum_v) top_v = sum_v;
  if (sum_v != sum_v || am != am) top_m = __builtin_nan("");
  const ScaleM sm(row_max(top_m));
  const ScaleV sv(row_max(top_v));
  if (!WHOLE || a.far || __any(sm.tiny || sv.tiny || sv.huge))
    finish8<true, P, COPY>(a, t, l, p, m, v, sm, sv);
  else
    finish8<false, P, COPY>(a, t, l, p, m, v, sm, sv);
  if (exists && threadIdx.x % 16 == 0) {
    *ms = sm.stored;
    *vs = sv.stored;
  }
}

// Three waves a SIMD, though registers allow four: 300M elements in eight
// tensors that begin off the cache lines 842 to 852 us against 882, back to
// back (float32 params, bfloat16 gradients and copies), that begin on them 767
// to 776 either way.
template <class P, class G, bool COPY>
__global__ __launch_bounds__(kBlock) __attribute__((amdgpu_waves_per_eu(3, 3))) void adamw8_step_kernel(AdamwStepArgs a) {
  // from the end, where the norm has just been, and where the last tile's
  // elements one by one would keep the rest waiting (6.5M elements: 25.1 us
  // in order, 22.5 from the end; 300M 803 and 798; as the step was then)
  const AdamwTile tile = reinterpret_cast<const AdamwTile*>(a.plan + a.tiles_at)[gridDim.x - 1 - blockIdx.x];
  const AdamwTensor t = reinterpret_cast<const AdamwTensor*>(a.plan + a.tensors_at)[tile.tensor];
  const float c = a.clip ? reinterpret_cast<const AdamwSums*>(a.plan + a.sums_at)->factor : a.factor;
  const uint64_t begin = wave_begin(tile);
  if (begin >= t.count) return;
  if (whole(begin, t.count, t.vec != 0))
    step8<true, P, G, COPY>(a, t, begin, c);
  else
    step8<false, P, G, COPY>(a, t, begin, c);
}

// --- decoding ---------------------------------------------------------------------------

// One rounding per value: the products are taken in float64 (m's is exact
// there) and rounded to float32.  Memory binds it: 300M codes of m 264 us (5.7
// TB/s), of v 288 us (5.2 TB/s).
template <bool WHOLE, class C>
__device__ __forceinline__ void decode(const C* codes, const float* scales, uint64_t begin, uint64_t count,
                                       float* out) {
  const Lanes<WHOLE> l = runs_of<WHOLE>(begin, count);
  Quad<C> code[kQuads];
  float scale[kQuads];
#pragma unroll
  for (int q = 0; q < kQuads; ++q) {
    code[q] = l.template load<C>(codes, q);
    const uint64_t first = begin + q * l.step;      // of the block that the wave's q-th run is
    scale[q] = scales[(WHOLE || first < count ? first : count - 1) / AR_ADAMW_BLOCK];
  }
#pragma unroll
  for (int q = 0; q < kQuads; ++q) {
    Quad<float> x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double y = units(code[q].e[i]) * static_cast<double>(scale[q]);
      x.e[i] = static_cast<float>(std::is_signed<C>::value ? y : y * y);
    }
    l.template store<float>(out, q, x);
  }
}

template <class C>
__global__ __launch_bounds__(kBlock) void adamw_dequantize_kernel(const C* codes, const float* scales,
                                                                  uint64_t count, int vec, float* out) {
  const AdamwTile tile = {0, blockIdx.x};
  const uint64_t begin = wave_begin(tile);
  if (begin >= count) return;
  if (whole(begin, count, vec != 0))
    decode<true>(codes, scales, begin, count, out);
  else
    decode<false>(codes, scales, begin, count, out);
}

template <class A> hipError_t launch1(void (*kernel)(A), uint64_t blocks, const A& a, hipStream_t stream) {
  A copy = a;
  void* args[] = {&copy};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(static_cast<uint32_t>(blocks)),
                         dim3(kBlock), args, 0, stream);
}

template <class P, class G, bool COPY> auto step_kernel(int bits, bool keep) {
  return bits == 8 ? adamw8_step_kernel<P, G, COPY>
         : keep    ? adamw_step_kernel<P, G, COPY, true>
                   : adamw_step_kernel<P, G, COPY, false>;
}

}  // namespace

hipError_t launch_adamw_norm(const AdamwNormArgs& a, ar_dtype_t grad_dtype, hipStream_t stream) {
  const uint32_t blocks = std::max(1u, std::min(a.tiles, kMaxNormBlocks));
  return launch1(grad_dtype == AR_FLOAT32 ? adamw_norm_kernel<float> : adamw_norm_kernel<uint16_t>,
                 blocks, a, stream);
}

hipError_t launch_adamw_step(const AdamwStepArgs& a, uint32_t tiles, ar_dtype_t param_dtype,
                             ar_dtype_t grad_dtype, int state_bits, bool copy, bool keep, hipStream_t stream) {
  const bool p32 = param_dtype == AR_FLOAT32, g32 = grad_dtype == AR_FLOAT32;
  void (*fn)(AdamwStepArgs);
  if (!p32)
    fn = g32 ? step_kernel<uint16_t, float, false>(state_bits, keep) : step_kernel<uint16_t, uint16_t, false>(state_bits, keep);
  else if (copy)
    fn = g32 ? step_kernel<float, float, true>(state_bits, keep) : step_kernel<float, uint16_t, true>(state_bits, keep);
  else
    fn = g32 ? step_kernel<float, float, false>(state_bits, keep) : step_kernel<float, uint16_t, false>(state_bits, keep);
  return launch1(fn, state_bits == 32 ? tiles * (kAdamwTile / kPiece) : tiles, a, stream);
}

hipError_t launch_adamw_dequantize(const void* codes, const float* scales, uint64_t count,
                                   bool is_signed, float* out, hipStream_t stream) {
  const uint64_t blocks = (count - 1) / kAdamwTile + 1;
  int vec = reinterpret_cast<uintptr_t>(codes) % 4 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
  void* args[] = {&codes, &scales, &count, &vec, &out};
  const void* fn = is_signed ? reinterpret_cast<const void*>(&adamw_dequantize_kernel<int8_t>)
                             : reinterpret_cast<const void*>(&adamw_dequantize_kernel<uint8_t>);
  return hipLaunchKernel(fn, dim3(static_cast<uint32_t>(blocks)), dim3(kBlock), args, 0, stream);
}

}  // namespace ar
