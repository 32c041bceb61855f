// The Muon step (gfx950): momentum, its orthogonalisation by Newton-Schulz
// products, the update.
//
// The products are the work.  Rounding X to 11 bits before them moves the
// result of a matrix with a few strong directions by 4 % (float16; bfloat16: 33
// %), since every step multiplies what the rounding adds in the weak directions
// by up to 3.4.  So X, X X^T and the polynomial are held as the sum of two
// float16 values of 22 bits together, scaled by 2^12 to stay above float16's
// subnormal numbers (|X| < 1.3, the polynomial's values < 3.5), and a product is
// three of matrix instructions, large by large and large by small either way,
// added up in float32.  The result is as exact as with float32 products (1 to 3
// times their error), at 2.9 times their rate.
#include "train/muon.hpp"

#include "train/tile.hpp"
#include "train/wave.hpp"

namespace ar {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScale = 4096.0f, kUnscale = 1.0f / 4096.0f;

typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;

__device__ __forceinline__ const MuonMatrix& matrix_of(const MuonStepArgs& a, uint32_t i) {
  return reinterpret_cast<const MuonMatrix*>(a.plan + a.matrices_at)[i];
}
__device__ __forceinline__ MuonNorm* norm_of(const MuonStepArgs& a, uint32_t i) {
  return reinterpret_cast<MuonNorm*>(a.plan + a.norms_at) + i;
}

template <class T> __device__ __forceinline__ float load(const T* p) { return static_cast<float>(*p); }

// A value times kScale as the sum of two float16.
__device__ __forceinline__ void split(float v, _Float16* large, _Float16* small) {
  *large = static_cast<_Float16>(v);
  *small = static_cast<_Float16>(v - static_cast<float>(*large));
}

// --- momentum and norm --------------------------------------------------------------

constexpr int kElementThreads = 256;

// m' = mu m + s g, and the norm of u = s g + mu m' (nesterov) or m': squares and
// their sums in float64, joined in the chunks' order by a matrix's last block.
template <class G> __global__ __launch_bounds__(kElementThreads) void muon_momentum(MuonStepArgs a) {
  const MuonChunk c = reinterpret_cast<const MuonChunk*>(a.plan + a.chunks_at)[blockIdx.x];
  const MuonMatrix& x = matrix_of(a, c.matrix);
  const uint64_t count = static_cast<uint64_t>(x.rows) * x.cols;
  const uint64_t first = static_cast<uint64_t>(c.index) * kMuonChunk;
  const uint32_t n = static_cast<uint32_t>(min(count - first, static_cast<uint64_t>(kMuonChunk)));
  const G* g = static_cast<const G*>(x.g) + first;
  float* m = x.m + first;
  double sum = 0;
  for (uint32_t i = threadIdx.x; i < n; i += kElementThreads) {
    const float s = a.grad_scale * load(g + i);
    const float next = __builtin_fmaf(a.momentum, m[i], s);
    m[i] = next;
    const double u = a.nesterov ? __builtin_fmaf(a.momentum, next, s) : next;
    sum += u * u;
  }
  sum = block_sum<kElementThreads>(sum);
  double* sums = reinterpret_cast<double*>(a.plan + a.sums_at) + x.first_chunk;
  MuonNorm* norm = norm_of(a, c.matrix);
  if (threadIdx.x == 0) shared_store(sums + c.index, sum);
  if (!last_to_arrive(&norm->arrived, x.chunks)) return;
  double all = 0;
  for (uint32_t i = threadIdx.x; i < x.chunks; i += kElementThreads) all += shared_load(sums + i);
  all = block_sum<kElementThreads>(all);
  if (threadIdx.x == 0) {
    norm->inverse = 1.0 / (sqrt(all) + a.eps);
    norm->arrived = 0;
  }
}

// X = u / (|u| + eps) in two parts, transposed where the matrix is taller than
// wide, zeros around it.  A block has a tile of SIDE x SIDE of X.
template <int SIDE, class G> __global__ __launch_bounds__(kElementThreads) void muon_start(MuonStepArgs a) {
  __shared__ float turned[SIDE][SIDE + 1];
  const MuonTile t = reinterpret_cast<const MuonTile*>(a.plan + a.tiles_at)[blockIdx.x];
  const MuonMatrix& x = matrix_of(a, t.matrix);
  const double scale = norm_of(a, t.matrix)->inverse * kScale;   // float32 would lose the far norms
  const G* g = static_cast<const G*>(x.g);
  const uint32_t m0 = t.m * SIDE, n0 = t.n * SIDE;          // of X
  const uint32_t r0 = x.tall ? n0 : m0, c0 = x.tall ? m0 : n0;
  for (uint32_t i = threadIdx.x; i < SIDE * SIDE; i += kElementThreads) {
    const uint32_t r = r0 + i / SIDE, c = c0 + i % SIDE;
    float v = 0.0f;
    if (r < x.rows && c < x.cols) {
      const uint64_t at = static_cast<uint64_t>(r) * x.cols + c;
      v = x.m[at];
      if (a.nesterov) v = __builtin_fmaf(a.momentum, v, a.grad_scale * load(g + at));
      v = static_cast<float>(v * scale);
    }
    turned[i / SIDE][i % SIDE] = v;
  }
  __syncthreads();
  _Float16* to = reinterpret_cast<_Float16*>(a.workspace + x.x[0]);
  const uint64_t plane = x.x_plane / sizeof(_Float16);
  for (uint32_t i = threadIdx.x * 4; i < SIDE * SIDE; i += kElementThreads * 4) {
    const uint32_t m = i / SIDE, n = i % SIDE;
    f16x4 large, small;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      _Float16 l, s;
      split(x.tall ? turned[n + q][m] : turned[m][n + q], &l, &s);
      large[q] = l;
      small[q] = s;
    }
    const uint64_t at = static_cast<uint64_t>(m0 + m) * x.width + n0 + n;
    *reinterpret_cast<f16x4*>(to + at) = large;
    *reinterpret_cast<f16x4*>(to + plane + at) = small;
  }
}

// --- products -------------------------------------------------------------------------

// The tile of D = A B: A [..][k] with `k` contiguous from row m0 on, B the same
// from its row n0 on (BR false) or [k][..] from its column n0 on.  All are padded
// to whole tiles, so nothing is checked.
template <int SIDE, int WM, int WN, bool BR> struct Product {
  using SA = Staged<SIDE, false>;
  using SB = Staged<SIDE, BR>;
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int kStage = 2 * (SA::kBytes + SB::kBytes);
  static constexpr int kBytes = 2 * kStage;
  static constexpr int kM = SIDE / WM / 16, kN = SIDE / WN / 16;

  f32x4 acc[kM][kN];
  int m, n, lane;              // of the wave's part; of the thread

  __device__ __forceinline__ void run(char* lds, const char* a, uint64_t a_plane, uint32_t a_line, uint32_t m0,
                                      const char* b, uint64_t b_plane, uint32_t b_line, uint32_t n0, uint32_t k) {
    constexpr int kLoadsA = SA::kChunks / kThreads, kLoadsB = SB::kChunks / kThreads;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    lane = tid % kWave;
    m = wave / WN * (SIDE / WM);
    n = wave % WN * (SIDE / WN);
#pragma unroll
    for (auto& row : acc)
#pragma unroll
      for (auto& v : row) v = f32x4{0, 0, 0, 0};
    const Source from_a[2] = {Source(a), Source(a + a_plane)}, from_b[2] = {Source(b), Source(b + b_plane)};
    uint32_t at_a[kLoadsA], at_b[kLoadsB];
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j) {
      const int slot = j * kThreads + tid, l = slot / SA::kPerLine;
      at_a[j] = ((m0 + l) * a_line + SA::place(l, slot % SA::kPerLine) * 8) * 2;
    }
#pragma unroll
    for (int j = 0; j < kLoadsB; ++j) {
      const int slot = j * kThreads + tid, l = slot / SB::kPerLine, c = SB::place(l, slot % SB::kPerLine) * 8;
      at_b[j] = BR ? (l * b_line + n0 + c) * 2 : ((n0 + l) * b_line + c) * 2;
    }
    const uint32_t next_a = kStep * 2, next_b = BR ? kStep * b_line * 2 : kStep * 2;
    const uint32_t base = lds_address(lds) + wave * (kWave * 16);
    const auto issue = [&](uint32_t step) {
      const uint32_t to = base + (step & 1) * kStage;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int j = 0; j < kLoadsA; ++j)
          load_to_lds(from_a[p], at_a[j] + step * next_a,
                      __builtin_amdgcn_readfirstlane(to + p * SA::kBytes + j * kThreads * 16));
#pragma unroll
        for (int j = 0; j < kLoadsB; ++j)
          load_to_lds(from_b[p], at_b[j] + step * next_b,
                      __builtin_amdgcn_readfirstlane(to + 2 * SA::kBytes + p * SB::kBytes + j * kThreads * 16));
      }
    };
    const uint32_t steps = k / kStep;
    issue(0);
    for (uint32_t s = 0; s < steps; ++s) {
      settled();
      __builtin_amdgcn_s_barrier();
      if (s + 1 < steps) issue(s + 1);
      const char* stage = lds + (s & 1) * kStage;
      multiply_step<kM, kN, f16x8, 2, SA, SB>(stage, stage + 2 * SA::kBytes, m, n, lane, acc);
    }
  }
};

template <int SIDE> struct Shape {
  static constexpr int kWavesM = 2, kWavesN = SIDE == 128 ? 4 : 2;
  static constexpr int kThreads = kWavesM * kWavesN * kWave;
  // blocks on a CU by their LDS: 128 KB or 64
  static constexpr int kWavesPerSimd = 2;
};

// Four values of a row in two parts.
__device__ __forceinline__ void store(_Float16* to, uint64_t plane, uint64_t at, f32x4 v, f16x4* large, f16x4* small) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    _Float16 l, s;
    split(v[q], &l, &s);
    (*large)[q] = l;
    (*small)[q] = s;
  }
  *reinterpret_cast<f16x4*>(to + at) = *large;
  *reinterpret_cast<f16x4*>(to + plane + at) = *small;
}

// POLY false: gram = X X^T.  POLY true: poly = a I + b gram + c gram gram.  Both are
// symmetric: tiles above the diagonal are stored a second time, transposed.
template <int SIDE, bool POLY>
__global__ __launch_bounds__(Shape<SIDE>::kThreads, Shape<SIDE>::kWavesPerSimd) void muon_square(MuonStepArgs a) {
  using P = Product<SIDE, Shape<SIDE>::kWavesM, Shape<SIDE>::kWavesN, false>;
  __shared__ __attribute__((aligned(1024))) char lds[P::kBytes];
  const MuonTile t = reinterpret_cast<const MuonTile*>(a.plan + a.squares_at)[blockIdx.x];
  const MuonMatrix& x = matrix_of(a, t.matrix);
  const uint32_t m0 = t.m * SIDE, n0 = t.n * SIDE, side = x.height;
  const char* from = a.workspace + (POLY ? x.gram : x.x[a.from]);
  const uint64_t from_plane = POLY ? x.gram_plane : x.x_plane;
  const uint32_t k = POLY ? x.height : x.width;
  P p;
  p.run(lds, from, from_plane, k, m0, from, from_plane, k, n0, k);

  const uint64_t plane = x.gram_plane / sizeof(_Float16);
  _Float16* to = reinterpret_cast<_Float16*>(a.workspace + (POLY ? x.poly : x.gram));
  const _Float16* gram = reinterpret_cast<const _Float16*>(a.workspace + x.gram);
#pragma unroll
  for (int i = 0; i < P::kM; ++i)
#pragma unroll
    for (int j = 0; j < P::kN; ++j) {
      const uint32_t m = m0 + p.m + 16 * i + p.lane % 16, n = n0 + p.n + 16 * j + 4 * (p.lane / 16);
      const uint64_t at = static_cast<uint64_t>(m) * side + n;
      f32x4 v = p.acc[i][j] * kUnscale;
      if (POLY) {
        const f16x4 gl = *reinterpret_cast<const f16x4*>(gram + at);
        const f16x4 gs = *reinterpret_cast<const f16x4*>(gram + plane + at);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float g = static_cast<float>(gl[q]) + static_cast<float>(gs[q]);
          v[q] = __builtin_fmaf(kC, v[q], kB * g) + (m == n + q ? kA * kScale : 0.0f);
        }
      }
      f16x4 large, small;
      store(to, plane, at, v, &large, &small);
      if (t.m != t.n) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint64_t mirror = static_cast<uint64_t>(n + q) * side + m;
          to[mirror] = large[q];
          to[plane + mirror] = small[q];
        }
      }
    }
}

// p' = (1 - lr wd) p - lr s x
template <class T, bool COPY>
__device__ __forceinline__ void update(const MuonMatrix& x, uint64_t at, float lr, float lr_wd, float v) {
  T* p = static_cast<T*>(x.p) + at;
  const float old = static_cast<float>(*p);
  const float next = old - __builtin_fmaf(lr, v, lr_wd * old);
  *p = static_cast<T>(next);
  if (COPY) static_cast<__bf16*>(x.copy)[at] = static_cast<__bf16>(next);
}

// X' = poly X; the last one updates the parameters instead.
template <int SIDE, class T, bool COPY>
__global__ __launch_bounds__(Shape<SIDE>::kThreads, Shape<SIDE>::kWavesPerSimd) void muon_apply(MuonStepArgs a) {
  using P = Product<SIDE, Shape<SIDE>::kWavesM, Shape<SIDE>::kWavesN, true>;
  __shared__ __attribute__((aligned(1024))) char lds[P::kBytes];
  const MuonTile t = reinterpret_cast<const MuonTile*>(a.plan + a.tiles_at)[blockIdx.x];
  const MuonMatrix& x = matrix_of(a, t.matrix);
  const uint32_t m0 = t.m * SIDE, n0 = t.n * SIDE;
  P p;
  p.run(lds, a.workspace + x.poly, x.gram_plane, x.height, m0, a.workspace + x.x[a.from], x.x_plane, x.width, n0,
        x.height);

  const float lr = a.lr * (a.rms != 0.0f ? a.rms * x.by_size : x.by_shape) * (kUnscale * kUnscale);
  _Float16* to = reinterpret_cast<_Float16*>(a.workspace + x.x[1 - a.from]);
#pragma unroll
  for (int i = 0; i < P::kM; ++i)
#pragma unroll
    for (int j = 0; j < P::kN; ++j) {
      const uint32_t m = m0 + p.m + 16 * i + p.lane % 16, n = n0 + p.n + 16 * j + 4 * (p.lane / 16);
      if (!a.last) {
        f16x4 large, small;
        store(to, x.x_plane / sizeof(_Float16), static_cast<uint64_t>(m) * x.width + n, p.acc[i][j] * kUnscale, &large,
              &small);
        continue;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t r = x.tall ? n + q : m, c = x.tall ? m : n + q;
        if (r < x.rows && c < x.cols)
          update<T, COPY>(x, static_cast<uint64_t>(r) * x.cols + c, lr, a.lr_wd, p.acc[i][j][q]);
      }
    }
}

}  // namespace

hipError_t launch_muon_momentum(const MuonStepArgs& a, uint32_t chunks, ar_dtype_t grad_dtype, hipStream_t stream) {
  (grad_dtype == AR_FLOAT32 ? muon_momentum<float> : muon_momentum<__bf16>)<<<chunks, kElementThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <int SIDE>
static hipError_t start(const MuonStepArgs& a, uint32_t tiles, ar_dtype_t grad_dtype, hipStream_t stream) {
  (grad_dtype == AR_FLOAT32 ? muon_start<SIDE, float> : muon_start<SIDE, __bf16>)<<<tiles, kElementThreads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_muon_start(const MuonStepArgs& a, uint32_t tiles, uint32_t side, ar_dtype_t grad_dtype,
                             hipStream_t stream) {
  return (side == 128 ? start<128> : start<64>)(a, tiles, grad_dtype, stream);
}

hipError_t launch_muon_gram(const MuonStepArgs& a, uint32_t squares, uint32_t side, hipStream_t stream) {
  if (side == 128)
    muon_square<128, false><<<squares, Shape<128>::kThreads, 0, stream>>>(a);
  else
    muon_square<64, false><<<squares, Shape<64>::kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_muon_poly(const MuonStepArgs& a, uint32_t squares, uint32_t side, hipStream_t stream) {
  if (side == 128)
    muon_square<128, true><<<squares, Shape<128>::kThreads, 0, stream>>>(a);
  else
    muon_square<64, true><<<squares, Shape<64>::kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <int SIDE>
static hipError_t apply(const MuonStepArgs& a, uint32_t tiles, ar_dtype_t param_dtype, bool copy, hipStream_t stream) {
  const auto kernel = param_dtype == AR_BFLOAT16 ? muon_apply<SIDE, __bf16, false>
                      : copy                     ? muon_apply<SIDE, float, true>
                                                 : muon_apply<SIDE, float, false>;
  kernel<<<tiles, Shape<SIDE>::kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_muon_apply(const MuonStepArgs& a, uint32_t tiles, uint32_t side, ar_dtype_t param_dtype, bool copy,
                             hipStream_t stream) {
  return (side == 128 ? apply<128> : apply<64>)(a, tiles, param_dtype, copy, stream);
}

}  // namespace ar
