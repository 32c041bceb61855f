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

__device__ __forceinline__ const MuonMatrix& matrix_of(const MuonStepArgs& a, uint32_t i) {
  return reinterpret_cast<const MuonMatrix*>(a.plan + a.matrices_at)[i];
}
__device__ __forceinline__ MuonNorm* norm_of(const MuonStepArgs& a, uint32_t i) {
  return reinterpret_cast<MuonNorm*>(a.plan + a.norms_at) + i;
}

typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;

// A value times kScale as the sum of two float16.
__device__ __forceinline__ void split(float v, _Float16* large, _Float16* small) {
  *large = static_cast<_Float16>(v);
  *small = static_cast<_Float16>(v - static_cast<float>(*large));
}

// --- momentum and norm --------------------------------------------------------------

// 1 / (|u| + eps), given |u|^2; a matrix of zeros has X = 0 without an eps too.
__device__ __forceinline__ double inverse(double square, double eps) {
  const double norm = sqrt(square) + eps;
  return norm == 0 ? 0 : 1.0 / norm;
}

constexpr int kElementThreads = 256;

// N elements from p on; `vec`: p allows them at once.
template <int N, class T> __device__ __forceinline__ void read(const T* p, bool vec, int n, float (&v)[N]) {
  typedef __attribute__((ext_vector_type(4))) T Four;
  if (vec && n >= N) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const Four f = *reinterpret_cast<const Four*>(p + i);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[i + q] = static_cast<float>(f[q]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? static_cast<float>(p[i]) : 0.0f;
  }
}

// m' = mu m + s g, and the norm of u = s g + mu m' (nesterov) or m': squares and
// their sums in float64, joined in the chunks' order by a matrix's last block.  A
// thread has four times eight elements.  67 million bfloat16 gradients 129 us, 5.2
// TB/s.
template <class G> __global__ __launch_bounds__(kElementThreads) void muon_momentum(MuonStepArgs a) {
  constexpr int kEach = 8;
  const MuonChunk c = reinterpret_cast<const MuonChunk*>(a.plan + a.chunks_at)[blockIdx.x];
  const MuonMatrix& x = matrix_of(a, c.matrix);
  const uint64_t count = static_cast<uint64_t>(x.rows) * x.cols;
  const uint64_t first = static_cast<uint64_t>(c.index) * kMuonChunk;
  const int n = static_cast<int>(min(count - first, static_cast<uint64_t>(kMuonChunk)));
  const G* g = static_cast<const G*>(x.g) + first;
  float* m = x.m + first;
  const bool flat = x.flat != 0;
  double sum = 0;
#pragma unroll
  for (int r = 0; r < static_cast<int>(kMuonChunk); r += kElementThreads * kEach) {
    const int i = r + threadIdx.x * kEach;
    if (i >= n) break;
    float s[kEach], v[kEach];
    read(g + i, flat, n - i, s);
    read(m + i, flat, n - i, v);
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      s[q] *= a.grad_scale;
      v[q] = __builtin_fmaf(a.momentum, v[q], s[q]);
      const double u = a.nesterov ? __builtin_fmaf(a.momentum, v[q], s[q]) : v[q];
      sum += u * u;
    }
    if (flat && i + kEach <= n) {
#pragma unroll
      for (int q = 0; q < kEach; q += 4) *reinterpret_cast<f32x4*>(m + i + q) = f32x4{v[q], v[q + 1], v[q + 2], v[q + 3]};
    } else {
#pragma unroll
      for (int q = 0; q < kEach; ++q)
        if (i + q < n) m[i + q] = v[q];
    }
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
    norm->inverse = inverse(all, a.eps);
    norm->arrived = 0;
  }
}

// Values of a row, times kScale, in two parts; `at` is a multiple of 8.
template <int N> __device__ __forceinline__ void store(_Float16* to, uint64_t plane, uint64_t at, const float (&v)[N]) {
#pragma unroll
  for (int h = 0; h < N; h += 8) {
    f16x8 large, small;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      _Float16 l, s;
      split(v[h + q], &l, &s);
      large[q] = l;
      small[q] = s;
    }
    *reinterpret_cast<f16x8*>(to + at + h) = large;
    *reinterpret_cast<f16x8*>(to + plane + at + h) = small;
  }
}

// X = u / (|u| + eps) in two parts, transposed where the matrix is taller than
// wide, zeros around it.  A block has 64 x 64 of X, a thread 16 of a row.  The same
// matrices 153 us, 4.4 TB/s.
template <int SIDE, class G> __global__ __launch_bounds__(kElementThreads) void muon_start(MuonStepArgs a) {
  constexpr uint32_t kPart = 64, kParts = SIDE / kPart;
  __shared__ float turned[kPart][kPart + 1];
  const MuonTile t = reinterpret_cast<const MuonTile*>(a.plan + a.tiles_at)[blockIdx.x];
  if (t.matrix == kMuonNoMatrix || t.part != 0) return;
  const MuonMatrix& x = matrix_of(a, t.matrix);
  const double scale = norm_of(a, t.matrix)->inverse * kScale;   // float32 would lose the far norms
  const uint32_t m0 = t.m * SIDE + blockIdx.y / kParts * kPart, n0 = t.n * SIDE + blockIdx.y % kParts * kPart;   // of X
  const uint32_t line = threadIdx.x / 4, piece = threadIdx.x % 4 * 16;
  const uint32_t r = (x.tall ? n0 : m0) + line, c = (x.tall ? m0 : n0) + piece;
  float v[16] = {};
  if (r < x.rows && c < x.cols) {
    const uint64_t at = static_cast<uint64_t>(r) * x.cols + c;
    const int n = static_cast<int>(min(x.cols - c, 16u));
    const bool vec = x.flat != 0 && x.cols % 4 == 0;
    read(x.m + at, vec, n, v);
    if (a.nesterov) {
      float s[16];
      read(static_cast<const G*>(x.g) + at, vec, n, s);
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = __builtin_fmaf(a.momentum, v[q], a.grad_scale * s[q]);
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) v[q] = static_cast<float>(v[q] * scale);
  }
  if (x.tall) {
#pragma unroll
    for (int q = 0; q < 16; ++q) turned[line][piece + q] = v[q];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 16; ++q) v[q] = turned[piece + q][line];
  }
  store(reinterpret_cast<_Float16*>(a.workspace + x.x[0]), x.x_plane / sizeof(_Float16),
        static_cast<uint64_t>(m0 + line) * x.width + n0 + piece, v);
}

// --- products -------------------------------------------------------------------------

// The tile of D = A B: A [..][k] with `k` contiguous from row m0 on, B the same
// from its row n0 on (BR false) or [k][..] from its column n0 on.  All are padded
// to whole tiles, so nothing is checked.
template <int SIDE> constexpr int kProductThreads = SIDE == 128 ? 512 : 256;
template <int SIDE> constexpr int kPerSimd = SIDE == 128 ? 4 : 2;

// Two blocks of 128 x 128 with steps of 32 on a CU: 1,390 TFLOP/s of matrix
// instructions for 131,072 x 1,024 by k = 2,048, against 1,213 of one block with
// steps of 64, and 1,299-1,324 of 256 x 128 and 128 x 256.  Eight waves a block:
// with four, steps of matrices of 512 to 1,024 rows take 3 to 8 % longer, those of
// 4,096 rows 1 % less.  64 x 64 is for few tiles, one or two on a CU: three steps
// under way (one of 1,024 x 1,024 220 us, 289 with one).
template <int SIDE, bool BR> struct Product {
  static constexpr int kStep = kMuonStep;
  using SA = Staged<SIDE, false, kStep, false>;
  using SB = Staged<SIDE, BR, kStep, true>;
  static constexpr int kWavesM = 4, kWavesN = SIDE / 64;
  static constexpr int kThreads = kWavesM * kWavesN * kWave;
  static_assert(kThreads == kProductThreads<SIDE>);
  static constexpr int kStage = 2 * (SA::kBytes + SB::kBytes);
  static constexpr int kStages = SIDE == 128 ? 2 : 4, kAhead = kStages - 1;
  static constexpr int kBytes = kStages * kStage;
  static constexpr int kM = SIDE / kWavesM / 16, kN = SIDE / kWavesN / 16;

  f32x4 acc[kM][kN];
  int m, n, lane;              // of the wave's part; of the thread

  __device__ __forceinline__ void run(char* lds, const char* a, uint64_t a_plane, uint32_t a_line, uint32_t m0,
                                      const char* b, uint64_t b_plane, uint32_t b_line, uint32_t n0,
                                      uint32_t first, uint32_t steps) {
    constexpr int kLoadsA = SA::kChunks / kThreads, kLoadsB = SB::kChunks / kThreads;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    lane = tid % kWave;
    m = wave / kWavesN * (SIDE / kWavesM);
    n = wave % kWavesN * (SIDE / kWavesN);
    clear(acc);
    const Source from_a[2] = {Source(a), Source(a + a_plane)}, from_b[2] = {Source(b), Source(b + b_plane)};
    uint32_t at_a[kLoadsA], at_b[kLoadsB];
#pragma unroll
    for (int j = 0; j < kLoadsA; ++j) {
      const int slot = j * kThreads + tid, l = slot / SA::kPerLine;
      at_a[j] = ((m0 + l) * a_line + SA::place(l, slot % SA::kPerLine) * 8) * 2 + first * kStep * 2;
    }
#pragma unroll
    for (int j = 0; j < kLoadsB; ++j) {
      const int slot = j * kThreads + tid, l = slot / SB::kPerLine, c = SB::place(l, slot % SB::kPerLine) * 8;
      at_b[j] = BR ? ((first * kStep + l) * b_line + n0 + c) * 2 : ((n0 + l) * b_line + first * kStep + c) * 2;
    }
    const uint32_t next_a = kStep * 2, next_b = BR ? kStep * b_line * 2 : kStep * 2;
    const uint32_t base = lds_address(lds) + wave * (kWave * 16);
    // (past the last step nothing is read, but as many loads are counted)
    const auto issue = [&](uint32_t step) {
      const uint32_t to = base + step % kStages * kStage;
      const bool more = step < steps;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int j = 0; j < kLoadsA; ++j)
          load_to_lds(from_a[p], more ? at_a[j] + step * next_a : kNowhere,
                      __builtin_amdgcn_readfirstlane(to + p * SA::kBytes + j * kThreads * 16));
#pragma unroll
        for (int j = 0; j < kLoadsB; ++j)
          load_to_lds(from_b[p], more ? at_b[j] + step * next_b : kNowhere,
                      __builtin_amdgcn_readfirstlane(to + 2 * SA::kBytes + p * SB::kBytes + j * kThreads * 16));
      }
    };
#pragma unroll
    for (uint32_t s = 0; s < kAhead; ++s) issue(s);
    for (uint32_t s = 0; s < steps; ++s) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kAhead - 1) * 2 * (kLoadsA + kLoadsB)) : "memory");
      __builtin_amdgcn_s_barrier();
      issue(s + kAhead);
      const char* stage = lds + s % kStages * kStage;
      multiply_step<kM, kN, f16x8, 2, kStep, SA, SB>(stage, stage + 2 * SA::kBytes, m, n, lane, acc);
    }
    settled();
  }

  // Joins the parts of a tile; true in the block that has the whole.  The sums
  // pass through memory as wave.hpp says, eight bytes at a time.
  __device__ __forceinline__ bool join(const MuonStepArgs& a, const MuonTile& t) {
    if (t.parts == 1) return true;
    constexpr uint32_t kPairs = SIDE * SIDE / 2;
    uint64_t* parts = reinterpret_cast<uint64_t*>(a.workspace + a.parts_at) + static_cast<uint64_t>(t.slot) * kPairs;
    union Pair {
      uint64_t word;
      float v[2];
    };
    uint64_t* mine = parts + t.part * kPairs + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < kN; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          Pair p;
          p.v[0] = acc[i][j][2 * h];
          p.v[1] = acc[i][j][2 * h + 1];
          shared_store(mine + ((i * kN + j) * 2 + h) * kThreads, p.word);
        }
    uint32_t* arrived = reinterpret_cast<uint32_t*>(a.plan + a.arrived_at) + t.counter;
    if (!last_to_arrive(arrived, t.parts)) return false;
    if (threadIdx.x == 0) *arrived = 0;
    clear(acc);
    for (uint32_t part = 0; part < t.parts; ++part) {
      const uint64_t* from = parts + part * kPairs + threadIdx.x;
      Pair p[kM][kN][2];
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) p[i][j][h].word = shared_load(from + ((i * kN + j) * 2 + h) * kThreads);
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] += p[i][j][q / 2].v[q % 2];
    }
    return true;
  }

  // The tile in LDS, so that neighbouring lanes can take neighbouring values of a
  // row: a row m of it, or TURNED a column n, has SIDE float32 in pieces of four
  // that are permuted by the row, against bank conflicts of the writes.
  template <bool TURNED> static __device__ __forceinline__ int place(int r, int c) {
    return r * SIDE + (c ^ (TURNED ? r / 16 % 4 * 16 : r % 16 * 4));
  }
  template <bool TURNED> __device__ __forceinline__ void put(float* tile) const {
    static_assert(SIDE * SIDE * sizeof(float) <= kBytes);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int r = m + 16 * i + lane % 16, c = n + column(j, lane / 16);
        if (TURNED) {
#pragma unroll
          for (int q = 0; q < 4; ++q) tile[place<true>(c + q, r)] = acc[i][j][q];
        } else {
          *reinterpret_cast<f32x4*>(tile + place<false>(r, c)) = acc[i][j];
        }
      }
    __syncthreads();
  }
  // Calls f(row, first column, values) for N of a row at a time.
  template <bool TURNED, int N, class F> static __device__ __forceinline__ void rows(const float* tile, F&& f) {
#pragma unroll 2
    for (int i = threadIdx.x * N; i < SIDE * SIDE; i += kThreads * N) {
      const int r = i / SIDE, c = i % SIDE;
      float v[N];
#pragma unroll
      for (int h = 0; h < N; h += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(tile + place<TURNED>(r, c + h));
#pragma unroll
        for (int q = 0; q < 4; ++q) v[h + q] = x[q];
      }
      f(r, c, v);
    }
  }
};

// The values of a tile of X X^T, or of the polynomial, from row m0 and column n0 on.
template <class P, bool POLY, bool TURNED>
__device__ __forceinline__ void store_square(const MuonStepArgs& a, const MuonMatrix& x, const float* tile, uint32_t m0,
                                             uint32_t n0) {
  const uint64_t plane = x.gram_plane / sizeof(_Float16);
  _Float16* to = reinterpret_cast<_Float16*>(a.workspace + (POLY ? x.poly : x.gram));
  const _Float16* gram = reinterpret_cast<const _Float16*>(a.workspace + x.gram);
  P::template rows<TURNED, 8>(tile, [&](uint32_t r, uint32_t c, float (&v)[8]) {
    const uint64_t at = static_cast<uint64_t>(m0 + r) * x.height + n0 + c;
    f16x8 gl, gs;
    if (POLY) {
      gl = *reinterpret_cast<const f16x8*>(gram + at);
      gs = *reinterpret_cast<const f16x8*>(gram + plane + at);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      v[q] *= kUnscale;
      if (POLY) {
        const float g = static_cast<float>(gl[q]) + static_cast<float>(gs[q]);
        v[q] = __builtin_fmaf(kC, v[q], kB * g) + (m0 + r == n0 + c + q ? kA * kScale : 0.0f);
      }
    }
    store(to, plane, at, v);
  });
}

// POLY false: gram = X X^T.  POLY true: poly = a I + b gram + c gram gram.  Both are
// symmetric: tiles above the diagonal are stored a second time, transposed.  Three
// of 4,096 rows, half of them by k = 8,192: 818 and 649 us, at 1,040 and 980 TFLOP/s
// of 16 bits.
template <int SIDE, bool POLY>
__global__ __launch_bounds__(kProductThreads<SIDE>, kPerSimd<SIDE>) void muon_square(MuonStepArgs a) {
  using P = Product<SIDE, false>;
  __shared__ __attribute__((aligned(1024))) char lds[P::kBytes];
  const MuonTile t = reinterpret_cast<const MuonTile*>(a.plan + (POLY ? a.polys_at : a.squares_at))[blockIdx.x];
  if (t.matrix == kMuonNoMatrix) return;
  const MuonMatrix& x = matrix_of(a, t.matrix);
  const uint32_t m0 = t.m * SIDE, n0 = t.n * SIDE;
  const char* from = a.workspace + (POLY ? x.gram : x.x[a.from]);
  const uint64_t from_plane = POLY ? x.gram_plane : x.x_plane;
  const uint32_t line = POLY ? x.height : x.width;
  P p;
  p.run(lds, from, from_plane, line, m0, from, from_plane, line, n0, t.first, t.steps);
  if (!p.join(a, t)) return;
  float* tile = reinterpret_cast<float*>(lds);
  p.template put<false>(tile);
  store_square<P, POLY, false>(a, x, tile, m0, n0);
  if (t.m == t.n) return;
  p.template put<true>(tile);
  store_square<P, POLY, true>(a, x, tile, n0, m0);
}

// p' = (1 - lr wd) p - lr s x for N consecutive elements
template <int N, class T, bool COPY>
__device__ __forceinline__ void update(const MuonMatrix& x, uint64_t at, float lr, float lr_wd, const float* v) {
  typedef __attribute__((ext_vector_type(N))) T Values;
  typedef __attribute__((ext_vector_type(N))) __bf16 Copies;
  Values* p = reinterpret_cast<Values*>(static_cast<T*>(x.p) + at);
  Values old = *p;
  Copies copy;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const float o = static_cast<float>(old[q]), next = o - __builtin_fmaf(lr, v[q], lr_wd * o);
    old[q] = static_cast<T>(next);
    copy[q] = static_cast<__bf16>(next);
  }
  *p = old;
  if (COPY) *reinterpret_cast<Copies*>(static_cast<__bf16*>(x.copy) + at) = copy;
}

template <class P, class T, bool COPY, bool TURNED>
__device__ __forceinline__ void update_tile(const MuonStepArgs& a, const MuonMatrix& x, const float* tile, uint32_t r0,
                                            uint32_t c0) {
  const float lr = a.lr * (a.rms != 0.0f ? a.rms * x.by_size : x.by_shape) * (kUnscale * kUnscale);
  P::template rows<TURNED, 4>(tile, [&](uint32_t r, uint32_t c, float (&v)[4]) {
    if (r0 + r >= x.rows || c0 + c >= x.cols) return;
    const uint64_t at = static_cast<uint64_t>(r0 + r) * x.cols + c0 + c;
    if (x.vec) {
      update<4, T, COPY>(x, at, lr, a.lr_wd, v);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c0 + c + q < x.cols) update<1, T, COPY>(x, at + q, lr, a.lr_wd, v + q);
    }
  });
}

// X' = poly X; the last one updates the parameters instead.  The same matrices: 1,395
// us, 1,180 TFLOP/s of 16 bits (a library's product of 8192^3 reaches 1,120).
template <int SIDE, class T, bool COPY>
__global__ __launch_bounds__(kProductThreads<SIDE>, kPerSimd<SIDE>) void muon_apply(MuonStepArgs a) {
  using P = Product<SIDE, true>;
  __shared__ __attribute__((aligned(1024))) char lds[P::kBytes];
  const MuonTile t = reinterpret_cast<const MuonTile*>(a.plan + a.tiles_at)[blockIdx.x];
  if (t.matrix == kMuonNoMatrix) return;
  const MuonMatrix& x = matrix_of(a, t.matrix);
  const uint32_t m0 = t.m * SIDE, n0 = t.n * SIDE;
  P p;
  p.run(lds, a.workspace + x.poly, x.gram_plane, x.height, m0, a.workspace + x.x[a.from], x.x_plane, x.width, n0,
        t.first, t.steps);
  if (!p.join(a, t)) return;
  float* tile = reinterpret_cast<float*>(lds);
  if (a.last && x.tall) {
    p.template put<true>(tile);
    update_tile<P, T, COPY, true>(a, x, tile, n0, m0);
    return;
  }
  p.template put<false>(tile);
  if (a.last) {
    update_tile<P, T, COPY, false>(a, x, tile, m0, n0);
    return;
  }
  _Float16* to = reinterpret_cast<_Float16*>(a.workspace + x.x[1 - a.from]);
  P::template rows<false, 8>(tile, [&](uint32_t r, uint32_t c, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] *= kUnscale;
    store(to, x.x_plane / sizeof(_Float16), static_cast<uint64_t>(m0 + r) * x.width + n0 + c, v);
  });
}

// --- small matrices -----------------------------------------------------------------

// A whole step of a matrix of up to MOST x SHORT in one block, X and X X^T in LDS:
// fifteen products whose launches would take longer than they do.
//
// Both are [line][k] in 16-byte chunks, permuted by the line; a product reads X's
// lines along k, or across it by transposing loads.  What binds is the reading of
// LDS, whose wait only other waves fill: matrices with a short side of up to 64
// are shared out in parts of 16 x 32, so that every SIMD has some (64 x 64 22 us in
// parts of 32 x 32, 18 so; 100 x 61 25 and 24); reading a step ahead leaves no
// registers (28 % more time).
template <int MOST, int SHORT> struct Whole {
  static constexpr int TM = SHORT == 128 ? 2 : 1, kRows = 16 * TM;      // a wave has kRows x 32 of a result
  static constexpr int kThreads = SHORT / kRows * (MOST / 32) * kWave;
  typedef f32x4 Sums[TM][2];

  // Eight lines' chunks of one k meet all banks, and so do two neighbouring chunks
  // of the lines that a transposing load reads: four whose pitch is that of the
  // banks, or two of half that (100 x 61: 25.0 us with the permutation of 64, 23.5
  // so; 64 x 64: 19.6 us with that of 128, 17.9 so).
  static __device__ __forceinline__ int place(int line, int k) {
    const int by = MOST == 128 ? (line & 3) * 2 | (line >> 2 & 1) : line & 7;
    return line * MOST + ((k / 8 ^ by) * 8 | k % 8);
  }

  // 8 k of row r0 + lane % 16, from lines or across them
  template <bool ACROSS> static __device__ __forceinline__ f16x8 fragment(const _Float16* x, int r0, int k0, int lane) {
    const int l = lane % 16;
    if (!ACROSS) return *reinterpret_cast<const f16x8*>(x + place(r0 + l, k0 + 8 * (lane / 16)));
    union {
      f16x8 v;
      s16x4 part[2];
    } u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const _Float16* at = x + place(k0 + 8 * (lane / 16) + 4 * i + l / 4, r0 + l % 4 * 4);
      u.part[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at));
    }
    return u.v;
  }

  // The wave's part of a result of rows x columns.
  struct Part {
    bool any;
    int m, n;
    __device__ __forceinline__ Part(int rows, int columns) {
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), wide = columns / 32;
      m = wave / wide * kRows;
      n = wave % wide * 32;
      any = m < rows;
    }
  };

  // This part of A B^T (or A B where ACROSS), k in steps of 32.
  template <bool ACROSS>
  static __device__ __forceinline__ void product(const _Float16* a, const _Float16* b, const Part& part, int k,
                                                 Sums& acc) {
    const int lane = threadIdx.x % kWave;
    clear(acc);
    if (!part.any) return;
    for (int k0 = 0; k0 < k; k0 += 32) {
      f16x8 fa[2][TM], fb[2][2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[p][i] = fragment<false>(a + p * (MOST * MOST), part.m + 16 * i, k0, lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) fb[p][j] = fragment<ACROSS>(b + p * (MOST * MOST), part.n + 16 * j, k0, lane);
      }
      // large by large, and large by small either way
#pragma unroll
      for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = multiply(fb[t == 0][j], fa[t == 1][i], acc[i][j]);
    }
  }

  // Calls f(row, first column, values) for what product() left in the thread.
  template <class F>
  static __device__ __forceinline__ void each(const Part& part, const Sums& acc, F&& f) {
    const int lane = threadIdx.x % kWave;
    if (!part.any) return;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) f(part.m + 16 * i + lane % 16, part.n + 16 * j + 4 * (lane / 16), acc[i][j]);
  }

  static __device__ __forceinline__ void keep(_Float16* to, int r, int c, float v) {
    split(v, to + place(r, c), to + MOST * MOST + place(r, c));
  }
  // Four of a row from a fourth column on.
  static __device__ __forceinline__ void keep(_Float16* to, int r, int c, f32x4 v) {
    f16x4 large, small;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      _Float16 l, s;
      split(v[q], &l, &s);
      large[q] = l;
      small[q] = s;
    }
    *reinterpret_cast<f16x4*>(to + place(r, c)) = large;
    *reinterpret_cast<f16x4*>(to + MOST * MOST + place(r, c)) = small;
  }
};

template <int MOST, int SHORT, class T, class G, bool COPY>
__global__ __launch_bounds__((Whole<MOST, SHORT>::kThreads), 4) void muon_whole(MuonStepArgs a) {
  using W = Whole<MOST, SHORT>;
  __shared__ __attribute__((aligned(16))) _Float16 held[4 * MOST * MOST];
  _Float16 *x = held, *gram = held + 2 * MOST * MOST;
  const MuonMatrix& matrix = matrix_of(a, blockIdx.x);
  const int rows = matrix.rows, cols = matrix.cols, tall = matrix.tall, count = rows * cols;
  const int height = (min(rows, cols) + 31) / 32 * 32, width = (max(rows, cols) + 31) / 32 * 32;
  const G* g = static_cast<const G*>(matrix.g);

  // Momentum and norm, as muon_momentum.  A thread's elements are read at once
  // and stay in registers until X is made of them.
  constexpr int kEach = MOST * MOST / W::kThreads;
  float u[kEach];
  {
    float s[kEach], m[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + e * W::kThreads;
      s[e] = i < count ? static_cast<float>(g[i]) : 0.0f;
      m[e] = i < count ? matrix.m[i] : 0.0f;
    }
    for (int i = threadIdx.x; i < 4 * MOST * MOST / 8; i += W::kThreads)
      *reinterpret_cast<f16x8*>(held + 8 * i) = f16x8{0, 0, 0, 0, 0, 0, 0, 0};      // around X
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + e * W::kThreads;
      s[e] *= a.grad_scale;
      m[e] = __builtin_fmaf(a.momentum, m[e], s[e]);
      u[e] = a.nesterov ? __builtin_fmaf(a.momentum, m[e], s[e]) : m[e];
      if (i < count) matrix.m[i] = m[e];
    }
  }
  double sum = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) sum += static_cast<double>(u[e]) * u[e];
  const double scale = inverse(block_sum<W::kThreads>(sum), a.eps) * kScale;
  int r = threadIdx.x / cols, c = threadIdx.x % cols;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    if (r < rows) W::keep(x, tall ? c : r, tall ? r : c, static_cast<float>(u[e] * scale));
    r += W::kThreads / cols;
    c += W::kThreads % cols;
    if (c >= cols) {
      c -= cols;
      ++r;
    }
  }
  __syncthreads();

  const typename W::Part square(height, height), wide(height, width);
  typename W::Sums acc;
  const float lr = a.lr * (a.rms != 0.0f ? a.rms * matrix.by_size : matrix.by_shape) * (kUnscale * kUnscale);
  for (int step = 0; step < a.steps; ++step) {
    W::template product<false>(x, x, square, width, acc);
    W::each(square, acc, [&](int r, int c, f32x4 v) { W::keep(gram, r, c, v * kUnscale); });
    __syncthreads();
    W::template product<false>(gram, gram, square, height, acc);
    __syncthreads();
    // the polynomial in the place of X X^T
    W::each(square, acc, [&](int r, int c, f32x4 v) {
      const f16x4 large = *reinterpret_cast<const f16x4*>(gram + W::place(r, c));
      const f16x4 small = *reinterpret_cast<const f16x4*>(gram + MOST * MOST + W::place(r, c));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float old = static_cast<float>(large[q]) + static_cast<float>(small[q]);
        v[q] = __builtin_fmaf(kC, v[q] * kUnscale, kB * old) + (r == c + q ? kA * kScale : 0.0f);
      }
      W::keep(gram, r, c, v);
    });
    __syncthreads();
    W::template product<true>(gram, x, wide, height, acc);
    if (step + 1 == a.steps) break;
    __syncthreads();
    W::each(wide, acc, [&](int r, int c, f32x4 v) { W::keep(x, r, c, v * kUnscale); });
    __syncthreads();
  }
  if (!wide.any) return;
  // p' = (1 - lr wd) p - lr s x; all of a thread's are read at once
  T* p = static_cast<T*>(matrix.p);
  float old[W::TM][2][4];
  int at[W::TM][2][4];
#pragma unroll
  for (int i = 0; i < W::TM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int lane = threadIdx.x % kWave, m = wide.m + 16 * i + lane % 16, n = wide.n + 16 * j + 4 * (lane / 16) + q;
        const int row = tall ? n : m, col = tall ? m : n;
        at[i][j][q] = row < rows && col < cols ? row * cols + col : -1;
        old[i][j][q] = at[i][j][q] >= 0 ? static_cast<float>(p[at[i][j][q]]) : 0.0f;
      }
#pragma unroll
  for (int i = 0; i < W::TM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (at[i][j][q] < 0) continue;
        const float o = old[i][j][q], next = o - __builtin_fmaf(lr, acc[i][j][q], a.lr_wd * o);
        p[at[i][j][q]] = static_cast<T>(next);
        if (COPY) static_cast<__bf16*>(matrix.copy)[at[i][j][q]] = static_cast<__bf16>(next);
      }
}

}  // namespace

template <int MOST, int SHORT, class G>
static hipError_t whole(const MuonStepArgs& a, uint32_t matrices, ar_dtype_t param_dtype, bool copy, hipStream_t stream) {
  const auto kernel = param_dtype == AR_BFLOAT16 ? muon_whole<MOST, SHORT, __bf16, G, false>
                      : copy                     ? muon_whole<MOST, SHORT, float, G, true>
                                                 : muon_whole<MOST, SHORT, float, G, false>;
  kernel<<<matrices, Whole<MOST, SHORT>::kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <class G>
static hipError_t whole(const MuonStepArgs& a, uint32_t matrices, uint32_t longest, uint32_t shortest, ar_dtype_t param_dtype, bool copy,
                        hipStream_t stream) {
  return (longest <= 64    ? whole<64, 64, G>
          : shortest <= 64 ? whole<128, 64, G>
                           : whole<128, 128, G>)(a, matrices, param_dtype, copy, stream);
}

hipError_t launch_muon_whole(const MuonStepArgs& a, uint32_t matrices, uint32_t longest, uint32_t shortest,
                             ar_dtype_t param_dtype, ar_dtype_t grad_dtype, bool copy, hipStream_t stream) {
  return (grad_dtype == AR_FLOAT32 ? whole<float> : whole<__bf16>)(a, matrices, longest, shortest, param_dtype, copy, stream);
}

hipError_t launch_muon_momentum(const MuonStepArgs& a, uint32_t chunks, ar_dtype_t grad_dtype, hipStream_t stream) {
  (grad_dtype == AR_FLOAT32 ? muon_momentum<float> : muon_momentum<__bf16>)<<<chunks, kElementThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <int SIDE>
static hipError_t start(const MuonStepArgs& a, uint32_t tiles, ar_dtype_t grad_dtype, hipStream_t stream) {
  (grad_dtype == AR_FLOAT32 ? muon_start<SIDE, float> : muon_start<SIDE, __bf16>)<<<dim3(tiles, (SIDE / 64) * (SIDE / 64)), kElementThreads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_muon_start(const MuonStepArgs& a, uint32_t tiles, uint32_t side, ar_dtype_t grad_dtype,
                             hipStream_t stream) {
  return (side == 128 ? start<128> : start<64>)(a, tiles, grad_dtype, stream);
}

hipError_t launch_muon_gram(const MuonStepArgs& a, uint32_t squares, uint32_t side, hipStream_t stream) {
  if (side == 128)
    muon_square<128, false><<<squares, kProductThreads<128>, 0, stream>>>(a);
  else
    muon_square<64, false><<<squares, kProductThreads<64>, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_muon_poly(const MuonStepArgs& a, uint32_t squares, uint32_t side, hipStream_t stream) {
  if (side == 128)
    muon_square<128, true><<<squares, kProductThreads<128>, 0, stream>>>(a);
  else
    muon_square<64, true><<<squares, kProductThreads<64>, 0, stream>>>(a);
  return hipGetLastError();
}

template <int SIDE>
static hipError_t apply(const MuonStepArgs& a, uint32_t tiles, ar_dtype_t param_dtype, bool copy, hipStream_t stream) {
  const auto kernel = param_dtype == AR_BFLOAT16 ? muon_apply<SIDE, __bf16, false>
                      : copy                     ? muon_apply<SIDE, float, true>
                                                 : muon_apply<SIDE, float, false>;
  kernel<<<tiles, kProductThreads<SIDE>, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_muon_apply(const MuonStepArgs& a, uint32_t tiles, uint32_t side, ar_dtype_t param_dtype, bool copy,
                             hipStream_t stream) {
  return (side == 128 ? apply<128> : apply<64>)(a, tiles, param_dtype, copy, stream);
}

}  // namespace ar
