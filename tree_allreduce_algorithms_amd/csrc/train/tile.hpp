// A block's tile of a matrix product by matrix instructions (gfx950), shared by
// the experts' products and the Muon step.
//
// D[m][n] = sum_k A[m][k] B[k][n], k in steps.  A step of each operand lies in
// LDS as 16-byte chunks (8 elements) of lines:
//   k-major   a line is one row m (or column n): the step's k, consecutive
//   r-major   a line is one k: consecutive rows (columns) of the tile
// so either order of an operand in memory is staged as it is.  A wave reads a
// k-major fragment by 16-byte loads and an r-major one by the transposing
// loads, which give a lane four k of one row.  Chunks are permuted within a
// line by the line's number, so that the lanes of one access meet different
// banks.
//
// Two or more steps are in LDS: the loads of later ones are under way while one is
// multiplied; one barrier a step.  For operands in the caches more than two measured
// slower (8192^3: 1,276 TFLOP/s with four half steps against 1,310 with two whole
// ones): it is not the loads' latency that binds but what L2 and LDS move, so tiles
// are as wide as the registers of two blocks on a CU allow.
//
// B's columns are dealt to the fragments so that a lane holds 16 consecutive
// ones in four fragments (`turned`), four of each, and so that the lanes of a
// transposing load meet all banks: see column().
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ar {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(4))) short s16x4;

__device__ __forceinline__ f32x4 multiply(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 multiply(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

typedef __attribute__((address_space(3))) char lds_char;

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_char*)p));
}

// The first of the four columns that place i of a turned fragment j has: the 16
// from 64 (j / 4) + 16 i on are dealt to four fragments, at each place in another
// order, so that half of an access' 8-byte pieces are first halves of chunks and
// half are second ones (in one order for all, 32 % of LDS' cycles were conflicts).
__device__ __forceinline__ constexpr int column(int j, int i) { return j / 4 * 64 + 16 * i + (j + i) % 4 * 4; }

// One operand's step in LDS: R rows (or columns) times STEP k.
template <int R, bool RMAJOR, int STEP, bool TURNED> struct Staged {
  static constexpr int kLines = RMAJOR ? STEP : R;
  static constexpr int kPerLine = (RMAJOR ? R : STEP) / 8;     // chunks
  static constexpr int kChunks = R * STEP / 8;
  static constexpr int kBytes = R * STEP * 2;
  static_assert(STEP == 32 || STEP == 64, "bank permutations are for these");
  static_assert(!TURNED || R % 64 == 0, "columns are dealt in groups of 64");

  // Where chunk `c` of a line lies among the line's chunks.  An access reads 16
  // bytes of 8 lines at a time (k-major), or 8 bytes at four places of each of
  // eight lines (r-major; four from each of two that are 8 apart), which lie in
  // different banks so.
  static __device__ __forceinline__ int place(int line, int c) {
    if (RMAJOR) {
      if (TURNED) return c ^ (kPerLine >= 16 ? (line & 1) | (line & 2) << 2 | (line >> 2 & 2) : (line >> 1 & 1) | (line >> 2 & 2));
      return c ^ ((2 * (line & 3) + (kPerLine >= 16 ? line & 8 : 0)) & (kPerLine - 1));
    }
    if (STEP == 64) return c ^ (TURNED ? (line & 3) | (line >> 2 & 4) : line & 7);
    return c ^ (TURNED ? (line >> 1 & 1) | (line >> 3 & 2) : line >> 1 & 3);
  }

  // The lane's 8 k (8 (lane / 16) and on, of 32 from k0) of a row of fragment j:
  // row r0 + 16 j + lane % 16, or turned, r0 + column(j, i) + q of lane % 16 = 4 i + q.
  template <class V>
  static __device__ __forceinline__ V fragment(const char* step, int r0, int j, int k0, int lane) {
    const int l = lane % 16;
    if (!RMAJOR) {
      const int line = r0 + (TURNED ? column(j, l / 4) + l % 4 : j * 16 + l), c = k0 / 8 + lane / 16;
      return *reinterpret_cast<const V*>(step + (line * kPerLine + place(line, c)) * 16);
    } else {
      // of each 16 lanes, four lie along a line and four lines are read; lane l
      // gets row l of the four k
      const int line = k0 + 8 * (lane / 16) + l / 4, row = r0 + (TURNED ? column(j, l % 4) : j * 16 + l % 4 * 4);
      union {
        V v;
        s16x4 part[2];
      } u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const char* at = step + ((line + 4 * i) * kPerLine + place(line + 4 * i, row / 8)) * 16 + row % 8 * 2;
        u.part[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at));
      }
      return u.v;
    }
  }
};

// The loads of operands whose rows allow 16-byte accesses: straight to LDS,
// 1 KB a wave, past the registers.  `limit` bytes from `base` may be read; an
// offset of kNowhere gives zeros.
constexpr uint32_t kNowhere = 0xfffffff0u;
constexpr uint32_t kReach = 0x80000000u;      // bytes that one base can reach

struct Source {
  u32x4 words;
  __device__ __forceinline__ explicit Source(const void* base) {
    const uint64_t p = reinterpret_cast<uintptr_t>(base);
    words[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p));
    words[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p >> 32) & 0xffffu);
    words[2] = kReach;
    words[3] = 0x00020000u;
  }
};

// 16 bytes a lane from `offset` of the source to lds + 16 lane; lds is uniform.
// Written as asm because the compiler takes every later LDS read for a reader
// of this load's target and would wait for all of them; settled() waits.
__device__ __forceinline__ void load_to_lds(const Source& s, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               ::"s"(lds), "v"(offset), "s"(s.words)
               : "m0", "memory");
}

// Waits until all of the wave's loads to LDS have arrived and its own LDS reads
// are done.
__device__ __forceinline__ void settled() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

// Multiplies one step: acc[i][j] holds rows 16 i and the columns of fragment j of
// the wave's part, D[n][m] in a lane: row lane % 16, columns 4 (lane / 16) +
// element of the fragment, so turned, column(j, lane / 16) + element.  With P = 2 a value is the sum of two planes, kBytes apart;
// their products without that of the two small parts are added up.
template <int TM, int TN, class V, int P, int STEP, class A, class B>
__device__ __forceinline__ void multiply_step(const char* a, const char* b, int m0, int n0, int lane,
                                              f32x4 (&acc)[TM][TN]) {
#pragma unroll
  for (int k0 = 0; k0 < STEP; k0 += 32) {
    V fa[P][TM], fb[P][TN];
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[p][i] = A::template fragment<V>(a + p * A::kBytes, m0, i, k0, lane);
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[p][j] = B::template fragment<V>(b + p * B::kBytes, n0, j, k0, lane);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if (P == 2) {
          acc[i][j] = multiply(fb[P - 1][j], fa[0][i], acc[i][j]);
          acc[i][j] = multiply(fb[0][j], fa[P - 1][i], acc[i][j]);
        }
        acc[i][j] = multiply(fb[0][j], fa[0][i], acc[i][j]);
      }
  }
}

template <int TM, int TN> __device__ __forceinline__ void clear(f32x4 (&acc)[TM][TN]) {
#pragma unroll
  for (auto& row : acc)
#pragma unroll
    for (auto& x : row) x = f32x4{0, 0, 0, 0};
}

}  // namespace
}  // namespace ar
