// Reductions across a wave's 64 lanes or a block, shared by the training
// kernels (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ar {
namespace {

constexpr int kWave = 64;

template <class T> __device__ __forceinline__ T wave_sum(T x) {
#pragma unroll
  for (int d = kWave / 2; d > 0; d /= 2) x += __shfl_xor(x, d);
  return x;
}

// Sum over the block's waves, in wave order; every thread gets it.
template <int BLOCK> __device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[BLOCK / kWave];
  x = wave_sum(x);
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = x;
  __syncthreads();
  double s = part[0];
#pragma unroll
  for (int w = 1; w < BLOCK / kWave; ++w) s += part[w];
  __syncthreads();
  return s;
}

// Values that pass from block to block within a launch go through memory by
// relaxed atomics of agent scope only: these are performed where every XCD
// sees them, past the L2s.  What is left to do is to wait for them before
// saying so, which settle() does for the wave's own; a release and an acquire
// of agent scope would also write back and drop the whole L2, which measured
// about 20 ns a block, one block after another (2,048 blocks: 40 us).
// This rests on what gfx950 does, not on C++'s memory model, by which a relaxed
// read need not see what came before the write it reads.  So every access to
// such values within a launch must be one of these: a plain load or store could
// stay in an XCD's L2, and no test would have to show it.  (What the last block
// resets by plain stores is read by later launches only.)
template <class T> __device__ __forceinline__ T shared_load(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T> __device__ __forceinline__ void shared_store(T* p, T x) {
  __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T> __device__ __forceinline__ T shared_add(T* p, T x) {
  return __hip_atomic_fetch_add(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void settle() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// True in every thread of the block that is the last of `blocks` to get here;
// it then sees what all threads of the others passed on before.  `arrived`
// counts the blocks, from 0.
__device__ __forceinline__ bool last_to_arrive(uint32_t* arrived, uint32_t blocks) {
  __shared__ bool last;
  settle();
  __syncthreads();
  if (threadIdx.x == 0) last = shared_add(arrived, 1u) == blocks - 1;
  __syncthreads();
  return last;
}

}  // namespace
}  // namespace ar
