// kda_fill.cuh - kernels whose buffers in shared memory have warps of their own
// to fill them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }


// Named barriers of a CTA: `threads` of them arrive, some of these wait.
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// Two buffers in shared memory: four warps fill them, groups of four warps, one
// on each of the SM's schedulers, empty them.  The groups never meet each other,
// so that one can be at its products while the other is at its elementwise work
// (BAR_START and the next: where a kernel has the first of them tell the second to begin).
constexpr int GROUP = 128, FILL = 128, BAR_FULL = 1, BAR_EMPTY = 5, BAR_GROUP = 9, BAR_START = 11;
__device__ __forceinline__ int bar_full(int stage, int group) { return BAR_FULL + 2 * stage + group; }
__device__ __forceinline__ int bar_empty(int stage, int group) { return BAR_EMPTY + 2 * stage + group; }

// Registers: the launch gives each of 12 warps 168 a thread; the four that fill
// give up what the eight that compute need, 128 * 40 + 256 * 232 = 384 * 168.
// With four computing warps there is room without.
template <int WARPS> __device__ __forceinline__ void registers_to_fill() {
  if constexpr (WARPS == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
}
template <int WARPS> __device__ __forceinline__ void registers_to_compute() {
  if constexpr (WARPS == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
}

// The filling warps: load(c) starts chunk c's copies (c counts from 0 in the
// order of use).
template <int GROUPS, typename F> __device__ __forceinline__ void fill_buffers(int nc, F load) {
  for (int c = 0; c <= nc; ++c) {
    if (c >= 1) {  // the one before has arrived: first of all this is told
      cp_wait<0>();
      __threadfence_block();
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) bar_arrive(bar_full((c - 1) & 1, g), GROUP + FILL);
    }
    if (c == nc) break;
    if (c >= 2) {
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) bar_sync(bar_empty(c & 1, g), GROUP + FILL);
    }
    load(c);
    cp_commit();
  }
}

}  // namespace kda
