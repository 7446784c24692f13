// What the kernels over ragged batches of tokens share: programmatic launch and
// the sequences of a window of tokens.
#pragma once

#include <climits>

#include "device.cuh"

namespace pkv {

constexpr int kWindow = 32;         // consecutive tokens that one CTA (column) handles: a warp's lanes
constexpr int kWindowThreads = 256;

// Sequences of the window's tokens of a ragged batch, by the whole CTA: lane i of
// warp 0 gets the number of sequences that end at or before token t0 + i, i.e. its
// sequence (num_seqs if it lies past the last).  One pass over the offsets with
// every load in flight, not a chain of dependent ones.
__device__ __forceinline__ int window_seq(const int32_t* cu, int num_seqs, int t0, int* cnt_s) {
  const int tid = threadIdx.x;
  if (tid < kWindow) cnt_s[tid] = 0;  // [0]: ends at or before t0; [i]: ends at t0 + i
  __syncthreads();
  const int t1 = t0 + min(kWindow, INT_MAX - t0);
  int before = 0;
#pragma unroll 4
  for (int i = tid; i < num_seqs; i += kWindowThreads) {
    const int end = cu[i + 1];
    if (end <= t0) ++before;
    else if (end < t1) atomicAdd(cnt_s + (end - t0), 1);
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if ((tid & 31) == 0 && before > 0) atomicAdd(cnt_s, before);
  __syncthreads();
  if (tid >= kWindow) return 0;
  int x = cnt_s[tid];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (tid >= o) x += y;
  }
  return x;
}

// Programmatic launch: this kernel may have started while the one before it
// ends.  Everything that it reads may still be written then, by a kernel of the
// library or of the caller: lengths, offsets and tables as well as the cache.  Here
// and in the attention kernels all of it is read with ordinary loads, after the
// wait: read-only ones (__ldg) are for data that nothing changes while the kernel
// runs, and may be moved before the wait.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may start while this one runs (and waits in the same way).
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace pkv
