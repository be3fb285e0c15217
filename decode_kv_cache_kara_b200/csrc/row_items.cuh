// Work items over ragged rows, found on the device: the host knows neither lengths nor counts,
// so every block numbers the items itself. Rows are taken THREADS at a time; one thread counts
// one row's items, a block-wide prefix sum numbers them, and item -> row is a binary search
// over the prefix in shared memory.
#pragma once

#include "common.cuh"

namespace kara {

template <int THREADS>
struct RowItems {
  int start[THREADS + 1];        // first item of each row of the chunk; [THREADS] = total
  int warp_total[THREADS / 32];
};

// Numbers the items of THREADS rows (count: this thread's row). Every thread must call it.
template <int THREADS>
__device__ __forceinline__ void row_items_scan(RowItems<THREADS>& s, int count) {
  const int lane = lane_id(), warp = warp_id();
  int x = count;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();               // the previous chunk's items are no longer read
  if (lane == 31) s.warp_total[warp] = x;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) before += w < warp ? s.warp_total[w] : 0;
  s.start[threadIdx.x] = before + x - count;
  if (threadIdx.x == THREADS - 1) s.start[THREADS] = before + x;
  __syncthreads();
}

// The row of the chunk that holds item `i` (0 <= i < start[THREADS]).
template <int THREADS>
__device__ __forceinline__ int row_items_find(const RowItems<THREADS>& s, int i) {
  int lo = 0, hi = THREADS;      // start[lo] <= i < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.start[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace kara
