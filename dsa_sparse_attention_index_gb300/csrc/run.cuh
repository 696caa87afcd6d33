// run.cuh — an equal share of a line of work for every CTA of a persistent
// grid.  The rows' items (tiles, or parts) lie on one line, row after row; CTA
// c takes the run [c per, (c + 1) per).  Row lengths are read on the device, so
// a ragged batch balances without the host knowing its lengths.
#pragma once

#include <stdint.h>

namespace dsa {

struct Run {
  int64_t pos, hi;   // this CTA's run
  int row;           // the row that holds pos (rows if none does)
  int64_t start;     // that row's first item
};

// By all kThreads threads of the CTA: count(r) items of row r
// (fixed_per > 0: that many a CTA, and hi is the line's end).
// each(r, first, n, per) is called once for every row by CTA 0.  `scratch`: 32
// int64 of shared memory.
template <int kThreads, class Count, class Each>
__device__ __forceinline__ Run find_run(int rows, int fixed_per, int64_t* scratch, Count count, Each each) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps <= 30, "scratch");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // up to kThreads rows, one scan gives the total and every row's place
  const bool small = rows <= kThreads;
  int64_t total = 0, n = 0;
  if (!small) {
    int64_t sum = 0;
    for (int r = threadIdx.x; r < rows; r += kThreads) sum += count(r);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) scratch[warp] = sum;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) total += scratch[i];
    __syncthreads();
  }
  Run w;
  int64_t per = 0;
  auto place = [&]() {
    const int64_t even = (total + gridDim.x - 1) / (int64_t)gridDim.x;
    per = fixed_per ? fixed_per : (even > 1 ? even : 1);
    w.pos = (int64_t)blockIdx.x * per;
    w.hi = fixed_per ? total : (w.pos + per < total ? w.pos + per : total);
  };
  if (!small) place();
  if (threadIdx.x == 0) scratch[30] = rows;
  int64_t base = 0;
  for (int r0 = 0; r0 < rows; r0 += kThreads) {
    const int r = r0 + threadIdx.x;
    n = r < rows ? count(r) : 0;
    int64_t inc = n;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (r0 > 0) __syncthreads();
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int64_t before = base;
    for (int i = 0; i < kWarps; ++i) {
      const int64_t v = scratch[i];
      if (i < warp) before += v;
      base += v;
    }
    if (small) {
      total = base;
      place();
    }
    const int64_t first = before + inc - n;
    if (n > 0 && w.pos >= first && w.pos < first + n) {
      scratch[30] = r;
      scratch[31] = first;
    }
    if (blockIdx.x == 0 && r < rows) each(r, first, n, per);
    if (blockIdx.x != 0 && base > w.pos) break;  // the same in every thread
  }
  if (rows == 0) place();
  __syncthreads();
  w.row = (int)scratch[30];
  w.start = scratch[31];
  return w;
}

}  // namespace dsa
