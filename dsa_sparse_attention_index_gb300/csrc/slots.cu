// slots.cu — where a step's new tokens go: pages off the free stack into the
// block table, lengths, first rows, positions and cache slots.
//
// With c_i cached and n_i new tokens, request i has have_i = ceil(c_i / 64)
// pages and needs need_i = ceil((c_i + n_i) / 64).  Its rows start at R_i =
// sum_{j<i} n_j and its fresh pages come off the stack behind the F_i =
// sum_{j<i} (need_j - have_j) pages of the requests before it.  Row r of
// request i is position p = c_i + r - R_i on page j = p / 64: a page of the
// table for j < have_i, else entry count - 1 - (F_i + j - have_i) of the stack.
// The row with p % 64 = 0 is the only first one of a fresh page: it puts the
// page into the table.
//
// A step may not fit.  The rows of the one request `cut` at max_rows, and of those
// behind it, are not placed, and their pages stay on the stack.  Where the stack ends
// within the pages of the request `dry`, it and those behind it have rows without a page.
// Lengths count the tokens that have a place, so a table row is whole up to its length.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace dsa {

namespace {

constexpr int kPer = 2;         // requests a thread scans at once
constexpr int kSlotRows = 4;    // rows a thread places at once: 16 bytes of positions, 16 of slots

struct SlotArgs {
  const int32_t *cached, *fresh;
  int32_t batch;
  const int32_t* free_blocks;
  int32_t free_capacity;
  const int32_t* free_count;
  int32_t* free_left;
  int32_t num_blocks;
  int32_t* table;
  int32_t max_blocks;
  int32_t *seq_lens, *starts, *positions, *slots;
  int32_t max_rows;
  int32_t* status;
};

// Request i's lengths; one that does not fit its table row takes part with none.
__device__ __forceinline__ int2 lengths_of(const SlotArgs& a, int i) {
  const int c = a.cached[i], n = a.fresh[i];
  if (c < 0 || n < 0 || (int64_t)c + n > (int64_t)a.max_blocks * kBlock) return make_int2(0, -1);
  return make_int2(c, n);
}
__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kBlock - 1) / kBlock; }

// Bound by a chain of latencies: lengths, scan, search, page, store (64 requests: 3.9
// us in a graph, of which a launch takes 2.3), and with many rows by the search and
// the page's address, 16 bytes of positions and of slots a thread and turn (2,048
// requests, 262,144 rows: 14.7 us in 16 CTAs; row by row in 8 CTAs 26).
// One cluster.  Every CTA scans the requests (a tile of 2,048 at a time, kept
// in shared memory) and places its share of the rows; nothing that the caller
// may pass as input and output at once (lengths, the stack's count) is written
// before the whole cluster has read it.
template <int kSlotThreads>
__global__ void __launch_bounds__(kSlotThreads) assign_slots_kernel(const SlotArgs a) {
  namespace cg = cooperative_groups;
  constexpr int kSlotTile = kSlotThreads * kPer;   // requests of a tile
  __shared__ int s_start[kSlotTile + 1], s_cached[kSlotTile], s_page[kSlotTile];
  __shared__ long long s_warp[32], s_warp2[32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int cta = blockIdx.x, ctas = gridDim.x;
  int count = *a.free_count;
  if (count < 0 || count > a.free_capacity) {
    if (cta == 0 && tid == 0) report(a.status, DSA_ERR_BOUNDS);
    count = 0;
  }
  const bool wide = ((reinterpret_cast<uintptr_t>(a.positions) | reinterpret_cast<uintptr_t>(a.slots)) & 15) == 0;
  // what the one thread finds that scans the request: of `cut` the request, its rows that are placed and all pages up to
  // there; of `dry` the request and its pages
  __shared__ int s_cut, s_cut_rows, s_dry, s_dry_pages;
  __shared__ long long s_cut_pages;
  if (tid == 0) s_cut = s_dry = INT32_MAX;   // (the first tile's scan is before any other write)
  long long rows0 = 0, pages0 = 0;  // of the tiles before
  for (int base = 0; base < a.batch; base += kSlotTile) {
    // scans of rows and of pages, in 64 bits: lengths go up to 2^30
    int c[kPer], n[kPer];
    long long rsum = 0, psum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int i = base + tid * kPer + e;
      c[e] = n[e] = 0;
      if (i < a.batch) {
        const int2 v = lengths_of(a, i);
        if (v.y < 0 && cta == 0) report(a.status, DSA_ERR_BOUNDS);
        c[e] = v.x, n[e] = max(v.y, 0);
      }
      rsum += n[e];
      psum += pages_of(c[e] + n[e]) - pages_of(c[e]);
    }
    long long ri = rsum, pi = psum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long r = __shfl_up_sync(0xffffffffu, ri, o), p = __shfl_up_sync(0xffffffffu, pi, o);
      if (lane >= o) ri += r, pi += p;
    }
    if (lane == 31) s_warp[wid] = ri, s_warp2[wid] = pi;
    __syncthreads();
    constexpr int kWarps = kSlotThreads / 32;
    long long rt = lane < kWarps ? s_warp[lane] : 0, pt = lane < kWarps ? s_warp2[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long r = __shfl_up_sync(0xffffffffu, rt, o), p = __shfl_up_sync(0xffffffffu, pt, o);
      if (lane >= o) rt += r, pt += p;
    }
    const long long rall = __shfl_sync(0xffffffffu, rt, 31), pall = __shfl_sync(0xffffffffu, pt, 31);
    const long long rw = wid ? __shfl_sync(0xffffffffu, rt, wid - 1) : 0;
    const long long pw = wid ? __shfl_sync(0xffffffffu, pt, wid - 1) : 0;
    long long r = rows0 + rw + ri - rsum, p = pages0 + pw + pi - psum;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int j = tid * kPer + e;
      s_start[j] = (int)min(r, (long long)a.max_rows);
      s_cached[j] = c[e];
      s_page[j] = (int)min(p, (long long)INT32_MAX);
      if (cta == 0 && base + j < a.batch) a.starts[base + j] = s_start[j];
      const int have = pages_of(c[e]), need = pages_of(c[e] + n[e]);
      if (r <= a.max_rows && r + n[e] > a.max_rows) {
        s_cut = base + j, s_cut_rows = (int)(a.max_rows - r);
        s_cut_pages = p + pages_of(c[e] + s_cut_rows) - have;
      }
      if (p <= count && p + need - have > count) s_dry = base + j, s_dry_pages = have + (int)(count - p);
      r += n[e];
      p += need - have;
    }
    if (tid == kSlotThreads - 1) s_start[kSlotTile] = (int)min(r, (long long)a.max_rows);
    __syncthreads();
    // the tile's rows, four at a time, in turns over the cluster's threads
    const int first = s_start[0], last = s_start[kSlotTile];
    const int step = ctas * kSlotThreads * kSlotRows;
    for (int g = (first & ~(kSlotRows - 1)) + (cta * kSlotThreads + tid) * kSlotRows; g < last; g += step) {
      const int r0 = max(g, first);
      int lo = 0;   // the last request with start <= r0
#pragma unroll
      for (int w = kSlotTile / 2; w > 0; w >>= 1)
        if (s_start[lo + w] <= r0) lo += w;
      int pos[kSlotRows], page[kSlotRows];
      int32_t* entry[kSlotRows];
#pragma unroll
      for (int e = 0; e < kSlotRows; ++e) {
        const int row = g + e;
        pos[e] = -1, page[e] = 0, entry[e] = nullptr;
        if (row < first || row >= last) continue;
        while (s_start[lo + 1] <= row) ++lo;
        const int cached = s_cached[lo], have = pages_of(cached);
        pos[e] = cached + row - s_start[lo];
        const int j = pos[e] / kBlock;
        int32_t* to = a.table + (int64_t)(base + lo) * a.max_blocks + j;
        const long long at = (long long)count - 1 - ((long long)s_page[lo] + j - have);
        const int32_t* from = j < have ? to : a.free_blocks + at;
        page[e] = j < have || at >= 0 ? *from : -1;
        if (j >= have && pos[e] % kBlock == 0) entry[e] = to;
      }
      int slot[kSlotRows];
#pragma unroll
      for (int e = 0; e < kSlotRows; ++e) {
        slot[e] = -1;
        if (pos[e] < 0) continue;
        if ((unsigned)page[e] >= (unsigned)a.num_blocks) {
          report(a.status, DSA_ERR_BOUNDS);
          continue;
        }
        slot[e] = page[e] * kBlock + pos[e] % kBlock;
        if (entry[e]) *entry[e] = page[e];
      }
      if (wide && g >= first && g + kSlotRows <= last) {
        *reinterpret_cast<int4*>(a.positions + g) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4*>(a.slots + g) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
#pragma unroll
        for (int e = 0; e < kSlotRows; ++e)
          if (pos[e] >= 0) a.positions[g + e] = pos[e], a.slots[g + e] = slot[e];
      }
    }
    rows0 += rall, pages0 += pall;
    __syncthreads();
  }
  const int total = (int)min(rows0, (long long)a.max_rows);
  for (int r = total + cta * kSlotThreads + tid; r < a.max_rows; r += ctas * kSlotThreads) a.positions[r] = a.slots[r] = -1;
  if (ctas > 1) cg::this_cluster().sync();
  for (int i = cta * kSlotThreads + tid; i < a.batch; i += ctas * kSlotThreads) {
    const int2 v = lengths_of(a, i);
    int len = v.y < 0 ? 0 : v.x + v.y;
    if (i >= s_cut) len = v.x + (i == s_cut ? s_cut_rows : 0);
    if (i >= s_dry) len = (int)min((long long)len, (long long)kBlock * (i == s_dry ? s_dry_pages : pages_of(v.x)));
    a.seq_lens[i] = len;
  }
  if (cta == 0 && tid == 0) {
    a.starts[a.batch] = total;
    const long long taken = s_cut == INT32_MAX ? pages0 : s_cut_pages;
    if (rows0 > a.max_rows || taken > count) report(a.status, DSA_ERR_BOUNDS);
    *a.free_left = (int)max(0ll, (long long)count - taken);
  }
}

// CTAs of the largest cluster that the current device can schedule, 16 or 8 (asked once per device).
int most_ctas() {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && known[dev]) return known[dev];
  int n = 0;
  if (cudaFuncSetAttribute(assign_slots_kernel<1024>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 16, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(1024);
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, assign_slots_kernel<1024>, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  n = n > 0 ? 16 : 8;
  if (dev >= 0 && dev < 64) known[dev] = n;
  return n;
}

}  // namespace

dsa_status_t launch_assign_slots(const int32_t* cached, const int32_t* fresh, int batch, const int32_t* free_blocks,
                                 int free_capacity, const int32_t* free_count, int32_t* free_left, int num_blocks,
                                 int32_t* table, int max_blocks, int32_t* seq_lens, int32_t* starts, int32_t* positions,
                                 int32_t* slots, int max_rows, int32_t* status, cudaStream_t st) {
  const SlotArgs a{cached,     fresh,    batch,  free_blocks, free_capacity, free_count, free_left, num_blocks, table,
                   max_blocks, seq_lens, starts, positions,   slots,         max_rows,   status};
  // one CTA for up to 4,096 rows, so that a decode step's few take no cluster; 16 for many where they can be scheduled
  const bool small = max_rows <= 1024 && batch <= 1024;
  const int ctas = max_rows > 8 * 4096 ? most_ctas() : max_rows > 4096 ? 4 : 1;
  const auto kernel = small ? assign_slots_kernel<256> : assign_slots_kernel<1024>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(small ? 256 : 1024);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  count_launches(1);
  if (cuda_status(cudaLaunchKernelEx(&cfg, kernel, a)) != DSA_OK) return DSA_ERR_CUDA;
  return launch_status();
}

}  // namespace dsa
