// query.cu — a step's MLA queries in fp16, for the kernels whose keys are
// widened to fp16 (dense_mla.cu, mass.cu).
//
// bf16 reaches further than fp16, so a head's 576 values are multiplied by one
// power of two 2^e that brings the largest finite one into [2^14, 2^15); the
// kernels multiply that head's logits by 2^-e.  bf16's 8 significant bits fit
// fp16's 11 down to 2^-28 of the head's largest value, and what lies below loses
// at most 2^-39 of it.  A power of two per row would not do: a head's sums know
// nothing of another head's largest value, and one outlier of 2^40 would turn
// the other 95 heads of its row to zeros.
//
// For the attention weights a head whose LSE is -inf (it attended to nothing) counts
// as zeros, so that NaN or infinities in a masked row's query stay out of the sums.
//
// A warp a head and no barrier: 72 16-byte pieces, all loaded before the maximum is
// taken; the kernel that follows sets itself up meanwhile.  Bound by latency: 32
// rows take 5.3 us with cold caches.  A whole call over one row of 997 tokens takes
// 16.5 us with it and took 19.5 with a CTA, a barrier and one scale a row; converting
// inside the kernel that follows cost its softmax warps 5 us for every row a CTA
// touched.
#include "common.cuh"
#include "internal.h"

namespace dsa {

namespace {

constexpr int kWarps = 8;  // heads a CTA
constexpr int kPieces = kLatent / 8;  // 16-byte pieces a head: 72
constexpr int kPer = (kPieces + 31) / 32;
static_assert(kHeads % kWarps == 0 && kPieces * 8 == kLatent, "pieces");

__global__ void __launch_bounds__(32 * kWarps) query_f16_kernel(const uint4* __restrict__ q,
                                                                const float* __restrict__ lse,  // or null
                                                                uint4* __restrict__ out, float* __restrict__ inv) {
  grid_dep_wait();    // the queries may come from the previous kernel
  grid_dep_launch();  // so what the next one reads before its own wait is in place too
  const int lane = threadIdx.x & 31;
  const int64_t head = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), base = head * kPieces;  // of all rows' heads
  uint4 v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = lane + 32 * i < kPieces ? q[base + lane + 32 * i] : make_uint4(0, 0, 0, 0);
  if (lse && lse[head] == -INFINITY) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    m = bf16x2_abs_max(bf16x2_abs_max(bf16x2_abs_max(bf16x2_abs_max(m, v[i].x), v[i].y), v[i].z), v[i].w);
  const int e = f16_shift_of(__reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16)));
  const float scale = __int_as_float((127 + e) << 23);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < kPieces)
      out[base + lane + 32 * i] = make_uint4(bf16x2_to_f16x2(v[i].x, scale), bf16x2_to_f16x2(v[i].y, scale),
                                             bf16x2_to_f16x2(v[i].z, scale), bf16x2_to_f16x2(v[i].w, scale));
  if (lane == 0) inv[head] = __int_as_float((127 - e) << 23);
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t query_f16_bytes(int rows) { return al256((size_t)rows * kHeads * kLatent * 2) + al256((size_t)rows * kHeads * 4); }

dsa_status_t launch_query_f16(const uint16_t* q, const float* lse, int rows, void* workspace, uint16_t** q16,
                              float** inv, cudaStream_t st) {
  *q16 = static_cast<uint16_t*>(workspace);
  *inv = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + al256((size_t)rows * kHeads * kLatent * 2));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * (kHeads / kWarps));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cuda_status(cudaLaunchKernelEx(&cfg, query_f16_kernel, reinterpret_cast<const uint4*>(q), lse,
                                        reinterpret_cast<uint4*>(*q16), *inv));
}

}  // namespace dsa
