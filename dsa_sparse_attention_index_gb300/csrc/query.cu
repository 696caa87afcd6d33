// query.cu — a step's MLA queries in fp16, for the kernels whose keys are
// widened to fp16 (dense_mla.cu, mass.cu).
//
// bf16 reaches further than fp16, so a row's 96 x 576 values are multiplied by
// one power of two 2^e that brings the largest finite one into [2^14, 2^15); the
// kernels multiply the logits by 2^-e.  bf16's 8 significant bits fit fp16's 11
// down to 2^-28 of the row's largest value, and what lies below loses at most
// 2^-39 of it: far below the error of the fp32 sums it goes into.
//
// For the attention weights a head whose LSE is -inf (it attended to nothing) counts
// as zeros, so that NaN or infinities in a masked row's query stay out of the sums.
//
// One CTA a row, nine 16-byte pieces a thread, all loaded before the maximum is
// taken; the kernel that follows sets itself up meanwhile.  (Converting inside
// that kernel cost its softmax warps 5 us for every row a CTA touched.)
#include "common.cuh"
#include "internal.h"

namespace dsa {

namespace {

constexpr int kPieces = 9;
constexpr int kThreads = kHeads * kLatent / 8 / kPieces;  // 768
static_assert(kThreads * kPieces * 8 == kHeads * kLatent && kThreads % 32 == 0, "pieces");

__global__ void __launch_bounds__(kThreads) query_f16_kernel(const uint4* __restrict__ q,
                                                             const float* __restrict__ lse,  // or null
                                                             uint4* __restrict__ out, float* __restrict__ inv) {
  __shared__ uint32_t max_s[kThreads / 32];
  grid_dep_wait();    // the queries may come from the previous kernel
  grid_dep_launch();  // so what the next one reads before its own wait is in place too
  const int64_t base = (int64_t)blockIdx.x * kThreads * kPieces;
  uint4 v[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) v[i] = q[base + i * kThreads + threadIdx.x];
  if (lse) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (lse[blockIdx.x * (int64_t)kHeads + (i * kThreads + threadIdx.x) / (kLatent / 8)] == -INFINITY)
        v[i] = make_uint4(0, 0, 0, 0);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    m = bf16x2_abs_max(bf16x2_abs_max(bf16x2_abs_max(bf16x2_abs_max(m, v[i].x), v[i].y), v[i].z), v[i].w);
  m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
  if ((threadIdx.x & 31) == 0) max_s[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) m = max(m, max_s[i]);
  const int e = f16_shift_of(m);
  const float scale = __int_as_float((127 + e) << 23);
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    out[base + i * kThreads + threadIdx.x] = make_uint4(bf16x2_to_f16x2(v[i].x, scale), bf16x2_to_f16x2(v[i].y, scale),
                                                        bf16x2_to_f16x2(v[i].z, scale), bf16x2_to_f16x2(v[i].w, scale));
  if (threadIdx.x == 0) inv[blockIdx.x] = __int_as_float((127 - e) << 23);
}

}  // namespace

size_t query_f16_bytes(int rows) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  return al((size_t)rows * kHeads * kLatent * 2) + al((size_t)rows * 4);
}

dsa_status_t launch_query_f16(const uint16_t* q, const float* lse, int rows, void* workspace, uint16_t** q16,
                              float** inv, cudaStream_t st) {
  *q16 = static_cast<uint16_t*>(workspace);
  *inv = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                  (((size_t)rows * kHeads * kLatent * 2 + 255) & ~size_t(255)));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  return cuda_status(cudaLaunchKernelEx(&cfg, query_f16_kernel, reinterpret_cast<const uint4*>(q), lse,
                                        reinterpret_cast<uint4*>(*q16), *inv));
}

}  // namespace dsa
