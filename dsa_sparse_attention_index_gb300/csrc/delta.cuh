// delta.cuh — what the kernels of the gated delta rule share: their arguments
// and the sequences' rows and states.
#pragma once

#include "common.cuh"

namespace dsa {

constexpr int kDeltaDim = DSA_DELTA_DIM;
constexpr int kStateFloats = kDeltaDim * kDeltaDim;  // one head's state
// Sequences of a prompt call with up to this many rows go row by row.  A chunk of 64 rows takes the same time however
// few of them are there: one sequence of 96 heads 25-26 us, in rows 18.5 us for 16 rows, 25.9 for 24, 33 for 32;
// 64 sequences 840 us, in rows 105 us for 1 row, 627 for 16, 911 for 24.
constexpr int kFewRows = 20;
constexpr int kChunk = 64;

// dsa_delta_rows_t with the number of value heads.
struct DeltaRows {
  const uint16_t *q, *k, *v;
  const float *gate, *beta;
  int64_t ld_q, ld_k, ld_v, ld_gate, ld_beta;
  int32_t heads, qk_heads, gate_dim;
  float scale;
};

// The sequences of a call: rows of sequence b are nq b .. nq (b + 1) - 1, or
// starts[b] .. starts[b + 1] - 1 where starts is given.
struct DeltaSeqs {
  float* pool;
  int64_t slot_stride;      // floats
  int32_t num_slots;
  int32_t batch, rows, nq;
  const int32_t* starts;
  const int32_t *slots_in, *slots_out;   // out: [batch][nq], a state after each row; with starts [batch], the last one
  int32_t* status;
  // Prompt calls: the sequences of more than kFewRows rows, of which there can be `many`: their number in the first
  // entry, then for each its first row, its rows, the chunks of 64 rows of those before it, and its index.
  int4* index;
  int32_t many;
};

// First row and number of rows of a prompt call's sequence b; false where starts is not
// ascending within 0..rows (such a sequence is left out).
__device__ __forceinline__ bool seq_rows(const DeltaSeqs& s, int b, int64_t* row, int* n) {
  const int r0 = s.starts[b], r1 = s.starts[b + 1];
  if (r0 < 0 || r1 < r0 || r1 > s.rows) {
    if (threadIdx.x == 0) report(s.status, DSA_ERR_BOUNDS);
    return false;
  }
  *row = r0, *n = r1 - r0;
  return true;
}

// The state that head h of sequence b starts from; null: zeros.
__device__ __forceinline__ const float* state_in(const DeltaSeqs& s, int b, int h) {
  const int slot = s.slots_in[b];
  if (slot == -1) return nullptr;
  if (slot < 0 || slot >= s.num_slots) {
    if (threadIdx.x == 0) report(s.status, DSA_ERR_BOUNDS);
    return nullptr;
  }
  return s.pool + slot * s.slot_stride + (int64_t)h * kStateFloats;
}

// Where the state after row t goes; null: nowhere.
__device__ __forceinline__ float* state_out(const DeltaSeqs& s, int b, int t, int h) {
  const int slot = s.slots_out[s.starts ? b : b * s.nq + t];
  if (slot == -1) return nullptr;
  if (slot < 0 || slot >= s.num_slots) {
    if (threadIdx.x == 0) report(s.status, DSA_ERR_BOUNDS);
    return nullptr;
  }
  return s.pool + slot * s.slot_stride + (int64_t)h * kStateFloats;
}

__device__ __forceinline__ float bf16_to_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t float_to_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ __forceinline__ float4 bf16x4_to_float4(uint2 v) {
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xFFFF0000u));
}

// Row by row (delta.cu), and ragged prompts in chunks of 64 rows (delta_chunk.cu).
dsa_status_t launch_delta_rows(const DeltaRows& x, const DeltaSeqs& s, uint16_t* out, cudaStream_t st);
size_t delta_chunk_workspace_bytes(int rows, int batch, int heads);
dsa_status_t launch_delta_chunks(const DeltaRows& x, const DeltaSeqs& s, uint16_t* out, void* workspace, cudaStream_t st);

}  // namespace dsa
