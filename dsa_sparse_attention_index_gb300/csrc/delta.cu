// delta.cu — the gated delta rule of the recurrent layers, row by row.
//
// For a head with state S [128 values v][128 keys k], row t:
//   S~ = S diag(exp(gate_t)),  u = beta_t (v_t - S~ k_t),
//   S  = S~ + u k_t^T,         out_t = scale * S q_t = scale * (S~ q_t + u (k_t . q_t))
// so one pass over S~ gives both of its products, and S never leaves registers
// between the rows of a call.  The rows v of S do not touch each other: a CTA
// takes some of them, and a warp needs no other one.
#include <algorithm>

#include "common.cuh"
#include "delta.cuh"
#include "internal.h"

namespace dsa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// What a row brings for this thread's keys 4 l + 32 i .. + 3 (l = lane % 8) and its values.
template <int R>
struct RowData {
  float4 k[4], q[4], a[4];
  float v[R];
  float beta, kq;
};

template <int R>
__device__ __forceinline__ void load_row(const DeltaRows& x, int64_t row, int hq, int h, int l, int vrow, RowData<R>& d) {
  const uint2* kp = reinterpret_cast<const uint2*>(x.k + row * x.ld_k + hq * kDeltaDim) + l;
  const uint2* qp = reinterpret_cast<const uint2*>(x.q + row * x.ld_q + hq * kDeltaDim) + l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d.k[i] = bf16x4_to_float4(__ldg(kp + 8 * i));
    d.q[i] = bf16x4_to_float4(__ldg(qp + 8 * i));
  }
  if (x.gate_dim == 1) {
    const float a = expf(__ldg(x.gate + row * x.ld_gate + h));
#pragma unroll
    for (int i = 0; i < 4; ++i) d.a[i] = make_float4(a, a, a, a);
  } else {
    const float4* gp = reinterpret_cast<const float4*>(x.gate + row * x.ld_gate + (int64_t)h * kDeltaDim) + l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 g = __ldg(gp + 8 * i);
      d.a[i] = make_float4(expf(g.x), expf(g.y), expf(g.z), expf(g.w));
    }
  }
  const uint16_t* vp = x.v + row * x.ld_v + (int64_t)h * kDeltaDim + vrow;
#pragma unroll
  for (int r = 0; r < R; ++r) d.v[r] = bf16_to_float(__ldg(vp + 4 * r));
  d.beta = __ldg(x.beta + row * x.ld_beta + h);
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}
// Sum over the eight lanes that share a row of the state, the same in all of them.
__device__ __forceinline__ float sum8(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  return v + __shfl_xor_sync(0xffffffffu, v, 4);
}

// Grid batch * heads * (128 / (16 R)): a CTA holds 16 R value rows of one
// head's state, a warp 4 R of them; eight lanes share a row (16 keys each).
template <int R>
__global__ void __launch_bounds__(kThreads) delta_rows_kernel(const DeltaRows x, const DeltaSeqs s, uint16_t* out) {
  constexpr int kSplit = kDeltaDim / (4 * R * kWarps);
  const int part = blockIdx.x % kSplit, bh = blockIdx.x / kSplit;
  const int h = bh % x.heads, b = bh / x.heads, hq = h / (x.heads / x.qk_heads);
  const int lane = threadIdx.x & 31, l = lane & 7;
  const int vrow = part * (4 * R * kWarps) + (threadIdx.x >> 5) * 4 * R + (lane >> 3);  // this thread's rows: vrow + 4 r
  int64_t row;
  int n;
  if (!seq_rows(s, b, &row, &n)) return;

  float4 S[R][4];
  const float* in = state_in(s, b, h);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      S[r][i] = in ? *reinterpret_cast<const float4*>(in + (vrow + 4 * r) * kDeltaDim + 4 * l + 32 * i)
                   : make_float4(0.f, 0.f, 0.f, 0.f);

  RowData<R> d;
  if (n > 0) load_row<R>(x, row, hq, h, l, vrow, d);
  for (int t = 0; t < n; ++t) {
    RowData<R> next;
    if (t + 1 < n) load_row<R>(x, row + t + 1, hq, h, l, vrow, next);
    float kq = 0.f, p[R], w[R];
#pragma unroll
    for (int i = 0; i < 4; ++i) kq = dot4(d.k[i], d.q[i], kq);
    kq = sum8(kq);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      p[r] = w[r] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        S[r][i].x *= d.a[i].x, S[r][i].y *= d.a[i].y, S[r][i].z *= d.a[i].z, S[r][i].w *= d.a[i].w;
        p[r] = dot4(S[r][i], d.k[i], p[r]);
        w[r] = dot4(S[r][i], d.q[i], w[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float u = d.beta * (d.v[r] - sum8(p[r]));
      const float o = x.scale * fmaf(u, kq, sum8(w[r]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        S[r][i].x = fmaf(u, d.k[i].x, S[r][i].x), S[r][i].y = fmaf(u, d.k[i].y, S[r][i].y);
        S[r][i].z = fmaf(u, d.k[i].z, S[r][i].z), S[r][i].w = fmaf(u, d.k[i].w, S[r][i].w);
      }
      if (l == r) out[((row + t) * x.heads + h) * kDeltaDim + vrow + 4 * r] = float_to_bf16(o);
    }
    if (s.per_row || t == n - 1) {
      if (float* to = state_out(s, b, t, h)) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(to + (vrow + 4 * r) * kDeltaDim + 4 * l + 32 * i) = S[r][i];
      }
    }
    d = next;
  }
  if (n == 0 && !s.per_row) {
    // a sequence without rows hands its state on
    if (float* to = state_out(s, b, 0, h)) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(to + (vrow + 4 * r) * kDeltaDim + 4 * l + 32 * i) = S[r][i];
    }
  }
}

}  // namespace

dsa_status_t launch_delta_rows(const DeltaRows& x, const DeltaSeqs& s, uint16_t* out, cudaStream_t st) {
  const int64_t heads = (int64_t)s.batch * x.heads;
  if (heads * 2 >= 2 * num_sms()) {
    delta_rows_kernel<4><<<(unsigned)(heads * 2), kThreads, 0, st>>>(x, s, out);
  } else {
    delta_rows_kernel<1><<<(unsigned)(heads * 8), kThreads, 0, st>>>(x, s, out);
  }
  count_launches(1);
  return launch_status();
}

}  // namespace dsa
