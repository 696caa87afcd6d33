// delta.cu — the gated delta rule of the recurrent layers, row by row.
//
// For a head with state S [128 values v][128 keys k], row t:
//   S~ = S diag(exp(gate_t)),  u = beta_t (v_t - S~ k_t),
//   S  = S~ + u k_t^T,         out_t = scale * S q_t = scale * (S~ q_t + u (k_t . q_t))
// so one pass over S~ gives both of its products, and S never leaves registers
// between the rows of a call.  The rows v of S do not touch each other: a CTA
// takes some of them, and a warp needs no other one.
#include "common.cuh"
#include "delta.cuh"
#include "internal.h"

namespace dsa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int R = 4;                                  // value rows a thread has a part of
constexpr int kCtaRows = 4 * R * kWarps;              // 64: a CTA's value rows
constexpr int kSplit = kDeltaDim / kCtaRows;

// What a row brings for this thread's keys 4 l + 32 i .. + 3 (l = lane % 8) and its
// values, as loaded: half the registers that the converted numbers would take.
struct RowData {
  uint2 k[4], q[4];
  float4 g[4];   // one decay per head: g[0].x alone
  uint16_t v[R];
  float beta;
};

__device__ __forceinline__ void load_row(const DeltaRows& x, int64_t row, int hq, int h, int l, int vrow, RowData& d) {
  const uint2* kp = reinterpret_cast<const uint2*>(x.k + row * x.ld_k + hq * kDeltaDim) + l;
  const uint2* qp = reinterpret_cast<const uint2*>(x.q + row * x.ld_q + hq * kDeltaDim) + l;
  if (x.gate_dim == 1) {
    d.g[0].x = __ldg(x.gate + row * x.ld_gate + h);
  } else {
    const float4* gp = reinterpret_cast<const float4*>(x.gate + row * x.ld_gate + (int64_t)h * kDeltaDim) + l;
#pragma unroll
    for (int i = 0; i < 4; ++i) d.g[i] = __ldg(gp + 8 * i);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) d.k[i] = __ldg(kp + 8 * i), d.q[i] = __ldg(qp + 8 * i);
  const uint16_t* vp = x.v + row * x.ld_v + (int64_t)h * kDeltaDim + vrow;
#pragma unroll
  for (int r = 0; r < R; ++r) d.v[r] = __ldg(vp + 4 * r);
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

// First row and rows of sequence b where it is a long one; else {0, 0}.
__device__ __forceinline__ int2 long_rows(const DeltaSeqs& s, int b) {
  if (b >= s.batch) return make_int2(0, 0);
  const int r0 = s.starts[b], r1 = s.starts[b + 1];
  // (one outside of 0..rows is reported where it is left out)
  return r0 >= 0 && r1 >= r0 && r1 <= s.rows && r1 - r0 > kFewRows ? make_int2(r0, r1 - r0) : make_int2(0, 0);
}
__device__ __forceinline__ int chunks_of(int rows) { return (rows + kChunk - 1) / kChunk; }

// The long sequences of a prompt call, by one warp, the longest first: a CTA walks a sequence's chunks one after
// another, and one that started last would run alone (7 prompts of up to 1,501 rows, 96 heads: 3 % of the call).  Up to
// 32 sequences by their chunks, more of them by the power of two below.
__device__ __forceinline__ void list_long(const DeltaSeqs& s) {
  const int lane = threadIdx.x;
  int found = 0, chunks = 0;
  if (s.batch <= 32) {
    const int2 rows = long_rows(s, lane);
    const int c = chunks_of(rows.y);
    int at = 0, before = 0;   // the sequences that come first, their chunks
    for (int j = 0; j < s.batch; ++j) {
      const int cj = __shfl_sync(0xffffffffu, c, j);
      if (cj > c || (cj == c && j < lane)) ++at, before += cj;
    }
    found = __popc(__ballot_sync(0xffffffffu, c > 0));
    if (c > 0 && at < s.many) s.index[1 + at] = make_int4(rows.x, rows.y, before, lane);
  } else {
    uint32_t sizes = 0;   // bit e: there are sequences of 2^e to 2^(e + 1) - 1 chunks
    for (int b = lane; b < s.batch; b += 32) {
      const int c = chunks_of(long_rows(s, b).y);
      if (c > 0) sizes |= 1u << (31 - __clz(c));
    }
    sizes = __reduce_or_sync(0xffffffffu, sizes);
    while (sizes) {
      const int e = 31 - __clz(sizes);
      sizes ^= 1u << e;
      for (int b0 = 0; b0 < s.batch; b0 += 32) {
        const int2 rows = long_rows(s, b0 + lane);
        int c = chunks_of(rows.y);
        if (c >> e != 1) c = 0;
        const uint32_t any = __ballot_sync(0xffffffffu, c > 0);
        if (any == 0) continue;
        int before = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += v;
        }
        const int at = found + __popc(any & ((1u << lane) - 1));
        // starts that do not ascend can make more long sequences than there are rows for
        if (c > 0 && at < s.many) s.index[1 + at] = make_int4(rows.x, rows.y, chunks + before - c, b0 + lane);
        found += __popc(any);
        // (overlapping ones could also count past 32 bits; there is no room for any that begin so far behind)
        chunks = min(chunks + __shfl_sync(0xffffffffu, before, 31), 1 << 30);
      }
    }
  }
  if (lane == 0) s.index[0].x = min(found, s.many);
}

// Grid batch * heads * 2 (and one CTA before them in a prompt call): a CTA holds 64 value rows of one head's state, a warp 16
// of them; eight lanes share a row (16 keys each), so a product with the keys takes
// three shuffles.  Bound by the states' bytes: with 64 registers of state a thread
// and three CTAs an SM, 96 KB are on their way.  32 sequences x 96 heads read and
// write 0.41 GB in 61.4 us (6.6 TB/s, 0.97 of the measured copy); two CTAs an SM
// take 72, two rows a thread and five CTAs 67, one row a thread 90.  Few heads are
// no faster in smaller parts (32 heads: 2.8 us).  Prompt calls have an instance of their own:
// with their ranges and list in it decode takes 168 registers for 152, and 1 to 8 % longer.
template <bool PROMPT>
__global__ void __launch_bounds__(kThreads, 3) delta_rows_kernel(const DeltaRows x, const DeltaSeqs s, uint16_t* out) {
  const bool lists = PROMPT && s.index;
  if (lists && blockIdx.x == 0) {   // first, so that it is done before the others
    if (threadIdx.x < 32) list_long(s);
    return;
  }
  const int cta = (int)blockIdx.x - (lists ? 1 : 0), part = cta % kSplit, bh = cta / kSplit;
  const int h = bh % x.heads, b = bh / x.heads, hq = h / (x.heads / x.qk_heads);
  const int lane = threadIdx.x & 31, l = lane & 7;
  const int vrow = part * kCtaRows + (threadIdx.x >> 5) * 4 * R + (lane >> 3);  // this thread's rows: vrow + 4 r
  const int64_t at = (int64_t)vrow * kDeltaDim + 4 * l;
  int64_t row;
  int n;
  if (PROMPT) {
    if (!seq_rows(s, b, &row, &n)) return;
  } else {
    row = (int64_t)b * s.nq, n = s.nq;
  }
  if (PROMPT && n > kFewRows) return;

  float4 S[R][4];
  const float* in = state_in(s, b, h);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      S[r][i] = in ? *reinterpret_cast<const float4*>(in + at + r * 4 * kDeltaDim + 32 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
  auto store = [&](float* to) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(to + at + r * 4 * kDeltaDim + 32 * i) = S[r][i];
  };

  RowData d;
  if (n > 0) load_row(x, row, hq, h, l, vrow, d);
  for (int t = 0; t < n; ++t) {
    float kq = 0.f, p[R], w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) p[r] = w[r] = 0.f;
    const float a1 = x.gate_dim == 1 ? expf(d.g[0].x) : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 k = bf16x4_to_float4(d.k[i]), q = bf16x4_to_float4(d.q[i]);
      const float4 a = x.gate_dim == 1 ? make_float4(a1, a1, a1, a1)
                                       : make_float4(expf(d.g[i].x), expf(d.g[i].y), expf(d.g[i].z), expf(d.g[i].w));
      kq = dot4(k, q, kq);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        S[r][i].x *= a.x, S[r][i].y *= a.y, S[r][i].z *= a.z, S[r][i].w *= a.w;
        p[r] = dot4(S[r][i], k, p[r]);
        w[r] = dot4(S[r][i], q, w[r]);
      }
    }
    kq = sum8(kq);
    float u[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      u[r] = d.beta * (bf16_to_float(d.v[r]) - sum8(p[r]));
      const float o = x.scale * fmaf(u[r], kq, sum8(w[r]));
      if (l == r) out[((row + t) * x.heads + h) * kDeltaDim + vrow + 4 * r] = float_to_bf16(o);
    }
    uint2 kr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) kr[i] = d.k[i];
    if (t + 1 < n) load_row(x, row + t + 1, hq, h, l, vrow, d);   // on its way while the state is updated and stored
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 k = bf16x4_to_float4(kr[i]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        S[r][i].x = fmaf(u[r], k.x, S[r][i].x), S[r][i].y = fmaf(u[r], k.y, S[r][i].y);
        S[r][i].z = fmaf(u[r], k.z, S[r][i].z), S[r][i].w = fmaf(u[r], k.w, S[r][i].w);
      }
    }
    if (!PROMPT || t == n - 1)
      if (float* to = state_out(s, b, t, h)) store(to);
  }
  if (PROMPT && n == 0)   // a sequence without rows hands its state on
    if (float* to = state_out(s, b, 0, h)) store(to);
}

}  // namespace

dsa_status_t launch_delta_rows(const DeltaRows& x, const DeltaSeqs& s, uint16_t* out, cudaStream_t st) {
  const int64_t ctas = (int64_t)s.batch * x.heads * kSplit + (s.index ? 1 : 0);
  if (s.starts) {
    delta_rows_kernel<true><<<(unsigned)ctas, kThreads, 0, st>>>(x, s, out);
  } else {
    delta_rows_kernel<false><<<(unsigned)ctas, kThreads, 0, st>>>(x, s, out);
  }
  count_launches(1);
  return launch_status();
}

}  // namespace dsa
