// delta_chunk.cu — the gated delta rule over prompts, 64 rows at once.
//
// For the rows i = 1..64 of a chunk behind the state S0, with P_i = prod_{s<=i}
// a_s (a = exp(gate), by channel) and the decay D_ij = prod_{j<s<=i} a_s:
//   A_ij = beta_i sum_d k_i k_j D_ij (j < i),   T = (I + A)^-1 diag(m),
//   R = diag(p) (V - (K P) S0^T),   U = T R,   beta = m p, p a power of two, m in [1, 2)
//   out = scale ((Q P) S0^T + B U),  B_ij = sum_d q_i k_j D_ij (j <= i),
//   S = S0 diag(P_64) + U^T (K D_64)
// which is the rule of delta.cu with its 64 steps solved as one triangular system.
// It is the same rule for a key k / s with the value v / s and beta s^2, so every row
// is taken with the power of two s that brings its key's largest element into [1, 2):
// rows whose keys differ in length by any factor share the chunk's powers of two
// without loss, and with p in R, T's diagonal is one to two whatever beta is.  Queries are
// taken likewise, the scale as a number in [1, 2): a row's outputs, rounded to bf16, are
// multiplied by the powers of two that its query and the scale lost.
//
// Two kernels.  delta_prepare_kernel: everything that does not depend on the
// state, a CTA per chunk and head, into a record of operands laid out as the tensor
// core reads them.  delta_chain_kernel: a CTA per sequence and head walks the
// chunks; the state stays in registers in fp32.  2,048 rows of 96 heads: 177 us and
// 143 us (row by row 5,478 us).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "delta.cuh"
#include "internal.h"

namespace dsa {

namespace {

constexpr int kTileHalf = kChunk * 128;                // 64 rows of 64 fp16 (128 bytes, 128-byte swizzle)
constexpr int kTileBytes = 2 * kTileHalf;              // 64 rows x 128 channels
// A record: p K P (high and low parts), Q P, T (high and low), then B, K D (high and low), then the head's floats.
constexpr int kRecKp = 0;
constexpr int kRecQp = kRecKp + 2 * kTileBytes;
constexpr int kRecT = kRecQp + kTileBytes;
constexpr int kRecB = kRecT + 2 * kTileHalf;
constexpr int kRecKd = kRecB + kTileHalf;
constexpr int kRecHead = kRecKd + 2 * kTileBytes;      // 106,496
constexpr int kRecBytes = kRecHead + 1024;
constexpr int kPart1 = kRecB, kPart2 = kRecHead - kRecB;   // what is read first, and last
// floats of the record's head
enum : int { kHdBad = 0, kHdInvKp, kHdInvB, kHdInvK, kHdSumKp, kHdSumT, kHdSumKd, kHdP = 16, kHdV = kHdP + kDeltaDim, kHdO = kHdV + kChunk / 2 };
// (V, O: the powers of two that a row's value and its outputs are times, as bf16; V a row's, O its twice)
constexpr int kHeadBytes = 4 * (kHdO + kChunk);
constexpr int kHeadVBytes = 2 * kChunk;
// T's power of two: its diagonal is one to two, so 2^11 of room above it, and the parts' last bit is 2^-28.
constexpr float kScaleT = 8.f;

struct ChunkArgs {
  DeltaRows x;
  DeltaSeqs s;
  uint8_t* records;   // [chunks of the long sequences, one sequence after another][heads]
  int32_t chunks;     // room for so many
  uint16_t* out;
  int resident;       // CTAs of the first kernel that run at once
};

// The power of two that brings a bound below 2^(top + 1).
__device__ __forceinline__ float pow2_scale(float bound, int top) {
  const int e = (int)((__float_as_uint(bound) >> 23) & 0xFFu) - 127;
  return __uint_as_float((uint32_t)(max(-126, min(126, top - e)) + 127) << 23);
}
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }

// Two neighbouring channels.  (The packed fp32 instructions take fewer slots, but the
// moves into register pairs cost more: a chain of 32 chunks 164 us with them, 145 without.)
using f32x2 = float2;
__device__ __forceinline__ f32x2 pack2(float x, float y) { return make_float2(x, y); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) { return make_float2(a.x - b.x, a.y - b.y); }
__device__ __forceinline__ float reciprocal(float x) {   // within one unit in the last place
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f32x2 bf16x2_to_f32x2(uint32_t v) {
  return pack2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

// Two values as fp16: the upper 11 bits of each, and 11 bits of what they leave,
// so 21 bits in all (the first part is cut, not rounded: that takes no way back
// from fp16, and the rest holds its sign).
__device__ __forceinline__ uint32_t f16x2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void split_f16(f32x2 v, uint32_t& hi, uint32_t& lo) {
  const float2 f = v;
  const float hx = __uint_as_float(__float_as_uint(f.x) & 0xFFFFE000u), hy = __uint_as_float(__float_as_uint(f.y) & 0xFFFFE000u);
  const float2 r = sub2(v, pack2(hx, hy));
  hi = f16x2(hx, hy);
  lo = f16x2(r.x, r.y);
}
// The same with the first part rounded to nearest, where it is also used alone (cut ones would make
// the outputs 3.5e-4 too small).
__device__ __forceinline__ void split_f16_rn(f32x2 v, uint32_t& hi, uint32_t& lo) {
  hi = f16x2(v.x, v.y);
  f32x2 r;   // v - hi without a way back to fp32 (2,048 rows of 96 heads: 326 us for 329)
  asm("{\n .reg .f16 a, b, m;\n mov.b32 {a, b}, %2;\n mov.b16 m, 0xBC00;\n fma.rn.f32.f16 %0, a, m, %3;\n fma.rn.f32.f16 %1, b, m, %4;\n}\n"
      : "=f"(r.x), "=f"(r.y) : "r"(hi), "f"(v.x), "f"(v.y));
  lo = f16x2(r.x, r.y);
}
__device__ __forceinline__ uint32_t bf16x2(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// ---------------------------------------------------------------- prepare
// A thread has two channels of 16 rows: k, q and the decays in registers, running
// products of the decays forward (K P, Q P, X) and backward (K D, Y).  A and B by
// blocks of 16 rows, X Y^T:
//   within a block       X_i = k_i L_i c,  Y_j = k_j / (L_j c), L the decays from the block's
//                        start, c a power of two that centres them by channel: what a pair
//                        gets is a quotient of products of 16 factors at most.  A block whose
//                        decays leave 2^-120 .. 2^10 is computed pair by pair instead.
//   between two blocks   Y_j = k_j times the decays from row j to an anchor, X_i = k_i times those from there, all
//                        products of factors: nothing underflows that should not.  Three anchors
//                        (the starts of rows 16, 32 and 48) let X and Y stand in shared memory at once.
// Within a block the factors are fp32, since a quotient's factors may be large, cut into two tf32 on
// the way into the mma; between blocks they are two fp16 times a power of two, made once.
// Three products either way, 21 bits; the queries one factor of 11 bits, rounded (as bf16 in the blocks
// they put outputs 2.0e-3 off instead of 1.7e-3, which is bf16's own rounding).  (Two bf16 parts everywhere left states 7 to 10e-7
// off instead of 4 to 6e-7; tf32 everywhere took 5 % longer.)  The inverse of I + A goes by
// blocks: the diagonal ones by substitution, a thread a column, while other warps make
// tiles, then two levels of products.
// What bounds it: 34,800 warp instructions a chunk and head at 2.1 a cycle, ten phases that wait for
// each other's warps; its memory traffic could go at twice the rate.  16 warps an SM, as registers and
// shared memory allow; 512 threads a CTA or 16-byte pieces a thread were slower, and
// so was K D made by the warps that the inverse leaves idle (312 us for 302 in all).
constexpr int kPrepThreads = 256;
constexpr int kPX = 0;                            // X = k L c, fp32: 64 rows x 512 bytes
constexpr int kPY = kPX + kChunk * 512;           // Y, fp32
constexpr int kPQ = kPY + kChunk * 512;           // q L c, tf32: 64 rows x 512 bytes, of which the second half in A's place
constexpr int kPartHalf = kChunk * 256;           // X and Y as two fp16 parts, one behind the other
constexpr int kLdA = kChunk + 4;                  // floats: rows start four banks apart
constexpr int kPA = kPQ + kChunk * 256;           // A, then (I + A)^-1, fp32 [64][68]
constexpr int kPB = kPA + kChunk * kLdA * 4;    // B, fp16, the record's image
constexpr int kPTab = kPB + kTileHalf;            // block products [4][128]
constexpr int kPSum = kPTab + 4 * kDeltaDim * 4;  // sums of their logarithms
constexpr int kPBeta = kPSum + 4 * kDeltaDim * 4;
constexpr int kPMisc = kPBeta + kChunk * 4;
constexpr int kPRowMax = kPMisc + 256;            // [2 halves of the channels][64 rows]: largest |k| and |q|, as bf16
constexpr int kPRowScale = kPRowMax + 2 * kChunk * 4;   // [64] keys, [64] queries: what a row's is times, twice as bf16
constexpr int kPBetaM = kPRowScale + 2 * kChunk * 4;    // [64]: m
constexpr int kPBetaP = kPBetaM + kChunk * 4;           // [64]: p
constexpr int kPrepSmem = kPBetaP + kChunk * 4;
static_assert(kChunk * 256 <= kChunk * kLdA * 4, "queries in A's place");
static_assert(2 * (kPrepSmem + 2048) <= 233472, "two CTAs per SM");

// Offset of eight channels c of row r in rows of 512 bytes of fp32 and of 256 bytes of
// bf16: pieces are exchanged so that neighbouring rows' same piece lie in other banks.
__device__ __forceinline__ uint32_t at512(int r, int c) { return (uint32_t)(r * 512 + ((c ^ (r & 7)) << 5)); }
__device__ __forceinline__ uint32_t at256(int r, int c) { return (uint32_t)(r * 256 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ void mma_16x8x8(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t tf32_rn(float v) {   // to nearest, ties away from zero
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
  return r;
}
// fp32 as two tf32: the upper 11 bits and what they leave, 21 bits in all and fp32's range.
__device__ __forceinline__ void split_tf32(float v, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(v) & 0xFFFFE000u;
  lo = __float_as_uint(v - __uint_as_float(hi));
}

// The 16 x 8 tile of X Y^T at rows x0 of X and y0 of Y, for keys (three products of the
// parts) and queries (two).  A lane's two columns of a step of eight are neighbours: the
// order of the channels in a sum is free.
__device__ __forceinline__ void tile_xy(const uint8_t* smem, int x0, int y0, float (&kk)[4], float (&qk)[4]) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  // rows x0 + g, x0 + g + 8 and y0 + g: the same place in a row's exchanged pieces (x0 and y0 are multiples of eight)
  const uint8_t* X = smem + kPX + (x0 + g) * 512 + 8 * t;
  const uint8_t* Q = smem + kPQ + (x0 + g) * 512 + 8 * t;
  const uint8_t* Y = smem + kPY + (y0 + g) * 512 + 8 * t;
  float lh[4], hl[4], ql[4];   // sums of their own: short chains of products
#pragma unroll
  for (int i = 0; i < 4; ++i) kk[i] = qk[i] = lh[i] = hl[i] = ql[i] = 0.f;
#pragma unroll 8
  for (int c = 0; c < 16; ++c) {
    const int piece = c ^ g;
    const float2 xa = *reinterpret_cast<const float2*>(X + 32 * piece);
    const float2 xb = *reinterpret_cast<const float2*>(X + 32 * piece + 8 * 512);
    const float2 y = *reinterpret_cast<const float2*>(Y + 32 * piece);
    const uint2 qa = *reinterpret_cast<const uint2*>(Q + 32 * piece);
    const uint2 qb = *reinterpret_cast<const uint2*>(Q + 32 * piece + 8 * 512);
    uint32_t xh[4], xl[4], yh[2], yl[2];
    split_tf32(xa.x, xh[0], xl[0]), split_tf32(xb.x, xh[1], xl[1]), split_tf32(xa.y, xh[2], xl[2]), split_tf32(xb.y, xh[3], xl[3]);
    split_tf32(y.x, yh[0], yl[0]), split_tf32(y.y, yh[1], yl[1]);
    const uint32_t q[4] = {qa.x, qb.x, qa.y, qb.y};
    mma_16x8x8(lh, xl, yh);
    mma_16x8x8(hl, xh, yl);
    mma_16x8x8(kk, xh, yh);
    mma_16x8x8(ql, q, yl);
    mma_16x8x8(qk, q, yh);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) kk[i] += lh[i] + hl[i], qk[i] += ql[i];
}

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// 16 x 16 of X Y^T from fp16 parts, X and Y as [2 parts][64][128], queries [64][128]: for two different blocks.
__device__ __forceinline__ void tile_parts(uint32_t sm, int x0, int y0, float (&kk)[2][4], float (&qk)[2][4]) {
  const int lane = threadIdx.x & 31, r = lane & 7;
  const uint32_t X = sm + kPX + (x0 + (lane & 15)) * 256, Y = sm + kPY + (lane >> 4) * kPartHalf + (y0 + r) * 256;
  const uint32_t px = (uint32_t)((r ^ (lane >> 4)) << 4), py = (uint32_t)((r ^ ((lane >> 3) & 1)) << 4);
  float kl[2][4], ql[2][4];   // products with a low part
#pragma unroll
  for (int i = 0; i < 8; ++i) kk[i >> 2][i & 3] = qk[i >> 2][i & 3] = kl[i >> 2][i & 3] = ql[i >> 2][i & 3] = 0.f;
#pragma unroll 4
  for (int c = 0; c < 8; ++c) {
    uint32_t xh[4], xl[4], q[4], y[2][4];   // y: two pieces of the high part, two of the low one
    const uint32_t ax = X + (px ^ (c << 5)), ay = Y + (py ^ (c << 5));
    load_matrices(xh, ax);
    load_matrices(xl, ax + kPartHalf);
    load_matrices(q, ax + (kPQ - kPX));
    load_matrices(y[0], ay);
    load_matrices(y[1], ay + 8 * 256);
#pragma unroll
    for (int e = 0; e < 2; ++e) mma_16x8x16(kl[e], xl, y[e][0], y[e][1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) mma_16x8x16(kk[e], xh, y[e][0], y[e][1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) mma_16x8x16(ql[e], q, y[e][2], y[e][3]);
#pragma unroll
    for (int e = 0; e < 2; ++e) mma_16x8x16(qk[e], q, y[e][0], y[e][1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) mma_16x8x16(kl[e], xh, y[e][2], y[e][3]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) kk[i >> 2][i & 3] += kl[i >> 2][i & 3], qk[i >> 2][i & 3] += ql[i >> 2][i & 3];
}

// A 16 x 8 tile of sign * L R for fp32 matrices in shared memory: L's 16 rows, K columns; R's K
// rows, 8 columns.  Each factor as two tf32, three products.
template <int K>
__device__ __forceinline__ void mul_tile(const float* L, int ldl, const float* R, int ldr, float* out, int ldo, float sign) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  float d[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f}, d2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < K; k += 8) {
    const float l[4] = {L[g * ldl + k + t], L[(g + 8) * ldl + k + t], L[g * ldl + k + t + 4], L[(g + 8) * ldl + k + t + 4]};
    const float r[2] = {R[(k + t) * ldr + g], R[(k + t + 4) * ldr + g]};
    uint32_t lh[4], ll[4], rh[2], rl[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_tf32(l[i], lh[i], ll[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) split_tf32(r[i], rh[i], rl[i]);
    mma_16x8x8(d2, ll, rh);
    mma_16x8x8(d1, lh, rl);
    mma_16x8x8(d, lh, rh);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] += d1[i] + d2[i];
  out[g * ldo + 2 * t] = sign * d[0], out[g * ldo + 2 * t + 1] = sign * d[1];
  out[(g + 8) * ldo + 2 * t] = sign * d[2], out[(g + 8) * ldo + 2 * t + 1] = sign * d[3];
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float max_warp(float v) {  // of values >= 0
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

__device__ __forceinline__ float max_nan(float a, float b) {   // no number if one of them is none
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// First row and number of rows of record number `slot`'s chunk: of the last long sequence with no more chunks before it.
__device__ __forceinline__ bool chunk_rows(const ChunkArgs& p, int slot, int64_t* row0, int* n) {
  int at = 0, end = p.s.index[0].x;
  if (end == 0) return false;
  while (end - at > 1) {
    const int mid = (at + end) >> 1;
    if (p.s.index[1 + mid].z <= slot) at = mid; else end = mid;
  }
  const int4 seq = p.s.index[1 + at];
  const int c = slot - seq.z;
  if (c < 0 || c * kChunk >= seq.y) return false;
  *row0 = seq.x + c * kChunk;
  *n = min(seq.y - c * kChunk, kChunk);
  return true;
}
__device__ __forceinline__ void prefetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__global__ void __launch_bounds__(kPrepThreads, 2) delta_prepare_kernel(const ChunkArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sm = smem_u32(smem);
  const DeltaRows& x = p.x;
  const int h = blockIdx.x % x.heads, hq = h / (x.heads / x.qk_heads);
  const int tid = threadIdx.x, lane = tid & 31, warp = warp_number();
  int64_t row0;
  int n = 0;
  grid_dep_launch();   // the chain's first steps need nothing of this
  if (!chunk_rows(p, blockIdx.x / x.heads, &row0, &n)) return;
  uint8_t* rec = p.records + (int64_t)blockIdx.x * kRecBytes;

  float* tab = reinterpret_cast<float*>(smem + kPTab);
  float* beta = reinterpret_cast<float*>(smem + kPBeta);
  float* misc = reinterpret_cast<float*>(smem + kPMisc);   // per warp: (16) growth; (24) unsafe lanes; (32) largest p; (40) largest |T|
  float* A = reinterpret_cast<float*>(smem + kPA);
  bool bad = false;

  // ---- rows 16 I .. + 15, channels 2 q2 and 2 q2 + 1 of this thread
  const int q2 = tid & 63, I = tid >> 6;
  uint32_t kr[16], qr[16];
  f32x2 a[16];
  {
    const uint16_t* kp = x.k + (row0 + 16 * I) * x.ld_k + hq * kDeltaDim + 2 * q2;
    const uint16_t* qp = x.q + (row0 + 16 * I) * x.ld_q + hq * kDeltaDim + 2 * q2;
    const bool wide = x.gate_dim != 1;
    const float* gp = x.gate + (row0 + 16 * I) * x.ld_gate + (int64_t)h * x.gate_dim + (wide ? 2 * q2 : 0);
    const int left = n - 16 * I;   // rows of the block that are there
    if (left >= 16) {
#pragma unroll
      for (int t = 0; t < 16; ++t, kp += x.ld_k, qp += x.ld_q) {
        kr[t] = __ldg(reinterpret_cast<const uint32_t*>(kp));
        qr[t] = __ldg(reinterpret_cast<const uint32_t*>(qp));
      }
      if (wide) {
#pragma unroll
        for (int t = 0; t < 16; ++t, gp += x.ld_gate) a[t] = __ldg(reinterpret_cast<const float2*>(gp));
      } else {
#pragma unroll
        for (int t = 0; t < 16; ++t, gp += x.ld_gate) a[t].x = a[t].y = __ldg(gp);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        kr[t] = qr[t] = 0u;
        a[t] = make_float2(0.f, 0.f);
        if (t < left) {
          kr[t] = __ldg(reinterpret_cast<const uint32_t*>(kp + t * x.ld_k));
          qr[t] = __ldg(reinterpret_cast<const uint32_t*>(qp + t * x.ld_q));
          a[t].x = __ldg(gp + t * x.ld_gate);
          a[t].y = wide ? __ldg(gp + t * x.ld_gate + 1) : a[t].x;
        }
      }
    }
  }
  {
    // the inputs of the chunk that will take this CTA's place, towards L2: four threads a row
    const uint32_t next = blockIdx.x + (uint32_t)p.resident;
    int64_t row1;
    int n1 = 0;
    if (next < gridDim.x && chunk_rows(p, (int)(next / (uint32_t)x.heads), &row1, &n1) && (tid >> 2) < n1) {
      const int h1 = (int)(next % (uint32_t)x.heads), part = tid & 3;
      const int64_t r = row1 + (tid >> 2);
      const uint16_t* kq = (part & 1) ? x.q + r * x.ld_q : x.k + r * x.ld_k;
      prefetch_line(kq + h1 / (x.heads / x.qk_heads) * kDeltaDim + 64 * (part >> 1));
      if (x.gate_dim != 1) prefetch_line(x.gate + r * x.ld_gate + (int64_t)h1 * kDeltaDim + 32 * part);
    }
  }
  uint32_t* rowmax = reinterpret_cast<uint32_t*>(smem + kPRowMax);
  uint32_t *key_scale = reinterpret_cast<uint32_t*>(smem + kPRowScale), *query_scale = key_scale + kChunk;
  float *beta_m = reinterpret_cast<float*>(smem + kPBetaM), *beta_p = reinterpret_cast<float*>(smem + kPBetaP);
  const float bt = tid < kChunk && tid < n ? __ldg(x.beta + (row0 + tid) * x.ld_beta + h) : 0.f;
  {
    // a row's largest |k| (low half) and |q| (high half) over this warp's 64 channels: lanes hand half of their rows on
    uint32_t m[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const uint32_t ka = kr[t] & 0x7FFF7FFFu, qa = qr[t] & 0x7FFF7FFFu;
      m[t] = __vmaxu2(__byte_perm(ka, qa, 0x5410), __byte_perm(ka, qa, 0x7632));
    }
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) {
      const bool up = lane & (2 * w);
#pragma unroll
      for (int i = 0; i < w; ++i) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, up ? m[i] : m[i + w], 2 * w);
        m[i] = __vmaxu2(up ? m[i + w] : m[i], other);
      }
    }
    m[0] = __vmaxu2(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
    if ((lane & 1) == 0) rowmax[(warp & 1) * kChunk + 16 * I + (lane >> 1)] = m[0];
  }
  __syncthreads();
  if (tid < kChunk) {
    const uint32_t m = __vmaxu2(rowmax[tid], rowmax[kChunk + tid]), kb = m & 0xFFFFu, qb = m >> 16;
    uint32_t ke = kb >> 7, qe = qb >> 7;   // the exponents of the row's key and query
    bad = (kb != 0u && (ke < 27u || ke > 227u)) || (qb != 0u && (qe < 27u || qe > 227u));   // beyond 2^-100 .. 2^100 row by row
    if (kb == 0u || bad) ke = 127u;
    if (qb == 0u || bad) qe = 127u;
    key_scale[tid] = (254u - ke) * (128u * 0x10001u), query_scale[tid] = (254u - qe) * (128u * 0x10001u);
    // of the key's length and beta: A's beta, K P's p and the values' power of two (a beta of 0 leaves nothing of its row,
    // one below 2^-126 has a smaller m)
    const float length = __uint_as_float(ke << 23), bv = bt * length;
    const uint32_t be = bv == 0.f ? 0u : max(1u, (__float_as_uint(bv) >> 23) & 0xFFu);
    const float pv = __uint_as_float(be << 23), pk = pv * length;
    // the power of two of query and scale; of a row without outputs (a zero query or scale) any
    const int se = (int)((__float_as_uint(x.scale) >> 23) & 0xFFu);
    int oe = (int)qe + se - 127;
    if (qb == 0u || x.scale == 0.f) oe = 127;
    bad |= !(fabsf(bv) <= 0x1p60f) || !(pk <= 0x1p60f) || oe < 1 || oe > 254 || se == 255 || (se == 0 && x.scale != 0.f);
    beta[tid] = bv * length;
    beta_p[tid] = pk;
    beta_m[tid] = bv * __uint_as_float((254u - be) << 23);
    float* hd = reinterpret_cast<float*>(rec + kRecHead);
    reinterpret_cast<uint16_t*>(hd + kHdV)[tid] = (uint16_t)(be << 7);
    reinterpret_cast<uint32_t*>(hd)[kHdO + tid] = (uint32_t)oe * (128u * 0x10001u);
    const float mb = max_warp(bad ? 0.f : pk);
    if (lane == 0) misc[32 + warp] = mb;
  }
  const f32x2 one = pack2(1.f, 1.f);
  f32x2 block = one, sum = make_float2(0.f, 0.f);
  float grow = 1.f, amax = 0.f;
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    sum.x += a[t].x, sum.y += a[t].y;
    a[t].x = expf(a[t].x), a[t].y = expf(a[t].y);
    block = mul2(block, a[t]);
    amax = fmaxf(amax, fmaxf(a[t].x, a[t].y));
  }
  if (amax > 1.f) {
#pragma unroll
    for (int t = 0; t < 16; ++t) grow *= fmaxf(1.f, fmaxf(a[t].x, a[t].y));
  }
  const float Bx = block.x, By = block.y;
  bad |= !(amax <= 3.4e38f) || !(Bx <= 3.4e38f) || !(By <= 3.4e38f);   // a decay that is no number makes its product none
  tab[I * kDeltaDim + 2 * q2] = Bx, tab[I * kDeltaDim + 2 * q2 + 1] = By;
  *reinterpret_cast<f32x2*>(smem + kPSum + 4 * (I * kDeltaDim + 2 * q2)) = sum;
  {
    bad |= !(grow <= 3.4e38f);
    const bool unsafe = !(fminf(Bx, By) >= 7.6e-37f) || !(grow <= 1024.f);   // 2^-120, 2^10
    const float mg = max_warp(bad ? 1.f : grow);
    const uint32_t any = __ballot_sync(0xffffffffu, unsafe);
    if (lane == 0) {
      misc[16 + warp] = mg;
      reinterpret_cast<uint32_t*>(misc)[24 + warp] = any;
    }
  }
  // B's upper triangle stays zero
  for (int i = tid; i < kTileHalf / 16; i += kPrepThreads) reinterpret_cast<uint4*>(smem + kPB)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();

  constexpr float mk = 2.f;   // the largest element of a key or a query, as the rows are taken
  const float mb = fmaxf(misc[32], misc[33]);
  float mg = 1.f;
#pragma unroll
  for (int b = 0; b < 4; ++b) mg *= fmaxf(misc[16 + 2 * b], misc[17 + 2 * b]);
  const uint32_t* unsafe_w = reinterpret_cast<const uint32_t*>(misc) + 24;
  // (growth by more than 2^10 would leave the other channels too few bits of the common power of two)
  bad |= !(mg <= 1024.f);
  // powers of two that bring the operands into fp16's range, from bounds: products of decays grow no further than mg
  const float sc_k = pow2_scale(mk * mg, 14);                        // of K D and Q P
  const float sc_kp = pow2_scale(mb * mk * mg, 14);                  // of p K P
  const float sc_b = pow2_scale(mk * mk * mg * 128.f, 14);
#pragma unroll
  for (int t = 0; t < 16; t += 4) {
    const uint4 ks = *reinterpret_cast<const uint4*>(key_scale + 16 * I + t), qs = *reinterpret_cast<const uint4*>(query_scale + 16 * I + t);
    kr[t] = mul_bf16x2(kr[t], ks.x), kr[t + 1] = mul_bf16x2(kr[t + 1], ks.y);
    kr[t + 2] = mul_bf16x2(kr[t + 2], ks.z), kr[t + 3] = mul_bf16x2(kr[t + 3], ks.w);
    qr[t] = mul_bf16x2(qr[t], qs.x), qr[t + 1] = mul_bf16x2(qr[t + 1], qs.y);
    qr[t + 2] = mul_bf16x2(qr[t + 2], qs.z), qr[t + 3] = mul_bf16x2(qr[t + 3], qs.w);
  }

  // ---- decays by channel, forward: K P, Q P, X
  auto block_of = [&](int b) { return *reinterpret_cast<const f32x2*>(tab + b * kDeltaDim + 2 * q2); };
  f32x2 pre = one, post = one;   // the decays of the blocks before and behind
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (b < I) pre = mul2(pre, block_of(b));
    if (b > I) post = mul2(post, block_of(b));
  }
  // c^2 brings a block's product to about one; X carries c, Y its inverse
  auto centre1 = [](float B) {
    const int e = (int)((__float_as_uint(B) >> 23) & 0xFFu) - 127;
    return __uint_as_float((uint32_t)(127 + max(-60, min(60, -(e / 2)))) << 23);
  };
  auto centre = [&](int b) {
    const float2 v = block_of(b);
    return pack2(centre1(v.x), centre1(v.y));
  };
  // image offsets of channel pair q2 in rows of 128 bytes, 64 channels a block
  const uint32_t img = (uint32_t)((q2 >> 5) * kTileHalf + (q2 & 31) * 4);
  const uint32_t piece = (uint32_t)(q2 >> 2), in_piece = (uint32_t)(q2 & 3) * 4;
  {
    const f32x2 c = centre(I), pre_k = mul2(pre, pack2(sc_kp, sc_kp)), pre_q = mul2(pre, pack2(sc_k, sc_k));
    f32x2 l = one;
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const int r = 16 * I + t;
      l = mul2(l, a[t]);
      const f32x2 k = bf16x2_to_f32x2(kr[t]), ql = mul2(bf16x2_to_f32x2(qr[t]), l), w = mul2(l, c);
      uint32_t hi2, lo2;
      const uint32_t o = swz128(img + r * 128);
      const float b = beta_p[r];
      split_f16(mul2(mul2(k, pack2(b, b)), mul2(l, pre_k)), hi2, lo2);
      *reinterpret_cast<uint32_t*>(rec + kRecKp + o) = hi2;
      *reinterpret_cast<uint32_t*>(rec + kRecKp + kTileBytes + o) = lo2;
      const float2 qp = mul2(ql, pre_q), xq = mul2(ql, c), wf = w;
      *reinterpret_cast<uint32_t*>(rec + kRecQp + o) = f16x2(qp.x, qp.y);
      const uint32_t s = at512(r, piece) + 2 * in_piece;
      *reinterpret_cast<f32x2*>(smem + kPX + s) = mul2(k, w);
      *reinterpret_cast<uint2*>(smem + kPQ + s) = make_uint2(tf32_rn(xq.x), tf32_rn(xq.y));
      // Y of the block itself: k / (L c); no number where the block is not safe, and not used there
      *reinterpret_cast<f32x2*>(smem + kPY + s) = mul2(k, pack2(reciprocal(wf.x), reciprocal(wf.y)));
    }
    if (I == 3) {
      // the chunk's decay from the sum of the logarithms: the state is multiplied by it chunk after chunk, and a product
      // of 64 rounded factors a chunk costs a slow channel 1e-6 in a thousand rows
      f32x2 all = sum;
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        const f32x2 g = *reinterpret_cast<const f32x2*>(smem + kPSum + 4 * (b * kDeltaDim + 2 * q2));
        all.x += g.x, all.y += g.y;
      }
      *reinterpret_cast<f32x2*>(rec + kRecHead + 4 * (kHdP + 2 * q2)) = make_float2(expf(all.x), expf(all.y));
    }
  }
  // ---- backward: K D
  {
    f32x2 l = mul2(post, pack2(sc_k, sc_k));
#pragma unroll
    for (int t = 15; t >= 0; --t) {
      uint32_t hi2, lo2;
      const uint32_t o = swz128(img + (16 * I + t) * 128);
      split_f16(mul2(bf16x2_to_f32x2(kr[t]), l), hi2, lo2);
      *reinterpret_cast<uint32_t*>(rec + kRecKd + o) = hi2;
      *reinterpret_cast<uint32_t*>(rec + kRecKd + kTileBytes + o) = lo2;
      l = mul2(l, a[t]);
    }
  }
  __syncthreads();

  // ---- A and B within the blocks
  auto put = [&](int i, int j, float kk, float qk) {
    if (j < i) A[i * kLdA + j] = kk * beta[i];
    if (j <= i) *reinterpret_cast<__half*>(smem + kPB + swz128((uint32_t)(i * 128 + j * 2))) = __float2half_rn(qk * sc_b);
  };
  // a tile's lane has two neighbours of rows g and g + 8; above the diagonal there are zeros
  auto put_tile = [&](int i0, int j0, const float (&kk)[4], const float (&qk)[4]) {
    const int j = j0 + 2 * (lane & 3);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = i0 + (lane >> 2) + 8 * e;
      const float b = beta[i];
      *reinterpret_cast<float2*>(A + i * kLdA + j) = make_float2(j < i ? kk[2 * e] * b : 0.f, j + 1 < i ? kk[2 * e + 1] * b : 0.f);
      *reinterpret_cast<uint32_t*>(smem + kPB + swz128((uint32_t)(i * 128 + j * 2))) =
          f16x2(j <= i ? qk[2 * e] * sc_b : 0.f, j + 1 <= i ? qk[2 * e + 1] * sc_b : 0.f);
    }
  };
  const int D = warp >> 1;   // this warp's diagonal block
  const bool safe = (unsafe_w[2 * D] | unsafe_w[2 * D + 1]) == 0u;
  float dk[4], dq[4];
  if (safe) tile_xy(smem, 16 * D, 16 * D + 8 * (warp & 1), dk, dq);
  __syncthreads();
  // (now that nothing reads the queries) A and B within the blocks, and zeros right of A's diagonal blocks
  {
    for (int i = tid; i < 6 * 64; i += kPrepThreads) {
      const int blk = i >> 6, r = (i >> 2) & 15, br = blk < 3 ? 0 : blk < 5 ? 1 : 2, bc = blk < 3 ? blk + 1 : blk < 5 ? blk - 1 : 3;
      *reinterpret_cast<float4*>(A + (16 * br + r) * kLdA + 16 * bc + 4 * (i & 3)) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (safe) {
      put_tile(16 * D, 16 * D + 8 * (warp & 1), dk, dq);
    } else {
      // rows that are not there stay zero
      *reinterpret_cast<float4*>(A + (16 * D + ((tid & 63) >> 2)) * kLdA + 16 * D + 4 * (tid & 3)) = make_float4(0.f, 0.f, 0.f, 0.f);
      asm volatile("bar.sync %0, 64;" ::"r"(1 + D) : "memory");
      // decays that leave fp32's range within 16 rows: pair by pair, four channels a lane
      for (int j = 16 * D + (warp & 1); j < min(16 * D + 16, n); j += 2) {
        const uint2 kj = __ldg(reinterpret_cast<const uint2*>(x.k + (row0 + j) * x.ld_k + hq * kDeltaDim) + lane);
        float4 y = bf16x4_to_float4(kj);
        const float by = __uint_as_float(key_scale[j] & 0xFFFF0000u);
        y.x *= by, y.y *= by, y.z *= by, y.w *= by;
        for (int i = j; i < min(16 * D + 16, n); ++i) {
          if (i > j) {
            float4 g;
            if (x.gate_dim == 1) {
              g.x = g.y = g.z = g.w = __ldg(x.gate + (row0 + i) * x.ld_gate + h);
            } else {
              g = __ldg(reinterpret_cast<const float4*>(x.gate + (row0 + i) * x.ld_gate + (int64_t)h * kDeltaDim) + lane);
            }
            y.x *= expf(g.x), y.y *= expf(g.y), y.z *= expf(g.z), y.w *= expf(g.w);
          }
          const float4 ki = bf16x4_to_float4(__ldg(reinterpret_cast<const uint2*>(x.k + (row0 + i) * x.ld_k + hq * kDeltaDim) + lane));
          const float4 qi = bf16x4_to_float4(__ldg(reinterpret_cast<const uint2*>(x.q + (row0 + i) * x.ld_q + hq * kDeltaDim) + lane));
          float kk = fmaf(y.w, ki.w, fmaf(y.z, ki.z, fmaf(y.y, ki.y, y.x * ki.x)));
          float qk = fmaf(y.w, qi.w, fmaf(y.z, qi.z, fmaf(y.y, qi.y, y.x * qi.x)));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            kk += __shfl_xor_sync(0xffffffffu, kk, o);
            qk += __shfl_xor_sync(0xffffffffu, qk, o);
          }
          if (lane == 0) put(i, j, kk * __uint_as_float(key_scale[i] & 0xFFFF0000u), qk * __uint_as_float(query_scale[i] & 0xFFFF0000u));
        }
      }
    }
  }
  // ---- between the blocks.  Rows 32..63 meet columns 0..31 at the start of row 32, rows 48..63 meet 32..47 at that of
  // row 48, rows 16..31 meet 0..15 at that of row 16: decays up to there in Y, from there in X
  // Y at rows y0 .. + 15: k times the decay to the block's end, times l
  auto put_y = [&](int y0, f32x2 l) {
    l = mul2(l, pack2(sc_k, sc_k));
#pragma unroll
    for (int t = 15; t >= 0; --t) {
      uint32_t hi2, lo2;
      split_f16(mul2(bf16x2_to_f32x2(kr[t]), l), hi2, lo2);
      uint8_t* to = smem + kPY + at256(y0 + t, piece) + in_piece;
      *reinterpret_cast<uint32_t*>(to) = hi2;
      *reinterpret_cast<uint32_t*>(to + kPartHalf) = lo2;
      l = mul2(l, a[t]);
    }
  };
  // X at rows x0 .. + 15: k and q times l and the decays from the block's start
  auto put_x = [&](int x0, f32x2 l) {
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      l = mul2(l, a[t]);
      uint32_t hi2, lo2;
      const f32x2 ls = mul2(l, pack2(sc_k, sc_k));
      split_f16(mul2(bf16x2_to_f32x2(kr[t]), ls), hi2, lo2);
      const f32x2 xq = mul2(bf16x2_to_f32x2(qr[t]), ls);
      const uint32_t o = at256(x0 + t, piece) + in_piece;
      *reinterpret_cast<uint32_t*>(smem + kPX + o) = hi2;
      *reinterpret_cast<uint32_t*>(smem + kPX + kPartHalf + o) = lo2;
      *reinterpret_cast<uint32_t*>(smem + kPQ + o) = f16x2(xq.x, xq.y);
    }
  };
  // two pieces of work for every thread; X's free rows 0..15 hold rows 48..63 once more
#pragma unroll 1
  for (int e = 0; e < (I == 3 ? 2 : I > 0); ++e) put_x(e ? 0 : 16 * I, e ? block_of(2) : one);
#pragma unroll 1
  for (int e = 0; e < (I == 0 ? 2 : I < 3); ++e) put_y(e ? 48 : 16 * I, I == 0 && e == 0 ? block_of(1) : one);
  __syncthreads();
  if (warp < 6) {
    // blocks (1, 0), (2, 0), (2, 1), (3, 0), (3, 1), (3, 2)
    const int bi = warp == 0 ? 1 : warp < 3 ? 2 : 3, bj = warp == 0 ? 0 : warp < 3 ? warp - 1 : warp - 3;
    float kk[2][4], qk[2][4];
    tile_parts(sm, warp == 3 || warp == 4 ? 0 : 16 * bi, warp == 0 ? 48 : 16 * bj, kk, qk);
    const float ik = pow2_inverse(sc_k);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int i = 0; i < 4; ++i) kk[e][i] = kk[e][i] * ik * ik, qk[e][i] = qk[e][i] * ik * ik;
      put_tile(16 * bi, 16 * bj + 8 * e, kk[e], qk[e]);
    }
  }
  // meanwhile the inverses of I + A's diagonal blocks, in their place, by substitution: a thread a column
  if (warp >= 6) {
    const int j = tid & 15;
    float* D = A + (tid & 48) * (kLdA + 1);   // (threads 192..255)
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 r = *reinterpret_cast<const float4*>(D + i * kLdA + m);
        s0 = fmaf(r.x, t[m], s0);
        if (m + 1 < i) s1 = fmaf(r.y, t[m + 1], s1);
        if (m + 2 < i) s0 = fmaf(r.z, t[m + 2], s0);
        if (m + 3 < i) s1 = fmaf(r.w, t[m + 3], s1);
      }
      t[i] = i < j ? 0.f : i == j ? 1.f : -(s0 + s1);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) D[i * kLdA + j] = t[i];
  }
  __syncthreads();
  // ---- (I + A)^-1, in A's place: from its diagonal blocks twice [[T1, 0], [-T2 A21 T1, T2]], of 16 and of 32 rows
  float* tmp = reinterpret_cast<float*>(smem + kPX);   // [32][36]
  constexpr int kLdT = 36;
  if (warp < 4) {
    const int d = 32 * (warp >> 1), cc = 8 * (warp & 1);
    mul_tile<16>(A + (d + 16) * kLdA + d, kLdA, A + d * kLdA + d + cc, kLdA, tmp + (d >> 1) * kLdT + cc, kLdT, 1.f);
  } else {
#pragma unroll
    for (int q = tid - 128; q < kTileHalf / 16; q += 128)
      reinterpret_cast<uint4*>(rec + kRecB)[q] = reinterpret_cast<const uint4*>(smem + kPB)[q];
  }
  __syncthreads();
  if (warp < 4) {
    const int d = 32 * (warp >> 1), cc = 8 * (warp & 1);
    mul_tile<16>(A + (d + 16) * (kLdA + 1), kLdA, tmp + (d >> 1) * kLdT + cc, kLdT, A + (d + 16) * kLdA + d + cc, kLdA, -1.f);
  }
  __syncthreads();
  {
    const int r = 16 * (warp >> 2), cc = 8 * (warp & 3);
    mul_tile<32>(A + (32 + r) * kLdA, kLdA, A + cc, kLdA, tmp + r * kLdT + cc, kLdT, 1.f);
    __syncthreads();
    mul_tile<32>(A + (32 + r) * kLdA + 32, kLdA, tmp + cc, kLdT, A + (32 + r) * kLdA + cc, kLdA, -1.f);
  }
  __syncthreads();
  // ---- T = (I + A)^-1 diag(m) in two parts: a thread 16 columns of a row
  {
    const int i = tid >> 2, j0 = 16 * (tid & 3);
    float t[16], m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const float4 r = *reinterpret_cast<const float4*>(A + i * kLdA + j0 + j);
      const float4 bj = *reinterpret_cast<const float4*>(beta_m + j0 + j);
      t[j] = r.x * bj.x, t[j + 1] = r.y * bj.y, t[j + 2] = r.z * bj.z, t[j + 3] = r.w * bj.w;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max_nan(m, fabsf(t[j]));
    bad |= !(m * kScaleT <= 32768.f);   // no number, or beta |k|^2 much larger than one: the rows go one by one
    m = max_warp(bad ? 0.f : m);
    if (lane == 0) misc[40 + warp] = m;
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) split_f16(mul2(pack2(t[2 * j], t[2 * j + 1]), pack2(kScaleT, kScaleT)), hi[j], lo[j]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t o = swz128((uint32_t)(i * 128 + 2 * j0 + 16 * j));
      *reinterpret_cast<uint4*>(rec + kRecT + o) = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
      *reinterpret_cast<uint4*>(rec + kRecT + kTileHalf + o) = make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
    }
  }
  const int any = __syncthreads_or(bad);
  if (tid == 0) {
    float mt = misc[40];
#pragma unroll
    for (int w = 1; w < 8; ++w) mt = fmaxf(mt, misc[40 + w]);
    float* hd = reinterpret_cast<float*>(rec + kRecHead);
    reinterpret_cast<int*>(hd)[kHdBad] = any;
    hd[kHdInvKp] = pow2_inverse(sc_kp), hd[kHdInvB] = pow2_inverse(sc_b), hd[kHdInvK] = pow2_inverse(sc_k);
    // sums of a row's or a column's magnitudes, from above
    hd[kHdSumKp] = 128.f * mb * mk * mg, hd[kHdSumT] = 64.f * mt, hd[kHdSumKd] = 64.f * mk * mg;
  }
}

// ---------------------------------------------------------------- chain
// Warps 0..7 hold the state: row v = 32 (w % 4) + lane of it, keys 64 (w / 4) ..
// + 63, and turn each product into the next one's operand; warp 8 issues the MMAs,
// warp 9 copies the operands, two chunks deep, warp 10 stores the outputs.  All
// products are transposed, with the 128 values on the tensor core's rows:
//   R^T [v][t] = (V^T - S (K P)^T) diag(p)   A = S in two fp16 parts from TMEM, times p K P's two (three products)
//   U^T = R^T T^T                  A = R in two parts
//   dS  = U^T (K D)                A = U in two parts; K D as it lies (MN-major)
//   out^T = S (Q P)^T + U^T B^T    times a power of two a row; one product each: the high parts' 11 bits, rounded, are more than bf16 keeps
// The parts of a row of S, R or U are times a power of two, so that they keep 21 bits of
// its largest element whatever its size: of S from the row's largest element itself, which the
// two warps of a row exchange before they split it (a bound carried from chunk to chunk would
// not see a state decay, and its parts would be lost; 5 us of 2,048 rows); of R and U from bounds made of maxima
// that they exchange one step later, which may be loose: fp16's exponents leave room for 2^18.
// Where something in a chunk is no finite number, or leaves the powers' range, its rows
// go one by one: the zeros of T and B would carry a NaN to the rows before it.
// What bounds it: a chain of latencies, 7,300 to 7,600 cycles a chunk, of which the tensor pipe
// works 2,200: three products that wait for each other, their way through TMEM, and the
// conversions between them (S 660 cycles and 370 for its largest element, R 740, U 450, the update 940).  Outputs are
// converted while R is made, the next values read while the update is.
constexpr int kChainThreads = 12 * 32;   // three warpgroups: two of state warps, one of the rest (its last warp has no work)
// Of the block's 384 x 168 registers the state warps take 200 a thread and leave 104 to the others: with 168 they spill.
constexpr int kHelperRegs = 104, kStateRegs = 200;
constexpr int kMmaWarp = 8, kCopyWarp = 9, kStoreWarp = 10;
constexpr int kColS = 0;       // keys 64 h ..: high parts in columns 64 h .. + 31, low parts behind them
constexpr int kColAcc = 128;   // R, then U
constexpr int kColParts = 192; // R's, then U's parts: high 32 columns, low 32
constexpr int kColDs = 256;
constexpr int kColO1 = 384, kColO2 = 448;
constexpr int kRowBytes = kDeltaDim * 2;                // a row of values or outputs
constexpr int kCOffPart2 = 2 * kPart1;                  // one buffer: its products come last in a chunk
constexpr int kCOffV = kCOffPart2 + kPart2;
constexpr int kCOffOut = kCOffV + 2 * kChunk * kRowBytes;
constexpr int kCOffHead = kCOffOut + kChunk * kRowBytes;
constexpr int kCHead = (kHeadBytes + 127) & ~127;       // bytes of a head's buffer
constexpr int kCOffX = kCOffHead + 2 * kCHead;             // exchanged maxima [2 parities][3 kinds][2 halves][128]
constexpr int kCOffRow = kCOffX + 2 * 3 * 2 * 128 * 4;  // [2][64]: what the rows' outputs are times
constexpr int kCOffRowV = kCOffRow + 2 * kChunk * 4;    // [2][64] bf16: what the rows' values are times
constexpr int kCOffBars = kCOffRowV + 2 * kHeadVBytes;
constexpr int kCNumBars = 21;
constexpr int kCOffMisc = kCOffBars + kCNumBars * 8;
constexpr int kChainSmem = 1024 + kCOffMisc + 40;
static_assert(kChainSmem <= 232448 && kPart1 % 1024 == 0 && kPart2 % 1024 == 0 && kHeadBytes <= kCHead && kHeadBytes <= kRecBytes - kRecHead, "shared memory");

// The two warps that share 32 value rows of the state.
__device__ __forceinline__ void bar_pair(int pair) { asm volatile("bar.sync %0, 64;" ::"r"(2 + pair) : "memory"); }
__device__ __forceinline__ void bar_state() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool bar_state_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, 1, 256, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint32_t max_abs_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n .reg .b32 t;\n abs.f16x2 t, %2;\n max.f16x2 %0, %1, t;\n}\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float max_of_f16x2(uint32_t v) {
  const float2 m = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return fmaxf(m.x, m.y);
}

__global__ void __launch_bounds__(kChainThreads, 1) delta_chain_kernel(const ChunkArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sm = smem_u32(smem);
  const DeltaRows& x = p.x;
  const int h = blockIdx.x % x.heads, at = blockIdx.x / x.heads, hq = h / (x.heads / x.qk_heads);
  const int warp = warp_number(), lane = threadIdx.x & 31;
  // the list is of the kernel before the one that prepares the operands: complete when that one started
  const int4 seq = at < __ldcg(&p.s.index[0].x) ? __ldcg(p.s.index + 1 + at) : make_int4(0, 0, 0, 0);
  const int64_t row0 = seq.x;
  const int n = seq.y, slot = seq.z, b = seq.w, chunks = (n + kChunk - 1) / kChunk;
  if (n == 0 || slot + chunks > p.chunks) {   // (starts that do not ascend can make more chunks than there is room for)
    grid_dep_wait();
    return;
  }
  const uint8_t* rec = p.records + ((int64_t)slot * x.heads + h) * kRecBytes;
  const int64_t rec_step = (int64_t)x.heads * kRecBytes;

  const uint32_t bars = sm + kCOffBars;
  auto full = [&](int s) { return bars + 8u * s; };          // first part and head
  auto empty = [&](int s) { return bars + 16u + 8u * s; };
  const uint32_t full2 = bars + 32, empty2 = bars + 40, b_s = bars + 48, b_r = bars + 56, b_rp = bars + 64, b_u = bars + 72,
                 b_up = bars + 80, b_ds = bars + 88, b_o = bars + 96, b_of = bars + 104, out_full = bars + 112,
                 out_free = bars + 120, drain = bars + 128;
  auto full_v = [&](int s) { return bars + 136u + 8u * s; };
  auto empty_v = [&](int s) { return bars + 152u + 8u * s; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kCOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kCOffMisc + 4);
  volatile int* by_rows = reinterpret_cast<volatile int*>(smem + kCOffMisc + 8);    // [2]: this chunk goes row by row
  volatile int* out_job = reinterpret_cast<volatile int*>(smem + kCOffMisc + 16);   // chunk and rows to store; 0 rows: no more
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 9);
      mbar_init(full_v(s), 1);
      mbar_init(empty_v(s), 8);
    }
    for (uint32_t a : {full2, empty2, b_r, b_u, b_ds, b_o, out_free, drain}) mbar_init(a, 1);
    for (uint32_t a : {b_s, b_rp, b_up, b_of, out_full}) mbar_init(a, 8);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kHelperRegs));
    if (warp == kCopyWarp) {
      // the values one chunk further ahead than the operands: they are looked at during the chunk before theirs
      bool ok = true;
      int issued_v = 0, issued = 0, issued2 = 0;
      auto copy_v = [&](int c) {
        const int s = c & 1, rows = min(kChunk, n - c * kChunk);
        if (c >= 2 && !mbar_wait_warp(empty_v(s), ((c >> 1) & 1) ^ 1, abort_flag, p.s.status)) return false;
        if (elect_one()) {
          mbar_arrive_expect_tx(full_v(s), rows * kRowBytes + kHeadVBytes);
          if (c > 0) bulk_load(sm + kCOffRowV + s * kHeadVBytes, rec + c * rec_step + kRecHead + 4 * kHdV, kHeadVBytes, full_v(s));
        }
        __syncwarp();
        for (int t = lane; t < rows; t += 32)
          bulk_load(sm + kCOffV + (s * kChunk + t) * kRowBytes, x.v + (row0 + c * kChunk + t) * x.ld_v + (int64_t)h * kDeltaDim,
                    kRowBytes, full_v(s));
        __syncwarp();
        ++issued_v;
        return true;
      };
      ok = copy_v(0);
      grid_dep_wait();   // the records
      if (elect_one()) bulk_load(sm + kCOffRowV, rec + kRecHead + 4 * kHdV, kHeadVBytes, full_v(0));
      __syncwarp();
      for (int c = 0; c < chunks && ok; ++c) {
        const int s = c & 1;
        const uint8_t* src = rec + c * rec_step;
        if (c >= 2) ok = mbar_wait_warp(empty(s), ((c >> 1) & 1) ^ 1, abort_flag, p.s.status);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(full(s), kPart1 + kHeadBytes);
          for (int i = 0; i < 4; ++i) bulk_load(sm + s * kPart1 + i * (kPart1 / 4), src + i * (kPart1 / 4), kPart1 / 4, full(s));
          bulk_load(sm + kCOffHead + s * kCHead, src + kRecHead, kHeadBytes, full(s));
        }
        __syncwarp();
        ++issued;
        if (c + 1 < chunks) ok = copy_v(c + 1);
        if (ok && c >= 1) ok = mbar_wait_warp(empty2, (c - 1) & 1, abort_flag, p.s.status);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(full2, kPart2);
          for (int i = 0; i < 2; ++i) bulk_load(sm + kCOffPart2 + i * (kPart2 / 2), src + kRecB + i * (kPart2 / 2), kPart2 / 2, full2);
        }
        __syncwarp();
        ++issued2;
      }
      // no copy is in flight at the exit, also after another role gave up
      for (int c = max(0, issued_v - 2); c < issued_v; ++c) mbar_wait_drain(full_v(c & 1), (c >> 1) & 1, 10000000ull);
      for (int c = max(0, issued - 2); c < issued; ++c) mbar_wait_drain(full(c & 1), (c >> 1) & 1, 10000000ull);
      if (issued2 > 0) mbar_wait_drain(full2, (issued2 - 1) & 1, 10000000ull);
    } else if (warp == kStoreWarp) {
      for (uint32_t j = 0;; ++j) {
        if (!mbar_wait_warp(out_full, j & 1, abort_flag, p.s.status)) break;
        const int c = __shfl_sync(0xffffffffu, out_job[0], 0), rows = __shfl_sync(0xffffffffu, out_job[1], 0);
        if (rows == 0) break;
        // two rows at a time, 16 bytes a lane (bulk copies would stand in line behind the next operands')
        const uint4* src = reinterpret_cast<const uint4*>(smem + kCOffOut) + lane;
        uint16_t* dst = p.out + ((row0 + c * kChunk + (lane >> 4)) * x.heads + h) * kDeltaDim + 8 * (lane & 15);
        const uint32_t* by = reinterpret_cast<const uint32_t*>(smem + kCOffRow) + (c & 1) * kChunk + (lane >> 4);
#pragma unroll 8
        for (int t = 0; t < rows; t += 2)
          if (t + (lane >> 4) < rows) {
            const uint4 o = src[16 * t];
            const uint32_t f = by[t];
            *reinterpret_cast<uint4*>(dst + (int64_t)t * x.heads * kDeltaDim) =
                make_uint4(mul_bf16x2(o.x, f), mul_bf16x2(o.y, f), mul_bf16x2(o.z, f), mul_bf16x2(o.w, f));
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(out_free);
      }
    } else if (warp == kMmaWarp) {
      constexpr uint32_t kIdesc64 = make_idesc(kFmtF16, kFmtF16, 0, 0, 128, kChunk);
      constexpr uint32_t kIdescDs = make_idesc(kFmtF16, kFmtF16, 0, 1, 128, kDeltaDim);
      const uint64_t kdesc = smem_desc(sm, 16, 1024, kLayoutSw128);                  // K-major tiles
      const uint64_t bdesc = smem_desc(sm + kCOffPart2, 16, 1024, kLayoutSw128);     // B
      const uint64_t ndesc = smem_desc(sm + kCOffPart2 + kTileHalf, kTileHalf, 1024, kLayoutSw128);  // K D: 64 keys a block
      const uint32_t k_hi = (uint32_t)(kdesc >> 32), n_hi = (uint32_t)(ndesc >> 32);
      uint32_t f = 0;   // chunks that took the tensor core
      for (int c = 0; c < chunks; ++c) {
        const int s = c & 1;
        const uint32_t k0 = (uint32_t)kdesc + s * (kPart1 / 16), b0 = (uint32_t)bdesc, n0 = (uint32_t)ndesc;
        if (!mbar_wait_warp(full(s), (c >> 1) & 1, abort_flag, p.s.status)) break;
        if (!mbar_wait_warp(b_s, c & 1, abort_flag, p.s.status)) break;
        tc_fence_after();
        auto product_s = [&](uint32_t d, int part, int tile, bool more) {   // A: the state's part, 128 keys
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_bf16_tmem_a(tmem + d, tmem + kColS + 64 * (ks >> 2) + 32 * part + 8 * (ks & 3),
                            desc64(k0 + (tile + (ks >> 2) * kTileHalf) / 16 + 2 * (ks & 3), k_hi), kIdesc64, more || ks ? 1u : 0u);
        };
        auto product_t = [&](uint32_t d, int part, uint32_t tile, bool more) {   // A: R's or U's part, 64 rows
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_bf16_tmem_a(tmem + d, tmem + kColParts + 32 * part + 8 * ks, desc64(tile + 2 * ks, k_hi), kIdesc64,
                            more || ks ? 1u : 0u);
        };
        if (elect_one()) {
          product_s(kColAcc, 1, kRecKp, false);
          product_s(kColAcc, 0, kRecKp + kTileBytes, true);
          product_s(kColAcc, 0, kRecKp, true);
          mma_commit(b_r);
        }
        __syncwarp();
        if (!mbar_wait_warp(b_rp, c & 1, abort_flag, p.s.status)) break;
        if (__any_sync(0xffffffffu, by_rows[s] != 0)) {
          // nothing of this chunk comes from the tensor core: its buffers go back
          if (!mbar_wait_warp(full2, c & 1, abort_flag, p.s.status)) break;
          if (elect_one()) {
            mbar_arrive(empty(s));
            mbar_arrive(empty2);
          }
          __syncwarp();
          continue;
        }
        tc_fence_after();
        if (elect_one()) {
          product_t(kColAcc, 1, k0 + kRecT / 16, false);
          product_t(kColAcc, 0, k0 + (kRecT + kTileHalf) / 16, true);
          product_t(kColAcc, 0, k0 + kRecT / 16, true);
          mma_commit(b_u);
        }
        __syncwarp();
        if (!mbar_wait_warp(full2, c & 1, abort_flag, p.s.status)) break;
        if (!mbar_wait_warp(b_up, f & 1, abort_flag, p.s.status)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < 3; ++q)   // low x high, high x low, high x high
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_bf16_tmem_a(tmem + kColDs, tmem + kColParts + (q == 0 ? 32 : 0) + 8 * ks,
                              desc64(n0 + (q == 1 ? kTileBytes / 16 : 0) + ks * (16 * 128 / 16), n_hi), kIdescDs, q | ks ? 1u : 0u);
          mma_commit(b_ds);
        }
        __syncwarp();
        // the outputs' products run while the state is updated
        if (f > 0 && !mbar_wait_warp(b_of, (f - 1) & 1, abort_flag, p.s.status)) break;
        tc_fence_after();
        if (elect_one()) {
          product_s(kColO1, 0, kRecQp, false);
          product_t(kColO2, 0, b0, false);
          mma_commit(b_o);
          mma_commit(empty(s));
          mma_commit(empty2);
        }
        __syncwarp();
        ++f;
      }
      // every MMA completes before TMEM is released
      if (elect_one()) {
        mma_commit(drain);
        mbar_wait_drain(drain, 0, 10000000ull);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
    // ------------------------------------------------ state warps
    grid_dep_wait();
    // A wait that gave up leaves the loop running without waits (they return at
    // once then): the warps meet at named barriers and none may be missing there.
    const int half = warp >> 2, v = 32 * (warp & 3) + lane, tid = threadIdx.x;
    const uint32_t quad = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    float* ex = reinterpret_cast<float*>(smem + kCOffX);
    auto xchg = [&](int parity, int kind, int hf) -> float& { return ex[((parity * 3 + kind) * 2 + hf) * 128 + v]; };
    enum { kMaxS, kMaxV, kMaxR };
    float S[64];
    {
      const float* in = state_in(p.s, b, h);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 t = in ? *reinterpret_cast<const float4*>(in + v * kDeltaDim + 64 * half + 4 * i)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        S[4 * i] = t.x, S[4 * i + 1] = t.y, S[4 * i + 2] = t.z, S[4 * i + 3] = t.w;
      }
    }
    float sc_s = 1.f;     // what the row of the state in registers is times
    float bound_s = 0.f;  // the row's largest element
    auto measure = [&](int parity) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 64; i += 2) m = fmaxf(fmaxf(m, fabsf(S[i])), fabsf(S[i + 1]));
      xchg(parity, kMaxS, half) = m;
      bar_pair(warp & 3);
      m = fmaxf(xchg(parity, kMaxS, 0), xchg(parity, kMaxS, 1));
      bound_s = m * pow2_inverse(sc_s);
      // another power of two only where the largest element has left [2^4, 2^15): 21 bits of it down to 2^4
      const bool moved = m > 0.f && !(m >= 16.f && m < 32768.f);
      if (__any_sync(0xffffffffu, moved)) {
        const float by = moved ? fminf(pow2_scale(bound_s, 12) * pow2_inverse(sc_s), 0x1p126f) : 1.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] *= by;
        sc_s *= by;
      }
    };
    uint32_t f = 0;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      mbar_wait_warp(bar, parity, abort_flag, p.s.status);
      tc_fence_after();
    };
    auto arrive = [&](uint32_t bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };

    // a chunk's values of this lane, rows 32 half .. + 31, two a register, and whether it goes row by row: read while
    // the chunk before waits for its products
    uint32_t vr[16];
    auto read_v = [&](int c) {
      const int s = c & 1, left = min(kChunk, n - c * kChunk) - 32 * half;
      wait(full_v(s), (c >> 1) & 1);
      const uint32_t* by = reinterpret_cast<const uint32_t*>(smem + kCOffRowV + s * kHeadVBytes) + 16 * half;
      const uint16_t* vp = reinterpret_cast<const uint16_t*>(smem + kCOffV) + (s * kChunk + 32 * half) * kDeltaDim + v;
#pragma unroll
      for (int t = 0; t < 16; ++t)
        vr[t] = mul_bf16x2(__byte_perm((uint32_t)vp[2 * t * kDeltaDim], (uint32_t)vp[(2 * t + 1) * kDeltaDim], 0x5410), by[t]);
      if (left < 32) {   // rows that are not there
#pragma unroll
        for (int t = 0; t < 16; ++t) vr[t] = 2 * t >= left ? 0u : 2 * t + 1 >= left ? vr[t] & 0xFFFFu : vr[t];
      }
    };
    auto vote = [&](int c) {
      const int s = c & 1;
      uint32_t m = 0;
#pragma unroll
      for (int t = 0; t < 16; ++t) m = __vmaxu2(m, vr[t] & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16);
      xchg(s, kMaxV, half) = __uint_as_float(m << 16);
      __syncwarp();   // all lanes have read what the next copy overwrites
      if (lane == 0) mbar_arrive(empty_v(s));
      return bar_state_or(m >= 0x7F80u);
    };
    bool rowwise = false;   // a value of the chunk is no number, or not in bf16's range as it is taken
    if (chunks > 0) {
      read_v(0);
      rowwise = vote(0);
    }

    // the outputs of the last chunk that took the tensor core, behind the next one's first operand
    int out_rows = 0, out_c = 0;
    float out_f1 = 0.f, out_f2 = 0.f;
    const float scale = x.scale == 0.f ? 0.f : __uint_as_float((__float_as_uint(x.scale) & 0x807FFFFFu) | 0x3F800000u);
    uint32_t jobs = 0;
    auto put_out = [&](int q) {   // in two halves, each where the warps would wait
      if (out_rows == 0) return;
      uint32_t o1[16], o2[16];
      tmem_ld16(quad + kColO1 + 32 * half + 16 * q, o1);
      tmem_ld16(quad + kColO2 + 32 * half + 16 * q, o2);
      if (q == 0 && jobs > 0) wait(out_free, (jobs - 1) & 1);
      tmem_ld_wait();
      if (q == 1) arrive(b_of);
      uint16_t* op = reinterpret_cast<uint16_t*>(smem + kCOffOut) + (32 * half + 16 * q) * kDeltaDim + v;
#pragma unroll
      for (int t = 0; t < 16; t += 2) {
        const uint32_t o = bf16x2(fmaf(out_f1, __uint_as_float(o1[t]), out_f2 * __uint_as_float(o2[t])),
                                  fmaf(out_f1, __uint_as_float(o1[t + 1]), out_f2 * __uint_as_float(o2[t + 1])));
        op[t * kDeltaDim] = (uint16_t)o;
        op[(t + 1) * kDeltaDim] = (uint16_t)(o >> 16);
      }
      if (q == 0) return;
      if (tid == 0) out_job[0] = out_c, out_job[1] = out_rows;
      __syncwarp();
      if (lane == 0) mbar_arrive(out_full);
      ++jobs;
      out_rows = 0;
    };

    for (int c = 0; c < chunks; ++c) {
      const int s = c & 1;
      const int rows = min(kChunk, n - c * kChunk);
      const float* hd = reinterpret_cast<const float*>(smem + kCOffHead + s * kCHead);
      // ---- the state's parts; the outputs' products, which read the last ones, are through
      measure(s);
      if (out_rows > 0) wait(b_o, (f - 1) & 1);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) split_f16_rn(pack2(S[32 * g + 2 * i], S[32 * g + 2 * i + 1]), hi[i], lo[i]);
        tmem_st16(quad + kColS + 64 * half + 16 * g, hi);
        tmem_st16(quad + kColS + 64 * half + 32 + 16 * g, lo);
      }
      tmem_st_wait();
      arrive(b_s);
      put_out(0);
      wait(full(s), (c >> 1) & 1);
      rowwise |= reinterpret_cast<const int*>(hd)[kHdBad] != 0;
      if (tid == 0) by_rows[s] = rowwise;
      wait(b_r, c & 1);
      if (rowwise) {
        // back to the state itself
        const float un = pow2_inverse(sc_s);
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] *= un;
        sc_s = 1.f;
        // a value that is no number, or out of range, touches nothing of the rows before it: one row after another
        put_out(1);
        arrive(b_rp);
        if (jobs > 0) wait(out_free, (jobs - 1) & 1);   // the rows' powers of two of the chunk before are overwritten by the next one
        // in the place of operands that nothing reads now: a row's k, q and decay, two buffers, and partial sums
        float* rb = reinterpret_cast<float*>(smem + s * kPart1);     // [2][k, q, decay][128]
        float* part = rb + 2 * 3 * 128;                              // [p, w, k q][2 halves][128]
        for (int t = 0; t < rows; ++t) {
          const int64_t row = row0 + c * kChunk + t;
          float* r = rb + (t & 1) * 3 * 128;
          if (tid < 128) {
            r[tid] = bf16_to_float(__ldg(x.k + row * x.ld_k + hq * kDeltaDim + tid));
            r[128 + tid] = bf16_to_float(__ldg(x.q + row * x.ld_q + hq * kDeltaDim + tid));
            r[256 + tid] = expf(__ldg(x.gate + row * x.ld_gate + (x.gate_dim == 1 ? h : h * kDeltaDim + tid)));
          }
          bar_state();
          float pk = 0.f, pq = 0.f, kq = 0.f;
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            const int k = 64 * half + i;
            S[i] *= r[256 + k];
            pk = fmaf(S[i], r[k], pk), pq = fmaf(S[i], r[128 + k], pq), kq = fmaf(r[k], r[128 + k], kq);
          }
          part[half * 128 + v] = pk, part[256 + half * 128 + v] = pq, part[512 + half * 128 + v] = kq;
          bar_state();
          const float u = __ldg(x.beta + row * x.ld_beta + h) *
                          (bf16_to_float(__ldg(x.v + row * x.ld_v + (int64_t)h * kDeltaDim + v)) - (part[v] + part[128 + v]));
          const float o = x.scale * fmaf(u, part[512 + v] + part[640 + v], part[256 + v] + part[384 + v]);
          if (half == 0) p.out[(row * x.heads + h) * kDeltaDim + v] = float_to_bf16(o);
#pragma unroll
          for (int i = 0; i < 64; ++i) S[i] = fmaf(u, r[64 * half + i], S[i]);
        }
        bar_state();
        fence_proxy_async_smem();   // copies write there again
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(s));
        if (c + 1 < chunks) {
          read_v(c + 1);
          rowwise = vote(c + 1);
        }
        continue;
      }
      const float inv_s = pow2_inverse(sc_s);
      // ---- R
      const float inv_kp = inv_s * hd[kHdInvKp], sum_kp = hd[kHdSumKp];
      const float bound_r = fmaxf(xchg(s, kMaxV, 0), xchg(s, kMaxV, 1)) + bound_s * sum_kp;
      const float sc_r = pow2_scale(bound_r, 14);
      {
        uint32_t acc[32], hi[16], lo[16];
        tmem_ld32(quad + kColAcc + 32 * half, acc);
        tmem_ld_wait();
        uint32_t top = 0u;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const f32x2 r = fma2(pack2(-inv_kp, -inv_kp), pack2(__uint_as_float(acc[2 * t]), __uint_as_float(acc[2 * t + 1])),
                               bf16x2_to_f32x2(vr[t]));
          split_f16(mul2(r, pack2(sc_r, sc_r)), hi[t], lo[t]);
          top = max_abs_f16x2(top, hi[t]);
        }
        tmem_st16(quad + kColParts + 16 * half, hi);
        tmem_st16(quad + kColParts + 32 + 16 * half, lo);
        xchg(s, kMaxR, half) = max_of_f16x2(top) * pow2_inverse(sc_r) * 1.001f;
        tmem_st_wait();
        arrive(b_rp);
      }
      // ---- U
      const float inv_t = pow2_inverse(sc_r) * (1.f / kScaleT), sum_t = hd[kHdSumT];
      put_out(1);
      // for the store warp, which hears of it from all warps; it is through with the chunk before the last one, whose place this takes
      if (tid < kChunk) reinterpret_cast<uint32_t*>(smem + kCOffRow)[s * kChunk + tid] = reinterpret_cast<const uint32_t*>(hd)[kHdO + tid];
      wait(b_u, f & 1);
      const float sc_u = pow2_scale(fmaxf(xchg(s, kMaxR, 0), xchg(s, kMaxR, 1)) * sum_t, 14);
      {
        uint32_t acc[32], hi[16], lo[16];
        tmem_ld32(quad + kColAcc + 32 * half, acc);
        tmem_ld_wait();
        const float f_u = inv_t * sc_u;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          split_f16_rn(mul2(pack2(__uint_as_float(acc[2 * t]), __uint_as_float(acc[2 * t + 1])), pack2(f_u, f_u)), hi[t], lo[t]);
        }
        tmem_st16(quad + kColParts + 16 * half, hi);
        tmem_st16(quad + kColParts + 32 + 16 * half, lo);
        tmem_st_wait();
        arrive(b_up);
      }
      // ---- the state behind the chunk
      const float inv_u = pow2_inverse(sc_u);
      const float inv_o1 = inv_s * hd[kHdInvK] * scale, inv_o2 = inv_u * hd[kHdInvB] * scale;
      if (c + 1 < chunks) {
        read_v(c + 1);
        rowwise = vote(c + 1);
      }
      wait(b_ds, f & 1);
      // a state that is nothing beside its update: in a smaller power of two, for the sum to stay in fp32's range
      const float most = 32768.f * inv_u * hd[kHdSumKd];
      if (__any_sync(0xffffffffu, most * sc_s > 0x1p100f)) {
        const float to = most * sc_s > 0x1p100f ? pow2_scale(most, 12) : sc_s, by = to * pow2_inverse(sc_s);
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] *= by;
        sc_s = to;
      }
      const float inv_kd = inv_u * hd[kHdInvK] * sc_s;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t acc[32];
        tmem_ld32(quad + kColDs + 64 * half + 32 * g, acc);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 d = *reinterpret_cast<const float4*>(hd + kHdP + 64 * half + 32 * g + 4 * i);
          float* st = S + 32 * g + 4 * i;
          st[0] = fmaf(st[0], d.x, inv_kd * __uint_as_float(acc[4 * i]));
          st[1] = fmaf(st[1], d.y, inv_kd * __uint_as_float(acc[4 * i + 1]));
          st[2] = fmaf(st[2], d.z, inv_kd * __uint_as_float(acc[4 * i + 2]));
          st[3] = fmaf(st[3], d.w, inv_kd * __uint_as_float(acc[4 * i + 3]));
        }
      }
      __syncwarp();   // likewise
      if (lane == 0) mbar_arrive(empty(s));
      out_rows = rows, out_c = c, out_f1 = inv_o1, out_f2 = inv_o2;
      ++f;
    }
    if (out_rows > 0) wait(b_o, (f - 1) & 1);
    put_out(0);
    put_out(1);
    if (jobs > 0) wait(out_free, (jobs - 1) & 1);
    if (tid == 0) out_job[1] = 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(out_full);
    if (float* to = state_out(p.s, b, 0, h)) {
      const float un = pow2_inverse(sc_s);
#pragma unroll
      for (int i = 0; i < 64; ++i) S[i] *= un;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<float4*>(to + v * kDeltaDim + 64 * half + 4 * i) =
            make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

namespace {
int long_sequences(int rows, int batch) { return std::min(batch, rows / (kFewRows + 1)); }
int64_t long_chunks(int rows, int batch) { return (int64_t)rows / kChunk + long_sequences(rows, batch); }
size_t list_bytes(int rows, int batch) { return ((size_t)(1 + long_sequences(rows, batch)) * 16 + 1023) & ~size_t(1023); }
}  // namespace

size_t delta_chunk_workspace_bytes(int rows, int batch, int heads) {
  return list_bytes(rows, batch) + (size_t)long_chunks(rows, batch) * heads * kRecBytes;
}

dsa_status_t launch_delta_chunks(const DeltaRows& x, const DeltaSeqs& seqs, uint16_t* out, void* workspace, cudaStream_t st) {
  if (seqs.rows <= kFewRows) return launch_delta_rows(x, seqs, out, st);
  static std::atomic<uint64_t> ready{0};   // devices whose kernels may take their shared memory
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    cudaError_t e = cudaFuncSetAttribute(delta_prepare_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrepSmem + 1024);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(delta_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kChainSmem);
    cudaFuncAttributes at = {};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, delta_chain_kernel);
    if (e != cudaSuccess) return cuda_status(e);
    // the state warps would wait for registers that the block does not have
    if (at.numRegs * kChainThreads < 128 * kHelperRegs + 256 * kStateRegs) return DSA_ERR_UNSUPPORTED;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  DeltaSeqs s = seqs;
  s.index = static_cast<int4*>(workspace);
  s.many = long_sequences(s.rows, s.batch);
  const dsa_status_t first = launch_delta_rows(x, s, out, st);
  if (first != DSA_OK) return first;
  const int64_t chunks = long_chunks(s.rows, s.batch);
  const ChunkArgs a{x, s, static_cast<uint8_t*>(workspace) + list_bytes(s.rows, s.batch), (int32_t)chunks, out, 2 * num_sms()};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.gridDim = dim3((unsigned)(chunks * x.heads));
  cfg.blockDim = dim3(kPrepThreads);
  cfg.dynamicSmemBytes = kPrepSmem + 1024;
  count_launches(2);
  if (cuda_status(cudaLaunchKernelEx(&cfg, delta_prepare_kernel, a)) != DSA_OK) return DSA_ERR_CUDA;
  cfg.attrs = &attr;   // the chain may start while operands are still prepared
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(s.many * x.heads));
  cfg.blockDim = dim3(kChainThreads);
  cfg.dynamicSmemBytes = kChainSmem;
  if (cuda_status(cudaLaunchKernelEx(&cfg, delta_chain_kernel, a)) != DSA_OK) return DSA_ERR_CUDA;
  return launch_status();
}

}  // namespace dsa
