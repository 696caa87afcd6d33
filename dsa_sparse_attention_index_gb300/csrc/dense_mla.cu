// dense_mla.cu — exact MLA over every token a row sees in the paged cache.
//
// The same attention as the sparse kernel (absorbed MLA, 96 heads, keys = all
// 576 columns of a latent, values = its first 512), without a selection: for
// layers that have no indexer, contexts too short to select from, caches that
// eviction holds at a budget, and prefill chunks whose rows see the whole
// prefix.  For row r, head h and its visible tokens t:
//   l_t = sm_scale * latent_scale * (q[r][h] . c_t)
//   O   = latent_scale * sum_t softmax(l)_t c_t[0:512],  LSE = ln sum_t exp(l_t)
// with c_t the unscaled E4M3 or NVFP4 latent.
//
// GB300 design (persistent, one CTA per SM, 15 warps):
//   * All rows' 48-token tiles form one line; CTA c takes an equal run of it
//     (run.cuh), so ragged batches, one long context and a prefill chunk all fill
//     every SM to within a tile.  A row that lies in one CTA's run is written at
//     once; one that crosses runs leaves a partial (normalised fp16 O, reference
//     and sum) per CTA, merged through the log-sum-exp by the combine kernel.
//   * Operands are fp16, not bf16: E4M3 values and E2M1 x E4M3 products are exact
//     in it, the conversion instructions widen to it in a third of the
//     instructions that bf16 takes, and P keeps 11 bits.  query.cu turns Q into
//     fp16 times a power of two a head.
//   * Two roundings to fp16 are choices: P's as an operand (its sum, the
//     normaliser, is taken in fp32 before) and a partial's.  Each is off by 2^-11 of
//     the weighted mean of |c| at most, where the bf16 output's own rounding takes
//     2^-8 of the value; a partial in fp32 would double the workspace and what the
//     merge reads.  Below 2^-14 of a latent's unit a partial's step is 2^-24.
//   * warps 4..12, one per 64-dim block: two lanes a token, 16-byte loads a whole
//     tile ahead in registers, a token's page looked up two tiles ahead; widened,
//     stored 128-byte swizzled into one of two tile buffers, which are filled and
//     freed in halves.  A tile is the B operand of QK^T (K-major, N = 48 tokens)
//     and the A operand of P V (MN-major, M = 128 dims over two blocks).
//   * S = Q K^T has the heads on M = 128 rows (96 used).  Q dims 0..511 sit in
//     shared memory, 512..575 in TMEM, O^T [512 dims x 96 heads] in 384 TMEM
//     columns, two S tiles in 96.
//   * warp 13 issues QK^T, warp 14 P V, each as a whole with its MMAs under
//     elect.sync; warps 0..3 run the online softmax, one thread per head: P is
//     2^7 exp(l - reference) in fp16 (full precision down to 2^-21 of a head's
//     largest weight), its fp32 sum the normaliser; O^T is rescaled, 32 heads at a
//     time, only where a maximum grew by more than 2^8.  Tokens behind a row's last and
//     those of a page outside the pool are masked.
// What bounds it: the shared-memory port.  A tile's MMAs read 272 KB (QK^T 32 x
// (4 KB of Q + 1.5 KB of keys) + 4 x 1.5 KB, PV 12 x (4 KB of values + 3 KB of
// P)) and its stores and polls take about 85 KB: 2,800 cycles at 128 B a cycle,
// of which the measured 1.6 us use 86 % (32 contexts of 8K to 64K tokens, NVFP4:
// 272 us, 906 TFLOP/s, 0.47 of the measured bf16 burst rate).  The tensor pipe is
// active 47 % of the time.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "run.cuh"

namespace dsa {

namespace {

constexpr int kTile = 48;                              // tokens per tile
constexpr int kDB = kLatent / 64;                      // 9 blocks of 64 dims
constexpr int kVB = kValue / 64;                       // 8 of them are values
constexpr int kQTmemBlocks = 1;                        // Q dims 512..575 in TMEM
constexpr int kQSmemBlocks = kDB - kQTmemBlocks;       // Q dims 0..511 in shared memory
constexpr int kQBlockBytes = kHeads * 128;             // 12,288
constexpr int kBlkBytes = kTile * 128;                 // 6,144: 48 tokens x 64 dims of fp16
constexpr int kTileBytes = kDB * kBlkBytes;            // 55,296; block 8 holds the key-only dims
constexpr int kBufs = 2;                               // tile buffers, each filled and freed in two halves
constexpr int kPBytes = kHeads * 128;                  // 12,288: a head's 48 fp16 in a 128-byte row
constexpr int kNvRec = kValue / 2 + kValue / 16 + (kLatent - kValue);  // 352 B
constexpr int kThreads = 15 * 32;  // softmax 0-3, loaders 4-12 (one 64-dim block each), QK issuer 13, PV issuer 14
constexpr int kLoadWarp0 = 4;
constexpr int kQkWarp = 13;
constexpr int kPvWarp = 14;
static_assert(kLoadWarp0 + kDB == kQkWarp, "a loader warp a block");
constexpr int kOCols = 4 * kHeads;                     // 384
constexpr int kSCol = kOCols;                          // two S tiles: 384..479
constexpr int kQ8Col = kSCol + 2 * kTile;              // 480..511
static_assert(kQ8Col + 32 * kQTmemBlocks <= 512, "TMEM columns");
constexpr float kRescaleThreshold = 8.0f;              // log2 units
constexpr float kPShift = 7.0f;                        // P is stored times 2^7, at most 2^15
constexpr int kMaxGrid = 256;                          // CTAs the workspace is sized for
constexpr int kInvariantTiles = 80;                    // tiles per part in the batch-invariant mode

constexpr int kOffQ = 0;
constexpr int kOffTile = kOffQ + kQSmemBlocks * kQBlockBytes;  // 98,304
constexpr int kOffP = kOffTile + kBufs * kTileBytes;           // 208,896
constexpr int kOffAlpha = kOffP + kPBytes;                     // 221,184
constexpr int kOffBars = kOffAlpha + 512 + 16;
constexpr int kNumBars = 4 * kBufs + 11;
constexpr int kOffMisc = (kOffBars + kNumBars * 8 + 15) / 16 * 16;              // TMEM slot, abort flag, scan scratch
constexpr size_t kSmemBytes = 1024 + kOffMisc + 16 + 32 * 8;
static_assert(kOffTile % 1024 == 0 && kOffP % 1024 == 0 && kBlkBytes % 1024 == 0, "swizzle atoms");
static_assert(kSmemBytes <= 232448, "shared memory");

constexpr size_t kPartO = (size_t)kHeads * kValue;             // fp16 values of a partial

struct DenseParams {
  const uint8_t* latent_base;
  int64_t row_stride;
  int32_t num_blocks;
  const int32_t* block_table;
  int32_t max_blocks;
  const int32_t* seq_lens;
  int32_t nq, cap, rows;
  float logit_scale_log2;  // sm_scale * latent_scale * log2(e)
  float latent_scale;
  const uint16_t* q16;     // the queries in fp16 times a power of two a head
  const float* q_inv;      // its inverse, [rows][96]
  uint16_t* out;
  float* lse;
  uint16_t* opart;  // fp16 [slots][96][512]
  float* ml;        // [slots][96][2]: reference (log2), sum of 2^(l - reference)
  int2* row_info;   // [rows]: first slot key, number of parts (0: no token, 1: written by the kernel)
  int32_t unit;     // tiles of a fixed part in the batch-invariant mode, else 0
  int32_t* status;
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (a - m, b - m) in one instruction.
__device__ __forceinline__ void sub2f(uint32_t a, uint32_t b, float m, float& x, float& y) {
  asm("{\n .reg .b64 v, w;\n mov.b64 v, {%2, %3};\n mov.b64 w, {%4, %4};\n add.rn.f32x2 v, v, w;\n mov.b64 {%0, %1}, v;\n}\n"
      : "=f"(x), "=f"(y)
      : "r"(a), "r"(b), "f"(-m));
}

__device__ __forceinline__ bool bar_or_softmax(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, 1, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// A part of a row: tiles [t0, t1) of `row`, written to `slot` (< 0: the whole
// row, written to the outputs).
struct Segment {
  int row, vis, t0, t1, slot;
};

// Walks the CTA's parts.  Every role walks on its own and meets the same parts.
//   plain:      the CTA's run [pos, hi) of the line of all rows' tiles.  A row
//               that began before the run, or fills all of it, goes to slot
//               2 cta, one that goes on behind it to slot 2 cta + 1.
//   invariant:  parts of `unit` tiles counted over all rows, CTA c taking every
//               gridDim-th; a part's slot is its number.
struct Walk {
  const DenseParams& p;
  int row;        // next row
  int64_t start;  // first tile (or part) of `row` on the line
  int64_t pos, hi;

  __device__ int visible(int r) const {
    int len = p.seq_lens[r / p.nq];
    len = len < 0 ? 0 : (len > p.cap ? p.cap : len);
    return visible_len(len, p.nq, r % p.nq);
  }
  __device__ bool next(Segment& s) {
    while (pos < hi && row < p.rows) {
      const int vis = visible(row);
      const int tiles = (vis + kTile - 1) / kTile;
      const int64_t n = p.unit ? (tiles + p.unit - 1) / p.unit : tiles;
      if (pos >= start + n) {
        start += n;
        ++row;
        continue;
      }
      s.row = row;
      s.vis = vis;
      if (p.unit) {
        const int u = (int)(pos - start);
        s.t0 = u * p.unit;
        s.t1 = min(tiles, s.t0 + p.unit);
        s.slot = n == 1 ? -1 : (int)pos;
        pos += gridDim.x;
      } else {
        s.t0 = (int)(pos - start);
        s.t1 = (int)min((int64_t)tiles, hi - start);
        const bool ends = start + n <= hi;
        s.slot = s.t0 > 0 ? 2 * (int)blockIdx.x : (ends ? -1 : 2 * (int)blockIdx.x + 1);
        pos = start + s.t1;
      }
      return true;
    }
    return false;
  }
};

// This CTA's place on the line, by all threads; CTA 0 also writes row_info.
__device__ Walk make_walk(const DenseParams& p, int64_t* scratch) {
  Walk w{p, 0, 0, 0, 0};
  auto count = [&](int r) -> int64_t {
    const int tiles = (w.visible(r) + kTile - 1) / kTile;
    return p.unit ? (tiles + p.unit - 1) / p.unit : tiles;
  };
  auto each = [&](int r, int64_t first, int64_t n, int64_t per) {
    if (p.unit) {
      p.row_info[r] = make_int2((int)first, (int)n);
    } else {
      const int64_t c0 = first / per;
      p.row_info[r] = make_int2((int)c0, n == 0 ? 0 : (int)((first + n - 1) / per - c0 + 1));
    }
  };
  const Run run = find_run<kThreads>(p.rows, p.unit ? 1 : 0, scratch, count, each);
  w.row = run.row;
  w.start = run.start;
  w.pos = run.pos;
  w.hi = run.hi;
  return w;
}

// O^T of a part from TMEM (lanes: dims of a 128-dim block, columns: heads), times
// alpha per head, to dst [96][512] as bf16 or fp16, by sets of four warps, each set
// the pieces [c, end) of 12 (a piece: 32 heads of a 128-dim block): a warp turns
// 32 heads x 32 dims at a time in 2 KB of its own, the next 32 on the way from TMEM
// meanwhile, and writes 64 bytes a head.
template <bool kBf16>
__device__ __forceinline__ void write_part(int c, int end, uint32_t lane_base, const float* alpha, uint8_t* turn,
                                           uint16_t* dst) {
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  uint16_t* col = reinterpret_cast<uint16_t*>(turn) + lane;
  const uint4* rows = reinterpret_cast<const uint4*>(turn) + lane;
  uint16_t* to = dst + (lane >> 2) * kValue + warp * 32 + (lane & 3) * 8;
  auto fetch = [&](int c, uint32_t (&o)[32]) { tmem_ld32(lane_base + (c / 3) * kHeads + (c % 3) * 32, o); };
  auto put = [&](int c, const uint32_t (&o)[32]) {
    const int hg = (c % 3) * 32, d0 = (c / 3) * 128;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 a = *reinterpret_cast<const float4*>(alpha + hg + j);
      const float v0 = __uint_as_float(o[j]) * a.x, v1 = __uint_as_float(o[j + 1]) * a.y,
                  v2 = __uint_as_float(o[j + 2]) * a.z, v3 = __uint_as_float(o[j + 3]) * a.w;
      uint32_t x, y;
      if (kBf16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v0, v1), q = __floats2bfloat162_rn(v2, v3);
        x = *reinterpret_cast<const uint32_t*>(&p);
        y = *reinterpret_cast<const uint32_t*>(&q);
      } else {
        const __half2 p = __floats2half2_rn(v0, v1), q = __floats2half2_rn(v2, v3);
        x = *reinterpret_cast<const uint32_t*>(&p);
        y = *reinterpret_cast<const uint32_t*>(&q);
      }
      col[j * 32] = (uint16_t)x;
      col[(j + 1) * 32] = (uint16_t)(x >> 16);
      col[(j + 2) * 32] = (uint16_t)y;
      col[(j + 3) * 32] = (uint16_t)(y >> 16);
    }
    __syncwarp();
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = rows[32 * u];  // heads 8 u + lane / 4
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint2* p = reinterpret_cast<uint2*>(to + (hg + 8 * u) * kValue + d0);  // out is 8-byte aligned
      p[0] = make_uint2(v[u].x, v[u].y);
      p[1] = make_uint2(v[u].z, v[u].w);
    }
    __syncwarp();
  };
  uint32_t o0[32], o1[32];
  fetch(c, o0);
#pragma unroll 1
  for (; c < end; c += 2) {
    tmem_ld_wait();
    fetch(c + 1, o1);
    put(c, o0);
    tmem_ld_wait();
    if (c + 2 < end) fetch(c + 2, o0);
    put(c + 1, o1);
  }
}

// What a lane without a token reads: zeros take no part in the products.
__device__ const uint4 zero_record[kLatent / 16] = {};

template <bool kNV>
__global__ void __launch_bounds__(kThreads, 1)
    dense_mla_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ DenseParams p) {
  constexpr int kRec = kNV ? kNvRec : kLatent;
  constexpr uint32_t kIdescQK = make_idesc(kFmtF16, kFmtF16, 0, 0, 128, kTile);
  constexpr uint32_t kIdescPV = make_idesc(kFmtF16, kFmtF16, 1, 0, 128, kHeads);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + kOffBars;
  auto full = [&](uint32_t buf, int half) { return bars + 8u * (2 * buf + half); };
  auto empty = [&](uint32_t buf, int half) { return bars + 8u * (2 * kBufs + 2 * buf + half); };
  const uint32_t bars2 = bars + 8u * (4 * kBufs);
  const uint32_t q_full = bars2, q8_full = bars2 + 8, o_free = bars2 + 16, drain = bars2 + 24, p_full = bars2 + 32,
                 pv_done = bars2 + 40;
  auto s_full = [&](uint32_t b) { return bars2 + 48 + 8 * b; };
  auto s_empty = [&](uint32_t b) { return bars2 + 64 + 8 * b; };
  const uint32_t o_last = bars2 + 80;  // the CTA's last O^T is complete and its factors are in alpha_s
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int64_t* scratch = reinterpret_cast<int64_t*>(smem + kOffMisc + 16);
  float* alpha_s = reinterpret_cast<float*>(smem + kOffAlpha);  // 128 factors, then per softmax warp whether a head grew
  volatile int* grew_s = reinterpret_cast<volatile int*>(smem + kOffAlpha + 512);
  const int warp = warp_number(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kBufs; ++s)
      for (int h = 0; h < 2; ++h) {
        mbar_init(full(s, h), h ? kDB - kVB / 2 : kVB / 2);
        mbar_init(empty(s, h), 1);
      }
    mbar_init(q_full, 1);
    mbar_init(q8_full, 4);
    mbar_init(p_full, 4);
    mbar_init(pv_done, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(s_empty(b), 4);
    }
    mbar_init(o_free, 4);
    mbar_init(o_last, 4);
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_q);
  }
  if (warp == kQkWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // The queries come from the previous kernel, which let this one start only when
  // all before it had completed: the lengths can be read before the wait.
  Walk walk = make_walk(p, scratch);
  grid_dep_wait();
  grid_dep_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  Segment sg;
  // walk.next by a whole warp, with values that the compiler knows to be the same in every lane
  auto next_uniform = [&](Segment& s) -> bool {
    const bool more = __all_sync(0xffffffffu, walk.next(s));
    s.row = __shfl_sync(0xffffffffu, s.row, 0);
    s.t0 = __shfl_sync(0xffffffffu, s.t0, 0);
    s.t1 = __shfl_sync(0xffffffffu, s.t1, 0);
    return more;
  };

  if (warp == kQkWarp) {
    // ------------------------------------------------ QK issuer (the whole warp runs, one lane issues)
    const uint64_t q_desc = smem_desc(sbase + kOffQ, 16, 1024, kLayoutSw128);
    const uint32_t q_lo = (uint32_t)q_desc, hi = (uint32_t)(q_desc >> 32);
    const uint32_t t_lo0 = (uint32_t)smem_desc(sbase + kOffTile, 16, 1024, kLayoutSw128);
    uint32_t it = 0, seg = 0;
    bool ok = true;
    while (ok && next_uniform(sg)) {
      // the previous part's last QK^T has completed: Q may go
      if (it > 0) ok = mbar_wait_warp(s_full((it - 1) & 1), ((it - 1) >> 1) & 1, abort_flag, p.status);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(q_full, kQSmemBlocks * kQBlockBytes);
        for (int kb = 0; kb < kQSmemBlocks; ++kb)
          tma_load_2d(sbase + kOffQ + kb * kQBlockBytes, &tmap_q, kb * 64, sg.row * kHeads, q_full);
      }
      __syncwarp();
      ok = mbar_wait_warp(q_full, seg & 1, abort_flag, p.status);
      ok = ok && mbar_wait_warp(q8_full, seg & 1, abort_flag, p.status);
      ++seg;
      for (int t = sg.t0; ok && t < sg.t1; ++t, ++it) {
        ok = mbar_wait_warp(s_empty(it & 1), ((it >> 1) & 1) ^ 1, abort_flag, p.status);
        const uint32_t d = tmem + kSCol + (it & 1) * kTile;
        const uint32_t buf = it % kBufs, t_lo = t_lo0 + buf * (kTileBytes / 16);
        int kb = 0;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          ok = ok && mbar_wait_warp(full(buf, half), (it / kBufs) & 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const int end = half ? kQSmemBlocks : kVB / 2;
#pragma unroll 1
            for (; kb < end; ++kb) {
              const uint32_t a_lo = q_lo + kb * (kQBlockBytes / 16), b_lo = t_lo + kb * (kBlkBytes / 16);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_bf16(d, desc64(a_lo + 2 * kk, hi), desc64(b_lo + 2 * kk, hi), kIdescQK, (kb | kk) ? 1u : 0u);
            }
            if (half) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // dims 512..575: A from TMEM
                mma_bf16_tmem_a(d, tmem + kQ8Col + 8 * kk, desc64(t_lo + kQSmemBlocks * (kBlkBytes / 16) + 2 * kk, hi), kIdescQK, 1u);
              mma_commit(s_full(it & 1));
            }
          }
          __syncwarp();
          kb = kVB / 2;
        }
        if (!ok) break;
        __syncwarp();
      }
    }
    if (elect_one()) {
      if (seg > 0) mbar_wait_drain(q_full, (seg - 1) & 1, 10000000ull);  // no copy is in flight at the exit
      // both issuers' MMAs complete before TMEM is released
      mma_commit(drain);
      mbar_wait_drain(drain, 0, 10000000ull);
    }
  } else if (warp == kPvWarp) {
    // ------------------------------------------------ PV issuer (likewise)
    const uint64_t a_desc = smem_desc(sbase + kOffTile, kBlkBytes, 1024, kLayoutSw128);
    const uint32_t a_lo0 = (uint32_t)a_desc, a_hi = (uint32_t)(a_desc >> 32);
    const uint64_t p_desc = smem_desc(sbase + kOffP, 16, 1024, kLayoutSw128);
    const uint32_t p_lo = (uint32_t)p_desc, p_hi = (uint32_t)(p_desc >> 32);
    uint32_t it = 0, seg = 0;
    bool ok = true;
    while (ok && next_uniform(sg)) {
      // the previous part's O^T has been read
      if (seg > 0) ok = mbar_wait_warp(o_free, (seg - 1) & 1, abort_flag, p.status);
      ++seg;
      for (int t = sg.t0; ok && t < sg.t1; ++t, ++it) {
        ok = mbar_wait_warp(p_full, it & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t more = t > sg.t0;
        const uint32_t a_lo = a_lo0 + (it % kBufs) * (kTileBytes / 16);
        if (elect_one()) {
#pragma unroll 1
          for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              mma_bf16(tmem + mb * kHeads, desc64(a_lo + 2 * mb * (kBlkBytes / 16) + 2 * ks * 64, a_hi),
                       desc64(p_lo + 2 * ks, p_hi), kIdescPV, ks > 0 ? 1u : more);
            // QK^T of this tile completed before its P existed, so half the tile is free after these
            if (mb & 1) mma_commit(empty(it % kBufs, mb >> 1));
          }
          mma_commit(pv_done);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      mma_commit(drain);
      mbar_wait_drain(drain, 0, 10000000ull);
    }
  } else if (warp >= kLoadWarp0 && warp < kQkWarp) {
    // ------------------------------------------------ loaders: records -> fp16 blocks
    // Warp kb: the 64 dims of block kb, two lanes a token, 16 tokens at a time.
    // Eight neighbouring lanes store 16 bytes each to all 32 banks.  Codes are
    // loaded a whole tile before they are stored, a token's page is looked up two
    // tiles ahead, and codes are widened before the wait for the buffer.
    constexpr int kTt = kTile / 16;  // tokens of a lane
    const int kb = warp - kLoadWarp0, h = kb >= kVB / 2;
    const bool four = kNV && kb < kVB;  // E2M1 codes with block scales; else E4M3 codes
    const int sub = lane & 1, tok0 = lane >> 1;
    const uint32_t off = (uint32_t)(kb * kBlkBytes + tok0 * 128 + sub * 64);
    uint32_t o0 = swz128(off), o1 = swz128(off + 16), o2 = swz128(off + 32), o3 = swz128(off + 48);
    // byte offsets in a record of this lane's codes and scales
    const int c0 = four ? 32 * kb + 16 * sub : (kNV ? kValue / 2 + kValue / 16 : 64 * kb) + 32 * sub;
    const int s0 = kValue / 2 + 4 * kb + 2 * sub;
    uint4 buf[kTt][2];
    uint32_t sc[kTt];
    const uint8_t* none = reinterpret_cast<const uint8_t*>(zero_record);
    const uint8_t* rec[kTt];
    const int32_t* table = nullptr;
    int t = 0, t1 = 0, page[kTt], first = 0, vis = 0;
    bool have_page = false, have = false;
    auto step_page = [&]() {  // the next tile's pages
      have_page = t < t1;
      if (!have_page && walk.next(sg)) {
        table = p.block_table + (int64_t)(sg.row / p.nq) * p.max_blocks;
        vis = sg.vis;
        t = sg.t0;
        t1 = sg.t1;
        have_page = true;
      }
      if (!have_page) return;
      first = t++ * kTile + tok0;
#pragma unroll
      for (int i = 0; i < kTt; ++i)
        if (first + 16 * i < vis) page[i] = table[(first + 16 * i) / kBlock];
    };
    auto step_record = [&]() {
      have = have_page;
#pragma unroll
      for (int i = 0; i < kTt; ++i) {
        rec[i] = none;  // no such token, or a bad table entry: zeros
        const int token = first + 16 * i;
        if (!have || token >= vis) continue;
        if ((uint32_t)page[i] < (uint32_t)p.num_blocks)
          rec[i] = p.latent_base + (int64_t)page[i] * p.row_stride + token % kBlock * kRec;
        else
          report(p.status, DSA_ERR_BOUNDS);
      }
    };
    auto load = [&]() {
#pragma unroll
      for (int i = 0; i < kTt; ++i) {
        buf[i][0] = __ldg(reinterpret_cast<const uint4*>(rec[i] + c0));
        if (four)
          sc[i] = __ldg(reinterpret_cast<const uint16_t*>(rec[i] + s0));
        else
          buf[i][1] = __ldg(reinterpret_cast<const uint4*>(rec[i] + c0 + 16));
      }
    };
    step_page();
    step_record();
    step_page();
    if (have) load();
    uint32_t it = 0;
    while (have) {
      uint32_t o[2 * kTt][8];
#pragma unroll
      for (int i = 0; i < kTt; ++i) {
        if (four) {
          nvfp4x16_to_f16x16(buf[i][0].x, buf[i][0].y, sc[i] & 0xFFu, o[2 * i]);
          nvfp4x16_to_f16x16(buf[i][0].z, buf[i][0].w, sc[i] >> 8, o[2 * i + 1]);
        } else {
          e4m3x16_to_f16x16(buf[i][0], o[2 * i]);
          e4m3x16_to_f16x16(buf[i][1], o[2 * i + 1]);
        }
      }
      step_record();
      step_page();
      if (have) load();
      if (!mbar_wait_warp(empty(it % kBufs, h), ((it / kBufs) & 1) ^ 1, abort_flag, p.status)) break;
      uint8_t* tile = smem + kOffTile + (it % kBufs) * kTileBytes;
#pragma unroll
      for (int i = 0; i < kTt; ++i) {
        uint8_t* at = tile + 2048 * i;  // 16 tokens on: two swizzle atoms
        *reinterpret_cast<uint4*>(at + o0) = make_uint4(o[2 * i][0], o[2 * i][1], o[2 * i][2], o[2 * i][3]);
        *reinterpret_cast<uint4*>(at + o1) = make_uint4(o[2 * i][4], o[2 * i][5], o[2 * i][6], o[2 * i][7]);
        *reinterpret_cast<uint4*>(at + o2) = make_uint4(o[2 * i + 1][0], o[2 * i + 1][1], o[2 * i + 1][2], o[2 * i + 1][3]);
        *reinterpret_cast<uint4*>(at + o3) = make_uint4(o[2 * i + 1][4], o[2 * i + 1][5], o[2 * i + 1][6], o[2 * i + 1][7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(it % kBufs, h));
      ++it;
    }
    // The CTA's last part: eight of these warps write two thirds of it (the softmax
    // warps alone: 21.1 instead of 19.9 us for one row of 997 tokens, 57.0 instead of
    // 55.6 for 32 draft rows); the tile buffers are free when it is complete.
    if (it > 0 && !have && kb < kVB && mbar_wait_warp(o_last, 0, abort_flag, p.status)) {
      tc_fence_after();
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      uint8_t* turn = smem + kOffTile + kb * 2048;
      const int c = 4 + 4 * h;
      if (sg.slot < 0)
        write_part<true>(c, c + 4, lane_base, alpha_s, turn, p.out + (int64_t)sg.row * kPartO);
      else
        write_part<false>(c, c + 4, lane_base, alpha_s, turn, p.opart + (int64_t)sg.slot * kPartO);
    }
  } else if (warp < kLoadWarp0) {
    // ------------------------------------------------ softmax (thread = head) and the parts' outputs
    const int h = threadIdx.x;
    const bool live = h < kHeads;
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t it = 0;
    bool ok = true;
    while (ok && walk.next(sg)) {
      // ---- Q dims 512..575 of head h into TMEM (every QK^T of the previous part has completed)
      // logits in log2 units per unit of S
      const float c_raw = p.logit_scale_log2 * p.q_inv[(int64_t)sg.row * kHeads + (live ? h : 0)];
      // its magnitude; a scale of 0 becomes one that still sends a masked token's -inf to -inf, and one that
      // is no number makes every logit NaN
      const float c_log2 = fabsf(c_raw) < INFINITY ? fmaxf(fabsf(c_raw), 1e-38f) : __int_as_float(0x7FC00000);
      {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q16 + ((int64_t)sg.row * kHeads + (live ? h : 0)) * kLatent + 64 * kQSmemBlocks);
        uint4 v[8 * kQTmemBlocks];
#pragma unroll
        for (int c = 0; c < 8 * kQTmemBlocks; ++c) v[c] = live ? src[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < 8 * kQTmemBlocks; ++c)
          tmem_st4(lane_base + kQ8Col + 4 * c, v[c].x, v[c].y, v[c].z, v[c].w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q8_full);
      }
      // Whether a page of the part lies outside the pool (the loaders report it), by all lanes while the first S is
      // on its way: looked up in every tile, two entries cost 1 % of a decode batch and 4 % of one long context
      auto hole = [&](int page) {
        return (uint32_t)p.block_table[(int64_t)(sg.row / p.nq) * p.max_blocks + page] >= (uint32_t)p.num_blocks;
      };
      bool holes = false;
#pragma unroll 4
      for (int g = sg.t0 * kTile / kBlock + lane; g <= (min(sg.t1 * kTile, sg.vis) - 1) / kBlock; g += 32)
        holes |= hole(g);
      holes = __any_sync(0xffffffffu, holes);
      // the reference, in units of S
      float m_used = -INFINITY, l_sum = 0.f;
      for (int t = sg.t0; t < sg.t1; ++t, ++it) {
        ok = ok && mbar_wait_warp(s_full(it & 1), (it >> 1) & 1, abort_flag, p.status);
        tc_fence_after();
        uint32_t r[kTile];
        const uint32_t s_col = lane_base + kSCol + (it & 1) * kTile;
        tmem_ld32(s_col, *reinterpret_cast<uint32_t(*)[32]>(r));
        tmem_ld16(s_col + 32, r + 32);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty(it & 1));
        int lo = 0, up = sg.vis - t * kTile;  // the tile's tokens [lo, up) take part
        if (holes) {  // those of a page outside the pool do not; a tile lies on at most two pages
          up = min(up, kTile);
          const int split = min(kBlock - t * kTile % kBlock, up);  // tokens on the first
          const bool hole1 = hole((t * kTile + up - 1) / kBlock);
          if (hole(t * kTile / kBlock)) lo = split;
          if (hole1) up = split;
        }
        if (c_raw < 0.f) {  // a negative scale: the largest logit is that of the smallest product
#pragma unroll
          for (int j = 0; j < kTile; ++j) r[j] ^= 0x80000000u;
        }
        if (lo > 0 || up < kTile) {
#pragma unroll
          for (int j = 0; j < kTile; ++j) r[j] = j >= lo && j < up ? r[j] : 0xFF800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < kTile; j += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx[i] = fmaxf(fmaxf(mx[i], __uint_as_float(r[j + 2 * i])), __uint_as_float(r[j + 2 * i + 1]));
        const float m_tile = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // A maximum of -inf over a tile's tokens is that of logits that are all -inf or NaN (fmaxf drops NaN).
        // That, a NaN and +inf come from a query, a scale or a logit that is no fp32 number: a NaN row
        if (lo < up && !(fabsf(m_tile * c_log2) < INFINITY)) m_used = __int_as_float(0x7FC00000);
        const bool grow =
            live && (m_used == -INFINITY ? m_tile > -INFINITY : (m_tile - m_used) * c_log2 > kRescaleThreshold);
        // one barrier a tile: any head that grew, and any warp whose wait ran out
        if (bar_or_softmax(grow || !ok)) {
          const float m_new = grow ? m_tile : m_used;
          const float alpha = (m_used == -INFINITY) ? 0.f : ex2f((m_used - m_new) * c_log2);
          alpha_s[h] = alpha;
          if (lane == 0) grew_s[warp] = 0;
          __syncwarp();
          if (grow) grew_s[warp] = 1;
          l_sum *= alpha;
          m_used = m_new;
          if (t > sg.t0) ok = ok && mbar_wait_warp(pv_done, (it - 1) & 1, abort_flag, p.status);
          if (bar_or_softmax(!ok)) { ok = false; break; }  // also publishes alpha_s and grew_s
          if (t > sg.t0) {
            tc_fence_after();
#pragma unroll 1
            for (int g = 0; g < kHeads / 32; ++g) {
              if (!grew_s[g]) continue;  // the 32 heads of warp g
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t o[16];
                const int col = g * 32 + (c & 1) * 16;
                const uint32_t ta = lane_base + (c >> 1) * kHeads + col;
                tmem_ld16(ta, o);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha_s[col + j]);
                tmem_st16(ta, o);
              }
            }
            tmem_st_wait();
          }
        }
        uint32_t pk[kTile / 2];
        // times 2^7: fp16 keeps its 11 bits for weights down to 2^-21 of the largest.  The differences from the
        // reference are taken before the scaling: subtracted from the scaled logits, the steps of fp32 at a
        // logit of 2^26 take the largest P out of fp16 (by 24 packed subtractions: 512-row chunk 1.729 -> 1.750 ms)
        const float from = m_used == -INFINITY ? 0.f : m_used;  // no token so far: every logit is -inf, every P 0
        float se[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kTile; j += 2) {
          float x0, x1;
          sub2f(r[j], r[j + 1], from, x0, x1);
          const float p0 = ex2f(fmaf(x0, c_log2, kPShift)), p1 = ex2f(fmaf(x1, c_log2, kPShift));
          const __half2 bb = __floats2half2_rn(p0, p1);
          se[0] += p0;
          se[1] += p1;
          pk[j >> 1] = *reinterpret_cast<const uint32_t*>(&bb);
        }
        l_sum += se[0] + se[1];
        // the PV of the tile before has read the P buffer; a wait that runs out is
        // told to the other warps at the next barrier
        ok = it == 0 || mbar_wait_warp(pv_done, (it - 1) & 1, abort_flag, p.status);
        if (live && ok) {
          uint8_t* prow = smem + kOffP;
#pragma unroll
          for (int c = 0; c < kTile / 8; ++c)
            *reinterpret_cast<uint4*>(prow + swz128(h * 128 + c * 16)) =
                make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(p_full);
      }
      if (ok) ok = mbar_wait(pv_done, (it - 1) & 1, abort_flag, p.status);
      // ---- the part's O^T: lanes are dims of a 128-dim block, columns heads
      const bool direct = sg.slot < 0;
      alpha_s[h] = live && m_used != -INFINITY ? (direct ? p.latent_scale : 1.f) / l_sum : 0.f;
      if (bar_or_softmax(!ok)) { ok = false; break; }  // also publishes alpha_s
      const bool last = walk.pos >= walk.hi;
      if (last) {
        tc_fence_before();
        if (lane == 0) mbar_arrive(o_last);
      }
      tc_fence_after();
      if (live) {
        if (direct)
          p.lse[(int64_t)sg.row * kHeads + h] =
              m_used == -INFINITY ? -INFINITY : (m_used * c_log2 - kPShift + log2f(l_sum)) * 0.69314718055994531f;
        else
          reinterpret_cast<float2*>(p.ml)[(int64_t)sg.slot * kHeads + h] = make_float2(m_used * c_log2 - kPShift, l_sum);
      }
      // turned in the P buffer (free: every PV has completed): 2-byte stores straight
      // from the lanes took 12 us a part
      uint8_t* turn = smem + kOffP + warp * 2048;
      const int end = last ? 4 : 12;  // the loaders write the rest of the last part
      if (direct)
        write_part<true>(0, end, lane_base, alpha_s, turn, p.out + (int64_t)sg.row * kPartO);
      else
        write_part<false>(0, end, lane_base, alpha_s, turn, p.opart + (int64_t)sg.slot * kPartO);
      tc_fence_before();
      bar_or_softmax(false);  // alpha_s and the P buffer are free for the next part
      if (lane == 0) mbar_arrive(o_free);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kQkWarp) tmem_dealloc(tmem, 512);
}

// 16 bytes, loaded where it is written: the compiler otherwise puts a round's loads
// behind one another to save registers (four rows of 20,000 tokens: 47.7 instead of
// 44.9 us; with one group, at two parts a row, the free order is as fast).
__device__ __forceinline__ uint4 ld_now(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Merge the parts of a row that crossed CTAs, or fill a row that sees no token:
// kHpc heads a CTA, 64 threads (8 dims each) a head, and kGroups groups of threads
// that take every such part, joined in a fixed order.
template <int kHpc, int kGroups>
__device__ __forceinline__ void combine_row(int row, const uint16_t* __restrict__ opart, const float* __restrict__ ml,
                                            int2 info, int inv, float latent_scale, uint16_t* out, float* lse) {
  __shared__ float acc_s[kGroups > 1 ? kGroups - 1 : 1][64][8];
  const int w = threadIdx.x >> 6, th = threadIdx.x & 63;
  const int h = blockIdx.y * kHpc + w % kHpc, grp = w / kHpc;
  const int parts = info.y;
  uint16_t* dst = out + ((int64_t)row * kHeads + h) * kValue + th * 8;
  if (parts == 0) {
    if (grp == 0) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(0, 0);
      *reinterpret_cast<uint2*>(dst + 4) = make_uint2(0, 0);
      if (th == 0) lse[(int64_t)row * kHeads + h] = -INFINITY;
    }
    return;
  }
  auto slot_of = [&](int s) -> int64_t {
    return inv ? (int64_t)info.x + s : (s == 0 ? 2 * (int64_t)info.x + 1 : 2 * ((int64_t)info.x + s));
  };
  const float2* ml2 = reinterpret_cast<const float2*>(ml);
  float M = -INFINITY;
  bool bad = false;  // NaN logits in a part
  for (int s = th & 31; s < parts; s += 32) {
    const float x = ml2[slot_of(s) * kHeads + h].x;
    bad |= x != x;
    M = fmaxf(M, x);
  }
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (__any_sync(0xffffffffu, bad)) M = __int_as_float(0x7FC00000);
  float den = 0.f, a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  constexpr int kU = 4;
  for (int s0 = grp; s0 < parts; s0 += kU * kGroups) {
    float2 v[kU];
    uint4 x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int s = s0 + u * kGroups;
      v[u] = make_float2(-INFINITY, 0.f);
      x[u] = make_uint4(0, 0, 0, 0);
      if (s < parts) {
        const int64_t slot = slot_of(s);
        v[u] = ml2[slot * kHeads + h];
        const uint16_t* from = opart + (slot * kHeads + h) * kValue + th * 8;
        if (kGroups > 1)
          x[u] = ld_now(from);
        else
          x[u] = *reinterpret_cast<const uint4*>(from);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float wt = v[u].x == -INFINITY ? 0.f : ex2f(v[u].x - M) * v[u].y;  // a part is normalised by its own sum
      den += wt;
      const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&xs[i]));
        a[2 * i] = fmaf(wt, f.x, a[2 * i]);
        a[2 * i + 1] = fmaf(wt, f.y, a[2 * i + 1]);
      }
    }
  }
  if constexpr (kGroups > 1) {
    __shared__ float sum_s[kGroups - 1];
    if (grp > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc_s[grp - 1][th][i] = a[i];
      if (th == 0) sum_s[grp - 1] = den;
    }
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int g = 0; g < kGroups - 1; ++g) {
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] += acc_s[g][th][i];
      den += sum_s[g];
    }
  }
  const float inv_den = M == -INFINITY ? 0.f : latent_scale / den;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(a[2 * i] * inv_den, a[2 * i + 1] * inv_den);
    o[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
  *reinterpret_cast<uint2*>(dst + 4) = make_uint2(o[2], o[3]);
  if (th == 0) lse[(int64_t)row * kHeads + h] = M == -INFINITY ? -INFINITY : (M + log2f(den)) * 0.69314718055994531f;
}

template <int kHpc, int kGroups>
__global__ void __launch_bounds__(64 * kHpc * kGroups) dense_combine_kernel(
    const uint16_t* __restrict__ opart, const float* __restrict__ ml, const int2* __restrict__ row_info, int inv,
    float latent_scale, uint16_t* out, float* lse) {
  grid_dep_wait();  // the parts come from the previous kernel
  const int row = blockIdx.x;
  const int2 info = row_info[row];
  if (info.y == 1) return;  // written already
  combine_row<kHpc, kGroups>(row, opart, ml, info, inv, latent_scale, out, lse);
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

int64_t max_tiles(int rows, int max_len) { return (int64_t)rows * (((int64_t)std::max(max_len, 0) + kTile - 1) / kTile); }

// Partial slots for `rows` rows of at most max_len tokens.
int64_t dense_slots(int rows, int max_len, bool inv) {
  if (inv) {
    const int64_t tiles = max_tiles(1, max_len);
    return std::max<int64_t>(1, rows * ((tiles + kInvariantTiles - 1) / kInvariantTiles));
  }
  return 2 * std::max<int64_t>(1, std::min<int64_t>(kMaxGrid, max_tiles(rows, max_len)));
}

}  // namespace

size_t dense_mla_workspace_bytes(int rows, int max_len, bool inv) {
  const int64_t slots = dense_slots(rows, max_len, inv);
  return query_f16_bytes(rows) + al256((size_t)rows * sizeof(int2)) + al256((size_t)slots * kPartO * 2) + al256((size_t)slots * kHeads * 8);
}

dsa_status_t launch_dense_mla(const dsa_paged_cache_t& c, const dsa_batch_t& bt, const uint16_t* q_mla, float sm_scale,
                              bool inv, uint16_t* out, float* lse, void* workspace, int32_t* status, cudaStream_t st) {
  const int rows = bt.batch * bt.queries_per_seq;
  const int64_t slots = dense_slots(rows, bt.max_seq_len, inv);
  const bool nv = c.latent_format == DSA_LATENT_NVFP4;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    if (cuda_status(cudaFuncSetAttribute(dense_mla_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes)) != DSA_OK ||
        cuda_status(cudaFuncSetAttribute(dense_mla_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes)) != DSA_OK)
      return DSA_ERR_CUDA;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  uint16_t* q16 = nullptr;
  float* q_inv = nullptr;
  if (launch_query_f16(q_mla, nullptr, rows, workspace, &q16, &q_inv, st) != DSA_OK) return DSA_ERR_CUDA;
  CUtensorMap qmap;
  const uint64_t dims[2] = {(uint64_t)kLatent, (uint64_t)rows * kHeads};
  const uint64_t strides[1] = {(uint64_t)kLatent * 2};
  const uint32_t box[2] = {64, (uint32_t)kHeads};
  if (!encode_tmap(&qmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, q16, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return DSA_ERR_CUDA;
  uint8_t* w = static_cast<uint8_t*>(workspace) + query_f16_bytes(rows);
  DenseParams p = {};
  p.row_info = reinterpret_cast<int2*>(w);
  w += al256((size_t)rows * sizeof(int2));
  p.opart = reinterpret_cast<uint16_t*>(w);
  w += al256((size_t)slots * kPartO * 2);
  p.ml = reinterpret_cast<float*>(w);
  p.latent_base = static_cast<const uint8_t*>(c.base) + c.latent_off;
  p.row_stride = c.row_stride;
  p.num_blocks = c.num_blocks;
  p.block_table = bt.block_table;
  p.max_blocks = bt.max_blocks_per_seq;
  p.seq_lens = bt.seq_lens;
  p.nq = bt.queries_per_seq;
  p.cap = (int)std::min<int64_t>((int64_t)bt.max_blocks_per_seq * kBlock, bt.max_seq_len);
  p.rows = rows;
  p.logit_scale_log2 = sm_scale * c.latent_scale * 1.4426950408889634f;
  p.latent_scale = c.latent_scale;
  p.q16 = q16;
  p.q_inv = q_inv;
  p.out = out;
  p.lse = lse;
  p.unit = inv ? kInvariantTiles : 0;
  p.status = status;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(max_tiles(rows, p.cap), std::min(num_sms(), kMaxGrid)));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)want);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  if (cuda_status(cudaLaunchKernelEx(&cfg, nv ? dense_mla_kernel<true> : dense_mla_kernel<false>, qmap, p)) != DSA_OK)
    return DSA_ERR_CUDA;
  // Few rows have many parts each: a CTA a head, the parts over 16 or 4 groups of threads; else four heads a CTA.
  // The whole call with 16 groups, 4 groups and four heads, us: one row of 60,000 tokens 36, 54 and 80; two of 3,000
  // 25 and 29; four of 20,000 50 and 49; 16 of 6,000 71, 51 and 55; 32 of 8,000: 4 groups 90, four heads 87.
  // The groups' order of a row's sum differs, so the batch-invariant mode takes one whatever the batch.
  const bool wide = !inv && rows <= 2, one = inv || rows <= 16;
  auto combine = wide  ? dense_combine_kernel<1, 16>
                 : one ? dense_combine_kernel<1, 4>
                       : dense_combine_kernel<4, 1>;
  cfg.gridDim = dim3((unsigned)rows, (unsigned)(one ? kHeads : kHeads / 4));
  cfg.blockDim = dim3(wide ? 1024 : 256);
  cfg.dynamicSmemBytes = 0;
  count_launches(1);
  if (cuda_status(cudaLaunchKernelEx(&cfg, combine, (const uint16_t*)p.opart, (const float*)p.ml,
                                     (const int2*)p.row_info, inv ? 1 : 0, c.latent_scale, out, lse)) != DSA_OK)
    return DSA_ERR_CUDA;
  return launch_status();
}

}  // namespace dsa
