// mass.cu — the attention weight that each cached token received.
//
// For every sequence b and token t, summed over its query rows j and the 96 heads:
//   mass_out[b][t] = mass_in[b][t] + sum_j sum_h exp(sm_scale * latent_scale * (q[r][h] . c_t) - lse[r][h])
// over the tokens a row attended to: every visible one (the dense attention's
// LSE), or those its top-k selected (the sparse attention's).  The running total
// is what cache eviction ranks tokens by.
//
// attention_weights_kernel (persistent, one CTA per SM, 19 warps): the rows'
// tiles of 128 tokens lie on one line, equal runs of it to every CTA.
//   * S^T = K Q^T with the tokens on M = 128 rows and the heads on N = 96: the
//     sum over heads then stays inside a thread, and no MMA row is wasted.  Q
//     (110 KB, fp16 from query.cu) stays in shared memory while a CTA works on a
//     row.
//   * The widened keys, the A operand, go to TMEM (288 columns; two S tiles take
//     192 more), not to shared memory: storing 147 KB a tile there and reading
//     it back took most of the shared-memory port's cycles.
//   * warps 16, 17 find the tokens' records (index, page, slot; two stages ahead)
//     and copy them raw, 16 bytes a lane, into a ring of 64-token stages; a record
//     is padded by 16 bytes there, so that 32 lanes reading one 16-byte piece of
//     32 records meet all banks.
//   * warps 4..15 (thread = token, the TMEM lane; three sets of four warps, 192
//     dims each) widen them exactly to fp16; a set's three blocks are one step of
//     the MMA issuer (a step a block, or two sets, left it waiting).
//   * warps 0..3, one thread a token: sum over heads of 2^(s c_h - lse_h log2 e), from
//     one of two S tiles in TMEM while the next is computed (c_h: log2 units per unit
//     of S, a factor a head).  The exponential is ex2.approx, right to 2^-22, in whose
//     argument the fp32 products' sum is the larger error.  A token that the row does
//     not see, or whose page lies outside the pool, gets 0.
// With one row per sequence and no selection the kernel adds the running total
// itself; otherwise the rows' weights go to the workspace and a second kernel
// adds them, row after row, so the order of the sums is fixed:
// weights_reduce_kernel (every visible token) or weights_scatter_kernel (the
// selected ones: a CTA owns 4,096 tokens of a sequence in shared memory).
// What bounds it: a set's three key blocks exist once, so its converters and its
// MMAs take turns (per tile about 8,000 warp instructions, 42 % of the issue slots;
// the tensor pipe is active 36 % of the time).  16 contexts of 16K to 64K tokens,
// NVFP4: 89 us, 815 TFLOP/s, 2.7 TB/s; 64 rows of one 32,770-token context: 254 us,
// 912 TFLOP/s.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "run.cuh"

namespace dsa {

namespace {

constexpr int kTok = 128;                        // tokens per tile
constexpr int kDB = kLatent / 64;                // 9 blocks of 64 dims
constexpr int kQBlockBytes = kHeads * 128;       // 12,288
constexpr int kStageTok = 64;                    // tokens per stage of raw records
constexpr int kNvRec = kValue / 2 + kValue / 16 + (kLatent - kValue);
constexpr int kThreads = 19 * 32;                // epilogue 0-3, converters 4-15, producers 16-17, MMA issuer 18
constexpr int kConvWarp0 = 4;
constexpr int kProdWarp0 = 16;
constexpr int kMmaWarp = 18;
constexpr int kSets = 3;                         // of converters, four warps each
constexpr int kSetBlocks = kDB / kSets;          // blocks of a set
static_assert(kSets * kSetBlocks == kDB && kConvWarp0 + 4 * kSets == kProdWarp0, "converter split");
constexpr int kSCols = kHeads;                   // TMEM: two S tiles, then nine blocks of keys
constexpr int kKCol = 2 * kSCols;
constexpr int kTmemCols = 512;
static_assert(kKCol + 32 * kDB <= kTmemCols, "TMEM columns");

template <bool kNV>
struct Raw {
  static constexpr int kRec = kNV ? kNvRec : kLatent;
  static constexpr int kStride = kRec + 16;
  static constexpr int kBytes = kStageTok * kStride;  // 23,552 or 37,888
  static constexpr int kStages = kNV ? 4 : 3;
};

constexpr int kOffQ = 0;
constexpr int kOffRaw = kDB * kQBlockBytes;                    // 110,592
constexpr int kRawBytes = Raw<false>::kStages * Raw<false>::kBytes;  // 113,664
static_assert(Raw<true>::kStages * Raw<true>::kBytes <= kRawBytes, "raw ring");
constexpr int kOffHead = kOffRaw + kRawBytes;                  // the heads' LSE (log2), then log2 units per unit of S
constexpr int kOffBars = kOffHead + 2 * kHeads * 4;
constexpr int kNumBars = 2 * 4 + 2 * kSets + 6;
constexpr int kOffMisc = (kOffBars + kNumBars * 8 + 15) / 16 * 16;
constexpr size_t kSmemBytes = 1024 + kOffMisc + 16 + 32 * 8;
static_assert(kOffHead % 16 == 0 && kHeads % 4 == 0 && kOffBars % 8 == 0, "alignment");
static_assert(kSmemBytes <= 232448, "shared memory");

struct MassParams {
  const uint8_t* latent_base;
  int64_t row_stride;
  int32_t num_blocks;
  const int32_t* block_table;
  int32_t max_blocks;
  const int32_t* seq_lens;
  int32_t nq, cap, rows;
  const int32_t* idx;   // [rows][k] or null: every visible token
  int32_t k;
  float scale_log2;     // sm_scale * latent_scale * log2(e)
  const float* q_inv;   // [rows][96]: the inverse of the power of two in the fp16 queries
  const float* lse;     // [rows][96]
  const float* mass_in; // [batch][ld] (direct only)
  float* out;           // direct: mass_out [batch][ld]; else the rows' weights [rows][ld]
  int64_t ld;
  int32_t direct;
  int32_t* status;
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void bar_epilogue() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool bar_or_epilogue(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, 1, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

struct Tiles {  // a run's tiles, one after another
  const MassParams& p;
  int row, limit;  // limit: tokens (or entries) of `row`
  int64_t start, pos, hi;

  __device__ int visible(int r) const {
    int len = p.seq_lens[r / p.nq];
    len = len < 0 ? 0 : (len > p.cap ? p.cap : len);
    return visible_len(len, p.nq, r % p.nq);
  }
  __device__ int items(int r) const { return p.idx ? p.k : visible(r); }
  // The next tile: its row and first token (or entry); false behind the run.
  __device__ bool next(int& r, int& first, int& count) {
    if (pos >= hi) return false;
    if (limit < 0) limit = items(row);
    while (pos >= start + (limit + kTok - 1) / kTok) {
      start += (limit + kTok - 1) / kTok;
      limit = items(++row);
    }
    r = row;
    first = (int)(pos - start) * kTok;
    count = min(kTok, limit - first);
    ++pos;
    return true;
  }
};

// What a lane without a token reads.
__device__ const uint4 zero_record[kLatent / 16] = {};

template <bool kNV>
__global__ void __launch_bounds__(kThreads, 1)
    attention_weights_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ MassParams p) {
  using R = Raw<kNV>;
  constexpr int kRec = R::kRec, kStages = R::kStages;
  constexpr uint32_t kIdesc = make_idesc(kFmtF16, kFmtF16, 0, 0, kTok, kHeads);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + kOffBars;
  auto raw_full = [&](uint32_t s) { return bars + 8u * s; };
  auto raw_empty = [&](uint32_t s) { return bars + 8u * (4 + s); };
  auto k_full = [&](uint32_t g) { return bars + 8u * (8 + g); };
  auto k_empty = [&](uint32_t g) { return bars + 8u * (8 + kSets + g); };
  const uint32_t bars2 = bars + 8u * (8 + 2 * kSets);
  auto s_full = [&](uint32_t s) { return bars2 + 8u * s; };
  auto s_empty = [&](uint32_t s) { return bars2 + 16 + 8u * s; };
  const uint32_t q_full = bars2 + 32, drain = bars2 + 40;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int64_t* scratch = reinterpret_cast<int64_t*>(smem + kOffMisc + 16);
  float* lse_s = reinterpret_cast<float*>(smem + kOffHead);
  float* unit_s = lse_s + kHeads;  // logits in log2 units per unit of S
  const int warp = warp_number(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(raw_full(s), 64);  // both producer warps' lanes
      mbar_init(raw_empty(s), 2 * kSets);  // the converters of 64 tokens
    }
    for (int g = 0; g < kSets; ++g) {
      mbar_init(k_full(g), 4);
      mbar_init(k_empty(g), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(s_empty(s), 4);
    }
    mbar_init(q_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmap_q);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  // The queries come from the previous kernel, which let this one start only when
  // all before it had completed: the lengths can be read before the wait.
  Tiles tiles{p, 0, -1, 0, 0, 0};
  {
    const Run run = find_run<kThreads>(
        p.rows, 0, scratch, [&](int r) -> int64_t { return (tiles.items(r) + kTok - 1) / kTok; },
        [](int, int64_t, int64_t, int64_t) {});
    tiles.row = run.row;
    tiles.start = run.start;
    tiles.pos = run.pos;
    tiles.hi = run.hi;
  }
  grid_dep_wait();
  grid_dep_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  int row = -1, first = 0, count = 0;

  if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issuer (the whole warp runs, one lane issues)
    const uint64_t q_desc = smem_desc(sbase + kOffQ, 16, 1024, kLayoutSw128);
    const uint32_t q_lo = (uint32_t)q_desc, hi = (uint32_t)(q_desc >> 32);
    uint32_t it = 0, segs = 0;
    int cur = -1;
    bool ok = true;
    while (ok) {
      if (!__all_sync(0xffffffffu, tiles.next(row, first, count))) break;
      row = __shfl_sync(0xffffffffu, row, 0);
      const uint32_t b = it & 1;
      if (row != cur) {
        // Q may go once the previous row's last S tile is complete
        if (it > 0) ok = mbar_wait_warp(s_full(b ^ 1), ((it - 1) >> 1) & 1, abort_flag, p.status);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(q_full, kDB * kQBlockBytes);
          for (int kb = 0; kb < kDB; ++kb)
            tma_load_2d(sbase + kOffQ + kb * kQBlockBytes, &tmap_q, kb * 64, row * kHeads, q_full);
        }
        __syncwarp();
        ok = mbar_wait_warp(q_full, segs & 1, abort_flag, p.status);
        ++segs;
        cur = row;
      }
      ok = ok && mbar_wait_warp(s_empty(b), ((it >> 1) & 1) ^ 1, abort_flag, p.status);
#pragma unroll 1
      for (int g = 0; ok && g < kSets; ++g) {
        ok = mbar_wait_warp(k_full(g), it & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 1
          for (int kb = g * kSetBlocks; kb < (g + 1) * kSetBlocks; ++kb) {
            const uint32_t a_t = tmem + kKCol + 32 * kb, b_lo = q_lo + kb * (kQBlockBytes / 16);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_tmem_a(tmem + b * kSCols, a_t + 8 * kk, desc64(b_lo + 2 * kk, hi), kIdesc, (kb | kk) ? 1u : 0u);
          }
          mma_commit(k_empty(g));
          if (g == kSets - 1) mma_commit(s_full(b));
        }
        __syncwarp();
      }
      ++it;
    }
    if (elect_one()) {
      if (segs > 0) mbar_wait_drain(q_full, (segs - 1) & 1, 10000000ull);  // no copy is in flight at the exit
      mma_commit(drain);  // every MMA completes before TMEM is released
      mbar_wait_drain(drain, 0, 10000000ull);
    }
  } else if (warp >= kProdWarp0) {
    // ------------------------------------------------ producers: raw records into the ring
    // Lane: one of the warp's 32 tokens of a stage; a token's index is read two
    // stages ahead, its page one.
    const int pw = warp - kProdWarp0;
    const uint8_t* rec = nullptr;
    int part = 0, row_a = 0, tok_a = -1, tok_b = -1, page_b = -1, limit = 0, limit_row = -1;
    bool have_t = false, have_a = false, have_b = false, have = false;
    auto step_token = [&]() {
      if (part == 0) have_t = tiles.next(row, first, count);
      have_a = have_t;
      row_a = row;
      tok_a = -1;
      const int e = part * kStageTok + pw * 32 + lane;
      if (have_a && e < count) tok_a = p.idx ? p.idx[(int64_t)row * p.k + first + e] : first + e;
      part ^= 1;
    };
    auto step_page = [&]() {
      have_b = have_a;
      tok_b = -1;
      page_b = -1;
      if (!have_b) return;
      if (row_a != limit_row) {
        limit_row = row_a;
        limit = tiles.visible(row_a);
      }
      if (tok_a >= 0 && tok_a < limit) {
        tok_b = tok_a;
        page_b = p.block_table[(int64_t)(row_a / p.nq) * p.max_blocks + tok_a / kBlock];
      } else if (tok_a >= 0) {
        report(p.status, DSA_ERR_BOUNDS);  // an entry that its row does not see
      }
    };
    auto step_record = [&]() {
      have = have_b;
      rec = reinterpret_cast<const uint8_t*>(zero_record);  // no token: zeros
      if (tok_b < 0) return;
      if ((uint32_t)page_b < (uint32_t)p.num_blocks)
        rec = p.latent_base + (int64_t)page_b * p.row_stride + tok_b % kBlock * kRec;
      else
        report(p.status, DSA_ERR_BOUNDS);
    };
    step_token();
    step_page();
    step_token();
    bool ok = true;
    for (uint32_t n = 0;; ++n) {
      step_record();
      if (!have) break;
      step_page();
      step_token();
      const uint32_t slot = n % kStages;
      ok = mbar_wait_warp(raw_empty(slot), ((n / kStages) & 1) ^ 1, abort_flag, p.status);
      if (!ok) break;
      const uint32_t dst = sbase + kOffRaw + slot * R::kBytes + pw * 32 * R::kStride;
      const uint64_t mine = reinterpret_cast<uint64_t>(rec);
#pragma unroll 8
      for (int t = 0; t < 32; ++t) {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, mine, t));
#pragma unroll
        for (int u = 0; u < (kRec + 511) / 512; ++u)
          if (lane + 32 * u < kRec / 16) cp_async16(dst + t * R::kStride + 16 * (lane + 32 * u), src + 16 * (lane + 32 * u));
      }
      cp_async_arrive(raw_full(slot));
    }
    cp_async_wait_all();  // no copy is in flight at the exit
  } else if (warp >= kConvWarp0) {
    // ------------------------------------------------ converters: raw records -> fp16 keys in TMEM (thread = token)
    const int q = warp & 3, g = (warp - kConvWarp0) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16) + kKCol;
    const uint8_t* mine = smem + kOffRaw + ((q & 1) * 32 + lane) * R::kStride;
    const int64_t todo = tiles.hi - tiles.pos;
    bool ok = true;
    for (uint32_t it = 0; ok && (int64_t)it < todo; ++it) {
      const uint32_t st = 2 * it + (q >> 1), slot = st % kStages;
      ok = mbar_wait_warp(raw_full(slot), (st / kStages) & 1, abort_flag, p.status);
      if (!ok) break;
      const uint8_t* rec = mine + slot * R::kBytes;
#pragma unroll 1
      for (int kb = g * kSetBlocks; kb < (g + 1) * kSetBlocks; ++kb) {
        uint32_t o[32];
        if (kNV && kb < kDB - 1) {
          const uint4 a = *reinterpret_cast<const uint4*>(rec + 32 * kb), b = *reinterpret_cast<const uint4*>(rec + 32 * kb + 16);
          const uint32_t s = *reinterpret_cast<const uint32_t*>(rec + kValue / 2 + 4 * kb);  // four units' scales
          nvfp4x16_to_f16x16(a.x, a.y, s & 0xFFu, *reinterpret_cast<uint32_t(*)[8]>(o));
          nvfp4x16_to_f16x16(a.z, a.w, (s >> 8) & 0xFFu, *reinterpret_cast<uint32_t(*)[8]>(o + 8));
          nvfp4x16_to_f16x16(b.x, b.y, (s >> 16) & 0xFFu, *reinterpret_cast<uint32_t(*)[8]>(o + 16));
          nvfp4x16_to_f16x16(b.z, b.w, s >> 24, *reinterpret_cast<uint32_t(*)[8]>(o + 24));
        } else {
          const uint8_t* c = rec + (kNV ? kValue / 2 + kValue / 16 : 64 * kb);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            e4m3x16_to_f16x16(*reinterpret_cast<const uint4*>(c + 16 * u), *reinterpret_cast<uint32_t(*)[8]>(o + 8 * u));
        }
        if (kb == g * kSetBlocks) {
          ok = mbar_wait_warp(k_empty(g), (it & 1) ^ 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st32(lane_base + 32 * kb, o);
      }
      if (!ok) break;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(k_full(g));
        mbar_arrive(raw_empty(slot));
      }
    }
  } else {
    // ------------------------------------------------ weights (thread = token)
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const int tid = threadIdx.x;
    uint32_t it = 0;
    int cur = -1;
    bool ok = true, attended = false;  // attended: a head of the row has an LSE above -inf
    while (tiles.next(row, first, count)) {
      const uint32_t b = it & 1;
      if (row != cur) {
        bar_epilogue();  // the previous row's values have been read
        attended = false;
        if (tid < kHeads) {
          const float l = p.lse[(int64_t)row * kHeads + tid];
          lse_s[tid] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;  // no token attended: no weight
          unit_s[tid] = p.scale_log2 * p.q_inv[(int64_t)row * kHeads + tid];
          attended = l != -INFINITY;
        }
        attended = bar_or_epilogue(attended);
        cur = row;
      }
      ok = ok && mbar_wait_warp(s_full(b), (it >> 1) & 1, abort_flag, p.status);
      ++it;
      if (!ok) continue;
      tc_fence_after();
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kHeads / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(lane_base + b * kSCols + 32 * c, r);
        tmem_ld_wait();
        if (c == kHeads / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_empty(b));
        }
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 l = *reinterpret_cast<const float4*>(lse_s + 32 * c + j);
          const float4 u = *reinterpret_cast<const float4*>(unit_s + 32 * c + j);
          sum[0] += ex2f(fmaf(__uint_as_float(r[j]), u.x, -l.x));
          sum[1] += ex2f(fmaf(__uint_as_float(r[j + 1]), u.y, -l.y));
          sum[2] += ex2f(fmaf(__uint_as_float(r[j + 2]), u.z, -l.z));
          sum[3] += ex2f(fmaf(__uint_as_float(r[j + 3]), u.w, -l.w));
        }
      }
      if (tid < count) {
        // an entry of -1, one that the row does not see and a page outside the pool (the producers report the last
        // two) have no weight, whatever the products of their zeros give; nor has any token of a row that attended
        // to nothing, though its pages may never have been written (NaN codes)
        const int64_t at = (int64_t)row * p.ld + first + tid;  // direct: one row per sequence
        const int tok = p.idx ? p.idx[at] : first + tid;
        bool seen = attended && tok >= 0 && (!p.idx || tok < tiles.visible(row));
        if (seen) seen = (uint32_t)p.block_table[(int64_t)(row / p.nq) * p.max_blocks + tok / kBlock] < (uint32_t)p.num_blocks;
        float w = seen ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f;
        if (p.direct && p.mass_in) w += p.mass_in[at];
        p.out[at] = w;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// mass_out[b][t] = mass_in[b][t] + the rows' weights of token t in row order, every token below the length.
__global__ void __launch_bounds__(256) weights_reduce_kernel(const float* __restrict__ weights, int64_t ldw,
                                                             const int32_t* seq_lens, int nq, int cap,
                                                             const float* mass_in, float* mass_out, int64_t ld) {
  grid_dep_wait();
  const int b = blockIdx.x, t = blockIdx.y * 256 + threadIdx.x;
  int len = seq_lens[b];
  len = len < 0 ? 0 : (len > cap ? cap : len);
  if (t >= len) return;
  float acc = mass_in ? mass_in[(int64_t)b * ld + t] : 0.f;
  const float* w = weights + (int64_t)b * nq * ldw + t;
  // row j sees the first len - (nq - 1) + j tokens
  const int j0 = max(0, t - len + nq);
  int j = j0;
  for (; j + 8 <= nq; j += 8) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = w[(int64_t)(j + u) * ldw];
#pragma unroll
    for (int u = 0; u < 8; ++u) acc += v[u];
  }
  for (; j < nq; ++j) acc += w[(int64_t)j * ldw];
  mass_out[(int64_t)b * ld + t] = acc;
}

// The same for selected tokens: a CTA holds 4,096 tokens' totals of a sequence
// and adds the rows' entries that fall on them, one row after another.  An index
// that a row lists twice has the same weight twice, so the order of its two
// additions cannot change the sum.
constexpr int kScatterTokens = 4096;
__global__ void __launch_bounds__(512) weights_scatter_kernel(const float* __restrict__ weights,
                                                              const int32_t* __restrict__ idx, int k,
                                                              const int32_t* seq_lens, int nq, int cap,
                                                              const float* mass_in, float* mass_out, int64_t ld) {
  __shared__ float acc[kScatterTokens];
  grid_dep_wait();
  const int b = blockIdx.x, t0 = blockIdx.y * kScatterTokens;
  int len = seq_lens[b];
  len = len < 0 ? 0 : (len > cap ? cap : len);
  const int n = min(kScatterTokens, len - t0);
  if (n <= 0) return;
  for (int i = threadIdx.x; i < n; i += 512) acc[i] = mass_in ? mass_in[(int64_t)b * ld + t0 + i] : 0.f;
  for (int j = 0; j < nq; ++j) {
    __syncthreads();
    const int64_t at = ((int64_t)b * nq + j) * k;
    for (int i = threadIdx.x; i < k; i += 512) {
      const int t = idx[at + i] - t0;
      if (t >= 0 && t < n) atomicAdd(&acc[t], weights[at + i]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 512) mass_out[(int64_t)b * ld + t0 + i] = acc[i];
}

int64_t round4(int64_t x) { return (x + 3) & ~int64_t(3); }

}  // namespace

size_t mass_workspace_bytes(int rows, int max_len, int k) {
  // the fp16 queries and the rows' weights (one row per sequence without a selection needs none, but the query
  // does not know the batch)
  const int64_t ld = k > 0 ? k : round4(std::max(max_len, 1));
  return query_f16_bytes(rows) + (((size_t)rows * ld * 4 + 255) & ~size_t(255));
}

dsa_status_t launch_attention_mass(const dsa_paged_cache_t& c, const dsa_batch_t& bt, const uint16_t* q_mla,
                                   const float* lse, const int32_t* idx, int k, float sm_scale, const float* mass_in,
                                   float* mass_out, int64_t ld, void* workspace, int32_t* status, cudaStream_t st) {
  const int rows = bt.batch * bt.queries_per_seq;
  const bool nv = c.latent_format == DSA_LATENT_NVFP4;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    if (cuda_status(cudaFuncSetAttribute(attention_weights_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes)) != DSA_OK ||
        cuda_status(cudaFuncSetAttribute(attention_weights_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes)) != DSA_OK)
      return DSA_ERR_CUDA;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  uint16_t* q16 = nullptr;
  float* q_inv = nullptr;
  if (launch_query_f16(q_mla, lse, rows, workspace, &q16, &q_inv, st) != DSA_OK) return DSA_ERR_CUDA;
  CUtensorMap qmap;
  const uint64_t dims[2] = {(uint64_t)kLatent, (uint64_t)rows * kHeads};
  const uint64_t strides[1] = {(uint64_t)kLatent * 2};
  const uint32_t box[2] = {64, (uint32_t)kHeads};
  if (!encode_tmap(&qmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, q16, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return DSA_ERR_CUDA;
  MassParams p = {};
  p.latent_base = static_cast<const uint8_t*>(c.base) + c.latent_off;
  p.row_stride = c.row_stride;
  p.num_blocks = c.num_blocks;
  p.block_table = bt.block_table;
  p.max_blocks = bt.max_blocks_per_seq;
  p.seq_lens = bt.seq_lens;
  p.nq = bt.queries_per_seq;
  p.cap = (int)std::min<int64_t>((int64_t)bt.max_blocks_per_seq * kBlock, bt.max_seq_len);
  p.rows = rows;
  p.idx = idx;
  p.k = k;
  p.scale_log2 = sm_scale * c.latent_scale * 1.4426950408889634f;
  p.lse = lse;
  p.mass_in = mass_in;
  p.direct = !idx && p.nq == 1;
  p.q_inv = q_inv;
  p.out = p.direct ? mass_out : reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + query_f16_bytes(rows));
  p.ld = p.direct ? ld : (idx ? k : round4(std::max(bt.max_seq_len, 1)));
  p.status = status;
  const int64_t most = (int64_t)rows * (((idx ? k : p.cap) + kTok - 1) / kTok);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(most, num_sms())));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launches(1);
  if (cuda_status(cudaLaunchKernelEx(&cfg, nv ? attention_weights_kernel<true> : attention_weights_kernel<false>, qmap,
                                     p)) != DSA_OK)
    return DSA_ERR_CUDA;
  if (p.direct || p.cap == 0) return launch_status();
  const int per = idx ? kScatterTokens : 256;
  cfg.gridDim = dim3((unsigned)bt.batch, (unsigned)((p.cap + per - 1) / per));
  cfg.blockDim = dim3(idx ? 512 : 256);
  cfg.dynamicSmemBytes = 0;
  count_launches(1);
  cudaError_t e;
  if (idx)
    e = cudaLaunchKernelEx(&cfg, weights_scatter_kernel, (const float*)p.out, idx, k, bt.seq_lens, p.nq, p.cap, mass_in,
                           mass_out, ld);
  else
    e = cudaLaunchKernelEx(&cfg, weights_reduce_kernel, (const float*)p.out, p.ld, bt.seq_lens, p.nq, p.cap, mass_in,
                           mass_out, ld);
  if (cuda_status(e) != DSA_OK) return DSA_ERR_CUDA;
  return launch_status();
}

}  // namespace dsa
