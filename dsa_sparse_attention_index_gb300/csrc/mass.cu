// mass.cu — the attention weight that each cached token received.
//
// For every sequence b and token t, summed over its query rows j and the 96 heads:
//   mass_out[b][t] = mass_in[b][t] + sum_j sum_h exp(sm_scale * latent_scale * (q[r][h] . c_t) - lse[r][h])
// over the tokens a row attended to: every visible one (the dense attention's
// LSE), or those its top-k selected (the sparse attention's).  The running total
// is what cache eviction ranks tokens by.
//
// attention_weights_kernel (persistent, one CTA per SM, 13 warps): the rows'
// tiles of 128 tokens lie on one line, equal runs of it to every CTA.
//   * S^T = K Q^T with the tokens on M = 128 rows and the heads on N = 96: the
//     sum over heads then stays inside a thread, and no MMA row is wasted.  Q
//     (110 KB) stays in shared memory while a CTA works on a row; the tiles
//     stream past it in stages of three 64-dim blocks (two stages).
//   * warps 4..11 load the tiles' records a whole tile ahead in registers (two
//     lanes a token, 16-byte loads, contiguous or gathered alike), widen them
//     exactly to bf16 and store them 128-byte swizzled, as the attention does.
//   * warps 0..3, one thread a token: sum over heads of 2^(s c - lse c'), from
//     one of two S tiles in TMEM while the next is computed.
// With one row per sequence and no selection the kernel adds the running total
// itself; otherwise the rows' weights go to the workspace and a second kernel
// adds them, row after row, so the order of the sums is fixed:
// weights_reduce_kernel (every visible token) or weights_scatter_kernel (the
// selected ones: a CTA owns 4,096 tokens of a sequence in shared memory).
// What bounds it: the shared-memory port (per tile 36 x (4 KB of keys + 3 KB of
// Q) read and 147 KB written: 3,200 cycles at 128 B a cycle, against 1,730
// cycles of tensor time).
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
constexpr int kBlkBytes = kTok * 128;            // 16,384
constexpr int kStageBlocks = 3;
constexpr int kStagesPerTile = kDB / kStageBlocks;
constexpr int kStages = 2;
constexpr int kStageBytes = kStageBlocks * kBlkBytes;  // 49,152
constexpr int kNvRec = kValue / 2 + kValue / 16 + (kLatent - kValue);
constexpr int kThreads = 13 * 32;                // epilogue 0-3, loaders 4-11, MMA issuer 12
constexpr int kLoadWarp0 = 4;
constexpr int kLoadWarps = 8;
constexpr int kMmaWarp = 12;
constexpr int kSCols = 128;                      // columns between the two S tiles
constexpr int kTmemCols = 256;

constexpr int kOffQ = 0;
constexpr int kOffStage = kDB * kQBlockBytes;                  // 110,592
constexpr int kOffLse = kOffStage + kStages * kStageBytes;     // 208,896
constexpr int kOffBars = kOffLse + kHeads * 4;
constexpr int kNumBars = 2 * kStages + 6;
constexpr int kOffMisc = (kOffBars + kNumBars * 8 + 15) / 16 * 16;
constexpr size_t kSmemBytes = 1024 + kOffMisc + 256;
static_assert(kOffStage % 1024 == 0 && kOffBars % 8 == 0, "alignment");
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

struct Tiles {  // a run's tiles, one after another
  const MassParams& p;
  int row, limit;  // limit: tokens (or entries) of `row`
  int64_t start, pos, hi;

  __device__ int items(int r) const {
    if (p.idx) return p.k;
    int len = p.seq_lens[r / p.nq];
    len = len < 0 ? 0 : (len > p.cap ? p.cap : len);
    return visible_len(len, p.nq, r % p.nq);
  }
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

template <bool kNV>
__global__ void __launch_bounds__(kThreads, 1)
    attention_weights_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ MassParams p) {
  constexpr int kRec = kNV ? kNvRec : kLatent;
  constexpr uint32_t kIdesc = make_idesc(kFmtBF16, kFmtBF16, 0, 0, kTok, kHeads);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + kOffBars;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kStages + s); };
  auto s_full = [&](int s) { return bars + 8u * (2 * kStages + s); };
  auto s_empty = [&](int s) { return bars + 8u * (2 * kStages + 2 + s); };
  const uint32_t q_full = bars + 8u * (2 * kStages + 4), drain = bars + 8u * (2 * kStages + 5);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int64_t* scratch = reinterpret_cast<int64_t*>(smem + kOffMisc + 16);
  float* lse_s = reinterpret_cast<float*>(smem + kOffLse);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), kLoadWarps);
      mbar_init(empty(s), 1);
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
  grid_dep_wait();  // the LSE, the indices and the lengths may come from the previous kernel
  Tiles tiles{p, 0, -1, 0, 0, 0};
  {
    const Run run = find_run<kThreads>(
        p.rows, 1, 0, scratch, [&](int r) -> int64_t { return (tiles.items(r) + kTok - 1) / kTok; },
        [](int, int64_t, int64_t, int64_t) {});
    tiles.row = run.row;
    tiles.start = run.start;
    tiles.pos = run.pos;
    tiles.hi = run.hi;
  }
  grid_dep_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int row, first, count;

  if (warp == kMmaWarp) {
    if (lane == 0) {
      // ------------------------------------------------ MMA issuer
      const uint64_t q_desc = smem_desc(sbase + kOffQ, 16, 1024, kLayoutSw128);
      const uint32_t q_lo = (uint32_t)q_desc, hi = (uint32_t)(q_desc >> 32);
      const uint32_t st_lo = (uint32_t)smem_desc(sbase + kOffStage, 16, 1024, kLayoutSw128);
      uint32_t it = 0, stage = 0, segs = 0;
      int cur = -1;
      bool ok = true, q_pending = false;
      while (ok && tiles.next(row, first, count)) {
        const int b = it & 1;
        if (row != cur) {
          // Q may go once the previous row's last S tile is complete
          if (it > 0) ok = mbar_wait(s_full(b ^ 1), ((it - 1) >> 1) & 1, abort_flag, p.status);
          if (!ok) break;
          mbar_arrive_expect_tx(q_full, kDB * kQBlockBytes);
          for (int kb = 0; kb < kDB; ++kb)
            tma_load_2d(sbase + kOffQ + kb * kQBlockBytes, &tmap_q, kb * 64, row * kHeads, q_full);
          q_pending = true;
          ok = mbar_wait(q_full, segs & 1, abort_flag, p.status);
          if (!ok) break;
          q_pending = false;
          ++segs;
          cur = row;
        }
        ok = mbar_wait(s_empty(b), ((it >> 1) & 1) ^ 1, abort_flag, p.status);
        for (int g = 0; ok && g < kStagesPerTile; ++g, ++stage) {
          const uint32_t slot = stage % kStages;
          ok = mbar_wait(full(slot), (stage / kStages) & 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_lo = st_lo + slot * (kStageBytes / 16);
          const uint32_t b_lo = q_lo + g * (kStageBlocks * kQBlockBytes / 16);
#pragma unroll
          for (int j = 0; j < kStageBlocks; ++j)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16(tmem + b * kSCols, desc64(a_lo + j * (kBlkBytes / 16) + 2 * kk, hi),
                       desc64(b_lo + j * (kQBlockBytes / 16) + 2 * kk, hi), kIdesc, (g | j | kk) ? 1u : 0u);
          mma_commit(empty(slot));
        }
        if (!ok) break;
        mma_commit(s_full(b));
        ++it;
      }
      if (q_pending) mbar_wait_drain(q_full, segs & 1, 10000000ull);
      // every MMA completes before TMEM is released
      mma_commit(drain);
      mbar_wait_drain(drain, 0, 10000000ull);
    }
  } else if (warp >= kLoadWarp0) {
    // ------------------------------------------------ loaders: records -> bf16 stages
    // Lane (token, half) of 16 tokens a warp: 32 dims of each block.
    constexpr int kW = kNV ? 1 : 2;
    const int tok = (warp - kLoadWarp0) * 16 + (lane >> 1), half = lane & 1;
    uint4 buf[kDB - 1][kW], tail[2], sc[2];
    const uint8_t* rec = nullptr;
    // Three steps, each a tile ahead of the next: the token, its page, its record.
    int tok_a = -1, row_b = 0, tok_b = -1, page_b = -1;
    bool have_a = false, have_b = false, have = false;
    auto step_token = [&]() {
      have_a = tiles.next(row, first, count);
      tok_a = -1;
      if (have_a && tok < count) tok_a = p.idx ? p.idx[(int64_t)row * p.k + first + tok] : first + tok;
    };
    auto step_page = [&]() {
      have_b = have_a;
      tok_b = tok_a;
      page_b = -1;
      if (!have_b) return;
      row_b = row;
      if (tok_b >= 0) {
        if (tok_b >= p.cap || (p.idx && tok_b >= [&] {
              int len = p.seq_lens[row_b / p.nq];
              len = len < 0 ? 0 : (len > p.cap ? p.cap : len);
              return visible_len(len, p.nq, row_b % p.nq);
            }())) {
          report(p.status, DSA_ERR_BOUNDS);
          tok_b = -1;
        } else {
          page_b = p.block_table[(int64_t)(row_b / p.nq) * p.max_blocks + tok_b / kBlock];
        }
      }
    };
    auto step_record = [&]() {
      have = have_b;
      rec = nullptr;
      if (have && tok_b >= 0) {
        if (page_b >= 0 && page_b < p.num_blocks)
          rec = p.latent_base + (int64_t)page_b * p.row_stride + (tok_b % kBlock) * kRec;
        else
          report(p.status, DSA_ERR_BOUNDS);
      }
    };
    auto advance = [&]() {
      step_record();
      step_page();
      step_token();
    };
    auto ld = [&](int off) {
      return rec ? __ldg(reinterpret_cast<const uint4*>(rec + off)) : make_uint4(0, 0, 0, 0);
    };
    auto load_block = [&](int kb) {
      if (kb == kDB - 1) {
        constexpr int kTailOff = kNV ? kValue / 2 + kValue / 16 : kValue;
        tail[0] = ld(kTailOff + 32 * half);
        tail[1] = ld(kTailOff + 32 * half + 16);
      } else if (kNV) {
        buf[kb][0] = ld(32 * kb + 16 * half);
      } else {
        buf[kb][0] = ld(64 * kb + 32 * half);
        buf[kb][kW - 1] = ld(64 * kb + 32 * half + 16);
      }
    };
    auto load_scales = [&]() {
      if (kNV) {
        sc[0] = ld(kValue / 2);
        sc[1] = ld(kValue / 2 + 16);
      }
    };
    auto store_unit = [&](uint8_t* blk, int u, const uint32_t (&o)[8]) {
      const uint32_t off = (uint32_t)(tok * 128 + half * 64 + u * 32);
      *reinterpret_cast<uint4*>(blk + swz128(off)) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(blk + swz128(off + 16)) = make_uint4(o[4], o[5], o[6], o[7]);
    };
    step_token();
    step_page();
    step_token();
    advance();
    if (have) {
      load_scales();
#pragma unroll
      for (int kb = 0; kb < kDB; ++kb) load_block(kb);
    }
    uint32_t stage = 0;
    while (have) {
      const uint32_t scw[8] = {sc[0].x, sc[0].y, sc[0].z, sc[0].w, sc[1].x, sc[1].y, sc[1].z, sc[1].w};
      advance();
      if (have) load_scales();
      bool ok = true;
#pragma unroll
      for (int g = 0; g < kStagesPerTile; ++g, ++stage) {
        const uint32_t slot = stage % kStages;
        ok = mbar_wait(empty(slot), ((stage / kStages) & 1) ^ 1, abort_flag, p.status);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int j = 0; j < kStageBlocks; ++j) {
          const int kb = g * kStageBlocks + j;
          uint8_t* blk = smem + kOffStage + slot * kStageBytes + j * kBlkBytes;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t o[8];
            if (kNV && kb < kDB - 1) {
              const uint32_t pair = half ? scw[kb & 7] >> 16 : scw[kb & 7];
              const uint4 w = buf[kb < kDB - 1 ? kb : 0][0];
              nvfp4x16_to_bf16x16(u ? w.z : w.x, u ? w.w : w.y, (pair >> (8 * u)) & 0xFFu, o);
            } else {
              const uint4 w = kb == kDB - 1 ? tail[u] : buf[kb < kDB - 1 ? kb : 0][u * (kW - 1)];
              const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) e4m3x4_to_bf16x4(ws[q], o[2 * q], o[2 * q + 1]);
            }
            store_unit(blk, u, o);
          }
          if (have) load_block(kb);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(slot));
      }
      if (!ok) break;
    }
  } else {
    // ------------------------------------------------ weights (thread = token)
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const int tid = threadIdx.x;
    uint32_t it = 0;
    int cur = -1;
    bool ok = true;
    while (tiles.next(row, first, count)) {
      const int b = it & 1;
      if (row != cur) {
        bar_epilogue();  // the previous row's values have been read
        if (tid < kHeads) {
          const float l = p.lse[(int64_t)row * kHeads + tid];
          lse_s[tid] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;  // no token attended: no weight
        }
        bar_epilogue();
        cur = row;
      }
      ok = mbar_wait(s_full(b), (it >> 1) & 1, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
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
          sum[0] += ex2f(fmaf(__uint_as_float(r[j]), p.scale_log2, -l.x));
          sum[1] += ex2f(fmaf(__uint_as_float(r[j + 1]), p.scale_log2, -l.y));
          sum[2] += ex2f(fmaf(__uint_as_float(r[j + 2]), p.scale_log2, -l.z));
          sum[3] += ex2f(fmaf(__uint_as_float(r[j + 3]), p.scale_log2, -l.w));
        }
      }
      float w = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (tid < count) {
        const int64_t at = (int64_t)row * p.ld + first + tid;  // direct: one row per sequence
        if (p.direct)
          w += p.mass_in ? p.mass_in[at] : 0.f;
        else if (p.idx && p.idx[at] < 0)
          w = 0.f;
        p.out[at] = w;
      }
      ++it;
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
  // the rows' weights; one row per sequence without a selection needs none, but the query does not know the batch
  const int64_t ld = k > 0 ? k : round4(std::max(max_len, 1));
  return ((size_t)rows * ld * 4 + 255) & ~size_t(255);
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
  CUtensorMap qmap;
  const uint64_t dims[2] = {(uint64_t)kLatent, (uint64_t)rows * kHeads};
  const uint64_t strides[1] = {(uint64_t)kLatent * 2};
  const uint32_t box[2] = {64, (uint32_t)kHeads};
  if (!encode_tmap(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, q_mla, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
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
  p.out = p.direct ? mass_out : static_cast<float*>(workspace);
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
