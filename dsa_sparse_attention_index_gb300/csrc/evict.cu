// evict.cu — eviction from the paged cache by accumulated attention weight.
//
// For each sequence of L tokens and a budget of `keep`: the first `sink` and
// the last `recent` tokens stay, and of the tokens between them the
// keep - sink - recent with the largest accumulated weight (ties to the lower
// index, NaN below every number); with L <= keep every token stays.  The kept
// tokens' records (latent, index-key codes and scale) move, in order, into the
// pages of a second block table.  The model's attention has no position
// encoding (keys and queries carry none), so a token may change its slot.
//
// evict_select_kernel: a cluster of C CTAs per sequence, each over a C-th of
// its tokens.  The C-th largest key is found with three radix digits (11, 11,
// 10 bits of an order-preserving key): a histogram per CTA in shared memory,
// summed over the cluster through distributed shared memory (CTA r sums a C-th
// of the bins and writes the totals to all), then a suffix scan in every CTA.
// A last pass ranks the kept tokens (the CTAs' counts give each its first
// position) and writes their indices, weights and physical rows.  The weights
// are read from L2 on every pass but the first: 4 bytes a token against the
// several hundred of a kept record.
//
// evict_move_kernel: one CTA per destination page, its 64 records copied in
// 16-byte units with every load of a thread in flight before its first store.
// Bound by HBM: each kept record is read and written once.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace dsa {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;

struct SelectParams {
  const float* mass;
  int64_t ld_mass;
  const int32_t* seq_lens;
  int32_t cap, keep, sink, recent;
  const int32_t* block_table;
  int32_t max_blocks, num_blocks;
  int32_t* kept;      // [batch][keep]
  float* mass_out;    // [batch][ld_out] or null
  int64_t ld_out;
  int32_t* new_lens;  // [batch]
  int32_t* phys;      // [batch][keep]: block row * 64 + slot of each kept token, -1 padding
  int32_t* status;
};

// Exclusive prefix sum over the block of one value per thread; `total` gets the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* sh, uint32_t& total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += u;
  }
  if (lane == 31) sh[wid] = x;
  __syncthreads();
  if (wid == 0) {
    uint32_t w = sh[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += u;
    }
    sh[lane] = w;
  }
  __syncthreads();
  const uint32_t before = wid ? sh[wid - 1] : 0u;
  total = sh[kSelWarps - 1];
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const SelectParams p) {
  __shared__ uint32_t hist[kBins];   // this CTA's counts
  __shared__ uint32_t total[kBins];  // the cluster's
  __shared__ uint32_t sh[kSelWarps];
  __shared__ uint32_t found[2];
  __shared__ uint32_t counts[2];     // this CTA's tokens above and at the threshold
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int b = blockIdx.x / C, tid = threadIdx.x;
  grid_dep_wait();
  int L = p.seq_lens[b];
  if (L < 0 || L > p.cap) {
    if (rank == 0 && tid == 0) report(p.status, DSA_ERR_BOUNDS);
    L = 0;
  }
  const float* mass = p.mass + (int64_t)b * p.ld_mass;
  const int32_t* table = p.block_table + (int64_t)b * p.max_blocks;
  int32_t* kept = p.kept + (int64_t)b * p.keep;
  int32_t* phys = p.phys + (int64_t)b * p.keep;
  float* mass_out = p.mass_out ? p.mass_out + (int64_t)b * p.ld_out : nullptr;
  const int n = min(L, p.keep);
  auto put = [&](int pos, int t) {
    const int r = table[t / kBlock];
    const bool ok = r >= 0 && r < p.num_blocks;
    if (!ok) report(p.status, DSA_ERR_BOUNDS);
    kept[pos] = t;
    phys[pos] = ok ? r * kBlock + t % kBlock : -1;
    if (mass_out) mass_out[pos] = mass[t];
  };
  if (rank == 0 && tid == 0) p.new_lens[b] = n;
  for (int i = n + rank * kSelThreads + tid; i < p.keep; i += C * kSelThreads) kept[i] = phys[i] = -1;
  if (mass_out)
    for (int64_t i = n + rank * kSelThreads + tid; i < p.ld_out; i += C * kSelThreads) mass_out[i] = 0.f;
  if (L <= p.keep) {  // uniform over the cluster
    for (int t = rank * kSelThreads + tid; t < L; t += C * kSelThreads) put(t, t);
    return;
  }

  // ---- the threshold: the m-th largest key of the middle [sink, L - recent)
  const int lo = p.sink, hi = L - p.recent;
  const uint32_t m = (uint32_t)(p.keep - p.sink - p.recent);
  const int share = (((L + C - 1) / C) + 3) & ~3;  // tokens a CTA, a multiple of 4
  const int t0 = min(L, rank * share), t1 = min(L, t0 + share);
  uint32_t prefix = 0, mask = 0, want = m;         // key & mask == prefix: the keys still in question
  if (m > 0) {
    const int shifts[3] = {21, 10, 0};
    for (int d = 0; d < 3; ++d) {
      const uint32_t dmask = d < 2 ? 2047u : 1023u;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int t = max(t0, lo) + tid; t < min(t1, hi); t += kSelThreads) {
        const uint32_t key = score_key(mass[t]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shifts[d]) & dmask], 1u);
      }
      cl.sync();
      // bins rank, rank + C, ... summed over the cluster, the sums written to every CTA
      for (int i = rank + C * tid; i < kBins; i += C * kSelThreads) {
        uint32_t s = 0;
        for (int c = 0; c < C; ++c) s += cl.map_shared_rank(hist, c)[i];
        for (int c = 0; c < C; ++c) cl.map_shared_rank(total, c)[i] = s;
      }
      cl.sync();
      // the digit: bins from the top until `want` keys are covered
      const int i0 = kBins - 1 - 2 * tid;
      const uint32_t a = total[i0], c = total[i0 - 1];
      uint32_t all;
      const uint32_t before = block_scan(a + c, sh, all);
      if (want > before && want <= before + a) {
        found[0] = (uint32_t)i0;
        found[1] = before;
      } else if (want > before + a && want <= before + a + c) {
        found[0] = (uint32_t)(i0 - 1);
        found[1] = before + a;
      }
      __syncthreads();
      prefix |= found[0] << shifts[d];
      mask |= dmask << shifts[d];
      want -= found[1];
      __syncthreads();
    }
  }
  // `want` of the keys equal to `prefix` stay, those of the lowest indices; with m = 0 none does
  uint32_t gt = 0, eq = 0;
  if (m > 0)
    for (int t = max(t0, lo) + tid; t < min(t1, hi); t += kSelThreads) {
      const uint32_t key = score_key(mass[t]);
      gt += key > prefix;
      eq += key == prefix;
    }
  uint32_t tg, te;
  block_scan(gt, sh, tg);
  block_scan(eq, sh, te);
  if (tid == 0) {
    counts[0] = tg;
    counts[1] = te;
  }
  cl.sync();
  // kept tokens and equal keys of the CTAs before this one
  uint32_t eq_before = 0, pos = 0;
  for (int c = 0; c < rank; ++c) {
    const uint32_t* o = cl.map_shared_rank(counts, c);
    const int s0 = min(L, c * share), s1 = min(L, s0 + share);
    const uint32_t e = o[1], left = want > eq_before ? want - eq_before : 0u;
    pos += o[0] + min(e, left) + (uint32_t)max(0, min(s1, lo) - s0) + (uint32_t)max(0, s1 - max(s0, hi));
    eq_before += e;
  }
  cl.sync();  // the counts have been read: a CTA may exit
  for (int tb = t0; tb < t1; tb += kSelThreads) {
    const int t = tb + tid;
    const bool in = t < t1, middle = in && t >= lo && t < hi && m > 0;
    const uint32_t key = middle ? score_key(mass[t]) : 0u;
    const bool is_eq = middle && key == prefix;
    uint32_t eqs, kepts;
    const uint32_t er = block_scan(is_eq ? 1u : 0u, sh, eqs);
    const bool stay = in && ((t < lo || t >= hi) || (middle && (key > prefix || (is_eq && eq_before + er < want))));
    const uint32_t kr = block_scan(stay ? 1u : 0u, sh, kepts);
    if (stay) put((int)(pos + kr), t);
    pos += kepts;
    eq_before += eqs;
  }
}

struct MoveParams {
  const uint8_t* src;
  uint8_t* dst;
  int64_t src_stride, dst_stride;
  int64_t src_lat, src_idx, dst_lat, dst_idx;  // page offsets in a block row
  int32_t rec, code;                           // latent record and index-key code bytes, multiples of 16
  const int32_t* new_lens;
  const int32_t* phys;
  int32_t keep;
  const int32_t* dst_table;
  int32_t dst_max_blocks, dst_num_blocks;
  int32_t* status;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveParams p) {
  __shared__ int32_t src_s[kBlock];
  grid_dep_wait();
  const int pages = (p.keep + kBlock - 1) / kBlock;
  const int b = blockIdx.x / pages, page = blockIdx.x % pages, tid = threadIdx.x;
  const int n = min(p.new_lens[b] - page * kBlock, kBlock);
  if (n <= 0) return;
  const int dr = p.dst_table[(int64_t)b * p.dst_max_blocks + page];
  if (dr < 0 || dr >= p.dst_num_blocks) {
    if (tid == 0) report(p.status, DSA_ERR_BOUNDS);
    return;
  }
  if (tid < n) src_s[tid] = p.phys[(int64_t)b * p.keep + page * kBlock + tid];
  __syncthreads();
  uint8_t* row = p.dst + (int64_t)dr * p.dst_stride;
  const int lu = p.rec / 16, ku = p.code / 16;
  const int units = n * lu, all = units + n * ku;
  for (int u0 = tid; u0 < all; u0 += kMoveThreads * kMoveUnroll) {
    uint4 v[kMoveUnroll];
    uint8_t* to[kMoveUnroll];
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i) {
      const int u = u0 + i * kMoveThreads;
      to[i] = nullptr;
      if (u >= all) continue;
      const bool lat = u < units;
      const int w = lat ? u : u - units, per = lat ? lu : ku;
      const int tok = w / per, c = w % per, s = src_s[tok];
      if (s < 0) continue;  // a bad page of the source, reported
      const uint8_t* from = p.src + (int64_t)(s / kBlock) * p.src_stride + (lat ? p.src_lat : p.src_idx) +
                            (s % kBlock) * (per * 16) + c * 16;
      to[i] = row + (lat ? p.dst_lat : p.dst_idx) + tok * (per * 16) + c * 16;
      v[i] = *reinterpret_cast<const uint4*>(from);
    }
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i)
      if (to[i]) *reinterpret_cast<uint4*>(to[i]) = v[i];
  }
  // the 4-byte key scales behind the codes
  if (tid < n && src_s[tid] >= 0) {
    const int s = src_s[tid];
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p.src + (int64_t)(s / kBlock) * p.src_stride + p.src_idx +
                                                          kBlock * p.code + (s % kBlock) * 4);
    *reinterpret_cast<uint32_t*>(row + p.dst_idx + kBlock * p.code + tid * 4) = v;
  }
}

}  // namespace

size_t evict_workspace_bytes(int batch, int keep) { return ((size_t)batch * keep * 4 + 255) & ~size_t(255); }

dsa_status_t launch_cache_evict(const dsa_paged_cache_t& src, const dsa_batch_t& bt, const float* mass, int64_t ld_mass,
                                int keep, int sink, int recent, const dsa_paged_cache_t& dst, const int32_t* dst_table,
                                int dst_max_blocks, int32_t* kept, float* mass_out, int64_t ld_out, int32_t* new_lens,
                                void* workspace, int32_t* status, cudaStream_t st) {
  const int rec = src.latent_format == DSA_LATENT_NVFP4 ? 352 : kLatent;
  const int code = src.key_format == DSA_KEY_FP8_E4M3 ? kIdxDim : kIdxDim / 2;
  SelectParams s = {};
  s.mass = mass;
  s.ld_mass = ld_mass;
  s.seq_lens = bt.seq_lens;
  s.cap = (int)std::min<int64_t>((int64_t)bt.max_blocks_per_seq * kBlock, bt.max_seq_len);
  s.keep = keep;
  s.sink = sink;
  s.recent = recent;
  s.block_table = bt.block_table;
  s.max_blocks = bt.max_blocks_per_seq;
  s.num_blocks = src.num_blocks;
  s.kept = kept;
  s.mass_out = mass_out;
  s.ld_out = ld_out;
  s.new_lens = new_lens;
  s.phys = static_cast<int32_t*>(workspace);
  s.status = status;
  // CTAs a sequence: one up to 4,096 tokens, then one more for every 4,096
  int C = 1;
  while (C < kMaxCluster && C * 4096 < bt.max_seq_len) C *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(bt.batch * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  if (cuda_status(cudaLaunchKernelEx(&cfg, evict_select_kernel, s)) != DSA_OK) return DSA_ERR_CUDA;
  MoveParams m = {};
  m.src = static_cast<const uint8_t*>(src.base);
  m.dst = static_cast<uint8_t*>(dst.base);
  m.src_stride = src.row_stride;
  m.dst_stride = dst.row_stride;
  m.src_lat = src.latent_off;
  m.src_idx = src.index_off;
  m.dst_lat = dst.latent_off;
  m.dst_idx = dst.index_off;
  m.rec = rec;
  m.code = code;
  m.new_lens = new_lens;
  m.phys = s.phys;
  m.keep = keep;
  m.dst_table = dst_table;
  m.dst_max_blocks = dst_max_blocks;
  m.dst_num_blocks = dst.num_blocks;
  m.status = status;
  cfg.gridDim = dim3((unsigned)(bt.batch * ((keep + kBlock - 1) / kBlock)));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.numAttrs = 1;
  count_launches(1);
  if (cuda_status(cudaLaunchKernelEx(&cfg, evict_move_kernel, m)) != DSA_OK) return DSA_ERR_CUDA;
  return launch_status();
}

}  // namespace dsa
