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
// its tokens, whose order-preserving keys it loads once into shared memory.  The
// threshold is found with three radix digits (11, 11, 10 bits): a histogram per
// CTA, summed over the cluster through distributed shared memory (CTA r sums a
// C-th of the bins and writes the totals to all; every CTA reading all C
// histograms took twice as long), then a scan from the top.  Tokens of total 0,
// often a large part, are counted apart instead of all on one bin.  At last each
// warp ranks a run of the CTA's tokens (the CTAs' and warps' counts give its first
// position) and writes the kept ones' indices, totals and physical rows.  Bound
// by latency: the barriers and dependent loads of about ten steps.
//
// evict_move_kernel: one CTA per destination page, its 64 records copied in
// 16-byte units with every load of a thread in flight before its first store.
// Bound by HBM: each kept record is read and written once (40 us for 224 MB of
// NVFP4 records and MXFP4 keys, 58 us for 371 MB of E4M3 records and FP8 keys:
// 5.6 and 6.4 TB/s).
// The whole call: 32 contexts of 16K to 49K tokens to 8,192: 67 us; four of 128K
// to 160K to 65,536: 87 us.
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace dsa {

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr uint32_t kZeroKey = 0x80000000u;  // score_key(0)
constexpr int kUnroll = 4;            // tokens of a lane in flight
constexpr int kCtaTokens = 1024;      // a CTA's share before a sequence takes more of them
constexpr int kMaxCluster = 16;       // (8 where the device cannot schedule 16)
constexpr int kMaxShare = 44 * 1024;  // tokens whose keys a CTA holds in shared memory (176 KB)

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
  __syncthreads();  // sh may still be read by the scan before
  if (lane == 31) sh[wid] = x;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    const uint32_t s = sh[w];
    if (w < wid) before += s;
    total += s;
  }
  return before + x - v;
}

// The total whose key this is (-0 as +0, a NaN as the canonical one).
__device__ __forceinline__ float key_value(uint32_t key) {
  return key == 0 ? __uint_as_float(0x7FC00000u) : __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// kResident: the CTA's keys stay in shared memory; else every pass reads the totals again (L2).
template <bool kResident>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) uint32_t hist[kBins];   // this CTA's counts
  __shared__ __align__(16) uint32_t total[kBins];  // the cluster's
  __shared__ uint32_t sh[kSelWarps];
  __shared__ uint32_t found[2];
  __shared__ uint32_t counts[2];  // this CTA's tokens kept whatever their rank, and at the threshold
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int b = blockIdx.x / C, tid = threadIdx.x;
  for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
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
  auto put = [&](int pos, int t, int r, float x) {  // token t of block row r and total x is kept as token pos
    const bool ok = r >= 0 && r < p.num_blocks;
    if (!ok) report(p.status, DSA_ERR_BOUNDS);
    kept[pos] = t;
    phys[pos] = ok ? r * kBlock + t % kBlock : -1;
    if (mass_out) mass_out[pos] = x;
  };
  if (rank == 0 && tid == 0) p.new_lens[b] = n;
  for (int i = n + rank * kSelThreads + tid; i < p.keep; i += C * kSelThreads) kept[i] = phys[i] = -1;
  if (mass_out)
    for (int64_t i = n + rank * kSelThreads + tid; i < p.ld_out; i += C * kSelThreads) mass_out[i] = 0.f;
  if (L <= p.keep) {  // uniform over the cluster
    for (int t = rank * kSelThreads + tid; t < L; t += C * kSelThreads) put(t, t, table[t / kBlock], mass[t]);
    return;
  }

  // ---- the threshold: the m-th largest key of the middle [sink, L - recent)
  const int lo = p.sink, hi = L - p.recent;
  const uint32_t m = (uint32_t)(p.keep - p.sink - p.recent);
  const int share = (L + C - 1) / C;             // tokens a CTA
  const int t0 = (int)min((int64_t)L, (int64_t)rank * share), t1 = (int)min((int64_t)L, (int64_t)t0 + share);
  const int a0 = max(t0, lo), a1 = min(t1, hi);  // its part of the middle
  auto key_at = [&](int t) { return kResident ? keys[t - t0] : score_key(mass[t]); };
  if (kResident) {
    constexpr int kU = 12;  // loads of a thread in flight
    for (int tb = t0 + tid; tb < t1; tb += kU * kSelThreads) {
      float x[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) x[u] = tb + u * kSelThreads < t1 ? mass[tb + u * kSelThreads] : 0.f;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (tb + u * kSelThreads < t1) keys[tb + u * kSelThreads - t0] = score_key(x[u]);
    }
  }
  __syncthreads();
  uint32_t prefix = 0, mask = 0, want = m;  // key & mask == prefix: the keys still in question
  if (m > 0) {
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
      const uint32_t dmask = d < 2 ? 2047u : 1023u;
      uint32_t zeros = 0;
      for (int tb = a0 + tid; tb < a1; tb += kUnroll * kSelThreads) {
        uint32_t key[kUnroll];
        bool in[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int t = tb + u * kSelThreads;
          key[u] = t < a1 ? key_at(t) : 0u;
          in[u] = t < a1 && (key[u] & mask) == prefix;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (key[u] == kZeroKey)
            zeros += in[u];
          else if (in[u])
            atomicAdd(&hist[(key[u] >> shift) & dmask], 1u);
        }
      }
      zeros = __reduce_add_sync(0xffffffffu, zeros);
      if (zeros && (tid & 31) == 0) atomicAdd(&hist[(kZeroKey >> shift) & dmask], zeros);
      cl.sync();
      // bins [rank, rank + 1) * kBins / C summed over the cluster, the sums written to every CTA
      for (int i = tid; i < kBins / C; i += kSelThreads) {
        const int bin = rank * (kBins / C) + i;
        uint32_t x[kMaxCluster], s = 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) x[c] = c < C ? cl.map_shared_rank(hist, c)[bin] : 0u;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) s += x[c];
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c)
          if (c < C) cl.map_shared_rank(total, c)[bin] = s;
      }
      cl.sync();
      // the digit: bins from the top, four a thread, until `want` keys are covered
      static_assert(kBins == 4 * kSelThreads, "four bins a thread");
      const int bin = kBins - 4 - 4 * tid;
      const uint4 x = *reinterpret_cast<const uint4*>(total + bin);
      const uint32_t v[4] = {x.w, x.z, x.y, x.x};
      *reinterpret_cast<uint4*>(hist + bin) = make_uint4(0, 0, 0, 0);  // read by every CTA before the barrier
      uint32_t all, before = block_scan(v[0] + v[1] + v[2] + v[3], sh, all);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (want > before && want <= before + v[i]) {
          found[0] = (uint32_t)(bin + 3 - i);
          found[1] = before;
        }
        before += v[i];
      }
      __syncthreads();
      prefix |= found[0] << shift;
      mask |= dmask << shift;
      want -= found[1];
      __syncthreads();
    }
  }
  // `want` of the keys equal to `prefix` stay, those of the lowest indices; with m = 0 none does.
  // 1: a token that stays whatever its rank among the equals; 2: one of the equals.
  auto kind = [&](int t, uint32_t key) {
    return t < lo || t >= hi ? 1 : m == 0 ? 0 : key > prefix ? 1 : key == prefix ? 2 : 0;
  };
  // Each warp ranks a run of the CTA's tokens: first its counts, then, from its first position, the tokens.
  const int lane = tid & 31, wid = tid >> 5;
  const int run = (t1 - t0 + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
  const int w0 = min(t1, t0 + wid * run), w1 = min(t1, w0 + run);
  uint32_t hard = 0, equal = 0;
  for (int tb = w0; tb < w1; tb += 32 * kUnroll) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = tb + 32 * u + lane;
      const int k = t < w1 ? kind(t, key_at(t)) : 0;
      hard += k == 1;
      equal += k == 2;
    }
  }
  hard = __reduce_add_sync(0xffffffffu, hard);
  equal = __reduce_add_sync(0xffffffffu, equal);
  uint32_t th, te;
  const uint32_t hs = block_scan(lane == 0 ? hard : 0u, sh, th), es = block_scan(lane == 0 ? equal : 0u, sh, te);
  uint32_t hard_before = __shfl_sync(0xffffffffu, hs, 0), eq_before = __shfl_sync(0xffffffffu, es, 0);
  if (tid == 0) {
    counts[0] = th;
    counts[1] = te;
  }
  cl.sync();
  // of the CTAs before this one: lane c asks CTA c
  const uint32_t* o = lane < rank ? cl.map_shared_rank(counts, lane) : nullptr;
  hard_before += __reduce_add_sync(0xffffffffu, o ? o[0] : 0u);
  eq_before += __reduce_add_sync(0xffffffffu, o ? o[1] : 0u);
  cl.sync();  // the counts have been read: a CTA may exit
  const uint32_t below = (1u << lane) - 1u;
  for (int tb = w0; tb < w1; tb += 32 * kUnroll) {
    uint32_t key[kUnroll];
    int r[kUnroll], k[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = tb + 32 * u + lane;
      key[u] = t < w1 ? key_at(t) : 0u;
      r[u] = t < w1 ? table[t / kBlock] : -1;
      k[u] = t < w1 ? kind(t, key[u]) : 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t hm = __ballot_sync(0xffffffffu, k[u] == 1), em = __ballot_sync(0xffffffffu, k[u] == 2);
      const uint32_t hb = hard_before + __popc(hm & below), eb = eq_before + __popc(em & below);
      if (k[u] == 1 || (k[u] == 2 && eb < want)) put((int)(hb + min(eb, want)), tb + 32 * u + lane, r[u], key_value(key[u]));
      hard_before += __popc(hm);
      eq_before += __popc(em);
    }
  }
}

struct MoveParams {
  const uint8_t* src;
  uint8_t* dst;
  int64_t src_stride, dst_stride;
  int64_t src_lat, src_idx, dst_lat, dst_idx;  // page offsets in a block row
  const int32_t* new_lens;
  const int32_t* phys;
  int32_t keep, pages;
  const int32_t* dst_table;
  int32_t dst_max_blocks, dst_num_blocks;
  int32_t* status;
};

constexpr int kMoveThreads = 256;

// kRec, kCode: bytes of a latent record and of an index key's codes (its 4-byte scales lie behind the page's codes).
template <int kRec, int kCode>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveParams p) {
  constexpr int kLu = kRec / 16, kKu = kCode / 16, kUnits = kLu + kKu;  // 16-byte units of a token
  constexpr int kPer = (kBlock * kUnits + kMoveThreads - 1) / kMoveThreads;
  __shared__ int32_t src_s[kBlock];  // kept token's slot, block row * 64 + slot; -1: none, or a bad page (reported)
  grid_dep_wait();
  const int b = blockIdx.x / p.pages, page = blockIdx.x % p.pages, tid = threadIdx.x;
  const int n = min(p.new_lens[b] - page * kBlock, kBlock);
  const int dr = p.dst_table[(int64_t)b * p.dst_max_blocks + page];
  const int at = page * kBlock + tid;
  const int s = tid < kBlock && at < p.keep ? p.phys[(int64_t)b * p.keep + at] : -1;
  if (n <= 0) return;
  if (dr < 0 || dr >= p.dst_num_blocks) {
    if (tid == 0) report(p.status, DSA_ERR_BOUNDS);
    return;
  }
  if (tid < kBlock) src_s[tid] = at < page * kBlock + n ? s : -1;
  __syncthreads();
  uint8_t* row = p.dst + (int64_t)dr * p.dst_stride;
  uint4 v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int u = tid + i * kMoveThreads, tok = u / kUnits, c = u % kUnits;
    if (u >= kBlock * kUnits) continue;
    const int32_t q = src_s[tok];
    if (q < 0) continue;
    const int slot = q % kBlock;
    v[i] = *reinterpret_cast<const uint4*>(p.src + (int64_t)(q / kBlock) * p.src_stride +
                                           (c < kLu ? p.src_lat + slot * kRec + c * 16
                                                    : p.src_idx + slot * kCode + (c - kLu) * 16));
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int u = tid + i * kMoveThreads, tok = u / kUnits, c = u % kUnits;
    if (u >= kBlock * kUnits || src_s[tok] < 0) continue;
    uint8_t* to = row + (c < kLu ? p.dst_lat + tok * kRec + c * 16 : p.dst_idx + tok * kCode + (c - kLu) * 16);
    *reinterpret_cast<uint4*>(to) = v[i];
  }
  if (tid < n && s >= 0)
    *reinterpret_cast<uint32_t*>(row + p.dst_idx + kBlock * kCode + tid * 4) =
        *reinterpret_cast<const uint32_t*>(p.src + (int64_t)(s / kBlock) * p.src_stride + p.src_idx + kBlock * kCode +
                                           (s % kBlock) * 4);
}

}  // namespace

// Whether clusters of C of the largest select CTAs can be resident on this device (asked once per device).
static bool cluster_ok(int C) {
  static std::atomic<int> known[64];  // 0 unknown, 1 yes, 2 no
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return false;
  if (known[dev] == 0) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = kMaxShare * 4;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok = cudaOccupancyMaxActiveClusters(&n, evict_select_kernel<true>, &cfg) == cudaSuccess && n > 0;
    cudaGetLastError();  // a refused query leaves no error behind
    known[dev] = ok ? 1 : 2;
  }
  return known[dev] == 1;
}

size_t evict_workspace_bytes(int batch, int keep) { return ((size_t)batch * keep * 4 + 255) & ~size_t(255); }

dsa_status_t launch_cache_evict(const dsa_paged_cache_t& src, const dsa_batch_t& bt, const float* mass, int64_t ld_mass,
                                int keep, int sink, int recent, const dsa_paged_cache_t& dst, const int32_t* dst_table,
                                int dst_max_blocks, int32_t* kept, float* mass_out, int64_t ld_out, int32_t* new_lens,
                                void* workspace, int32_t* status, cudaStream_t st) {
  const bool nv = src.latent_format == DSA_LATENT_NVFP4, key8 = src.key_format == DSA_KEY_FP8_E4M3;
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
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    if (cuda_status(cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMaxShare * 4)) != DSA_OK ||
        cuda_status(cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) !=
            DSA_OK ||
        cuda_status(cudaFuncSetAttribute(evict_select_kernel<false>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                         1)) != DSA_OK)
      return DSA_ERR_CUDA;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  // CTAs a sequence: shares of kCtaTokens or less while the grid fits the SMs (the last doubling: two an SM).
  // One sequence of 5,001 tokens: 24.9 us with one CTA, 19.1, 16.0 and 15.4 with 2, 4 and 8.
  int most = kMaxCluster;
  while (most > 8 && !cluster_ok(most)) most /= 2;
  int C = 1;
  while (C < most && C * kCtaTokens < s.cap && (int64_t)C * bt.batch <= num_sms()) C *= 2;
  const int64_t share = ((int64_t)s.cap + C - 1) / C;
  const bool resident = share <= kMaxShare;
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
  cfg.dynamicSmemBytes = resident ? (size_t)std::max<int64_t>(share, 1) * 4 : 0;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  if (cuda_status(cudaLaunchKernelEx(&cfg, resident ? evict_select_kernel<true> : evict_select_kernel<false>, s)) !=
      DSA_OK)
    return DSA_ERR_CUDA;
  MoveParams m = {};
  m.src = static_cast<const uint8_t*>(src.base);
  m.dst = static_cast<uint8_t*>(dst.base);
  m.src_stride = src.row_stride;
  m.dst_stride = dst.row_stride;
  m.src_lat = src.latent_off;
  m.src_idx = src.index_off;
  m.dst_lat = dst.latent_off;
  m.dst_idx = dst.index_off;
  m.new_lens = new_lens;
  m.phys = s.phys;
  m.keep = keep;
  m.pages = (keep + kBlock - 1) / kBlock;
  m.dst_table = dst_table;
  m.dst_max_blocks = dst_max_blocks;
  m.dst_num_blocks = dst.num_blocks;
  m.status = status;
  cfg.gridDim = dim3((unsigned)(bt.batch * m.pages));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  count_launches(1);
  constexpr int kNv = kValue / 2 + kValue / 16 + (kLatent - kValue);
  auto move = nv ? (key8 ? evict_move_kernel<kNv, kIdxDim> : evict_move_kernel<kNv, kIdxDim / 2>)
                 : (key8 ? evict_move_kernel<kLatent, kIdxDim> : evict_move_kernel<kLatent, kIdxDim / 2>);
  if (cuda_status(cudaLaunchKernelEx(&cfg, move, m)) != DSA_OK) return DSA_ERR_CUDA;
  return launch_status();
}

}  // namespace dsa
