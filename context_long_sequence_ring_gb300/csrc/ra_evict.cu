// Eviction from the sharded paged cache by accumulated attention weight, per
// K/V head, and the packing of what is kept.
//
// Mathematics.  The weights map to 32-bit keys in their order (NaN 0, -0 as
// +0), and a radix select finds the key of the m-th heaviest token of the
// middle part, m = keep - n_sink - n_recent, 8 bits at a time from the top:
// all larger keys are kept, and of the equal ones the first as many as are
// missing.  Counts before each token, in token order, then number the kept ones.
//
// One cluster of up to 8 CTAs takes a (request, K/V head) from the weights to
// the moved rows in one launch.  Each CTA holds the keys of a contiguous part of
// the context in shared memory; histograms and counts meet through distributed
// shared memory, every CTA summing them for itself.  The move is bound by HBM
// (2 x 512 bytes per kept token of head dim 128 in bf16); selecting reads the
// weights once, 4 bytes per token, and is bound by latency: 4 digits of 2 us, reading
// 2.5, counting and numbering 4.  16 prompts of 8192-16384 cut to 2048 (8 heads of
// 128): 61 us, of which the move of 268 MB takes 41 (6.5 TB/s); moved with plain
// loads and stores 63.  16 of 16384: 65 us, in place 66.  2 requests of 900-1301 cut to 512: 13 us.
//
// Where the table has room for more tokens than a cluster's shared memory has keys
// (24576 to a CTA), the keys past that are read again for each digit and for the
// numbering, and single weights instead of four are read: 8 requests of 131072 cut to 2048
// take 217 us on a floor of 25, 32 of 32768 292 on 85; 16 of 16384 with a table for
// 131072 84 us instead of 65.
#include <algorithm>

#include "ra_paged.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_evict)

namespace {

constexpr int kThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kKeysCap = 24576;   // keys in shared memory: 96 KB, so that two CTAs share an SM
constexpr int kBatch = 256;       // tokens a CTA moves at a time
constexpr int kInFlight = 8;      // 16-byte words that a thread holds

struct EvictParams {
  uint4 *kc, *vc;
  float* w;
  Paged src, dst;  // dst.table may be src.table
  const int32_t* ctx;
  int row_words, keep, n_sink, n_recent, in_place, keys_cap, by_four;
  FastDiv by_words;   // by the words of a token's K and V
  int32_t *kept, *new_lens;
};

// Order-preserving key of a weight.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __noinline__ uint32_t load_key(const EvictParams& p, int r, int g, int x) {
  const int64_t at = paged_row(p.src, r, x, g, 701);
  return at < 0 ? 0u : key_of(p.w[at]);
}

// All threads of all CTAs of the cluster; what was written before is visible to them after.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The 32-bit word at p in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ int peer_word(const void* p, int rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return static_cast<int>(v);
}

// Exclusive sum over the block and its total (two 32-bit counts in one word).
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* warp_sums, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += warp_sums[i];
    total += warp_sums[i];
  }
  return before + x - v;
}

// FITS: a CTA's part of any context is in shared memory whole; else what is past the capacity is read again.
template <bool FITS>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ int hist[4][256], sums[256];
  __shared__ uint64_t warp_sums[kThreads / 32];
  __shared__ int counts[2];              // of this CTA's part: kept for certain, ties
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int64_t row_src[kBatch], row_dst[kBatch];
  const int C = gridDim.x, rank = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int r = blockIdx.y / p.src.Hkv, g = blockIdx.y - r * p.src.Hkv;
  const int N = paged_len(p.src, p.ctx[r], 700);
  const int n_new = min(N, p.keep);
  int32_t* kept = p.kept + static_cast<int64_t>(blockIdx.y) * p.keep;
  if (g == 0 && rank == 0 && tid == 0) p.new_lens[r] = n_new;
  for (int j = n_new + rank * kThreads + tid; j < p.keep; j += C * kThreads) kept[j] = -1;

  if (N <= p.keep) {
    for (int j = rank * kThreads + tid; j < N; j += C * kThreads) kept[j] = j;
    if (p.in_place) return;              // the same for all CTAs of the cluster
    cluster_barrier();                   // kept is read by all of them
  } else {
    const int m0 = p.n_sink, m1 = N - p.n_recent;      // the middle part [m0, m1)
    const int per = ((N + C - 1) / C + 3) & ~3;
    const int lo = min(N, rank * per), hi = min(N, lo + per);
    auto key = [&](int x) { return FITS || x - lo < p.keys_cap ? keys[x - lo] : load_key(p, r, g, x); };
    int need = p.keep - p.n_sink - p.n_recent;
    uint32_t prefix = need > 0 ? 0 : 0xffffffffu;      // 0xffffffff: above every key
    for (int i = tid; i < 4 * 256; i += kThreads) hist[i >> 8][i & 255] = 0;
    if (FITS && p.by_four) {
      // four tokens lie together: one place, one load and one store for them; two such of a thread in flight
      for (int x0 = lo + 4 * tid; x0 < hi; x0 += 8 * kThreads) {
        int64_t at[2];
        float4 w[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int x = x0 + u * 4 * kThreads;
          at[u] = x < hi ? paged_row(p.src, r, x, g, 701) : -1;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float nan = __int_as_float(0x7fffffff);
          w[u] = at[u] >= 0 ? *reinterpret_cast<const float4*>(p.w + at[u]) : make_float4(nan, nan, nan, nan);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int x = x0 + u * 4 * kThreads;   // keys past hi (of the same four) are in the buffer, never read
          if (x < hi)
            *reinterpret_cast<uint4*>(keys + x - lo) = make_uint4(key_of(w[u].x), key_of(w[u].y), key_of(w[u].z), key_of(w[u].w));
        }
      }
    } else {
      // four tokens of a thread in flight
      for (int x0 = lo; x0 < hi; x0 += 4 * kThreads) {
        float w[4];
        int64_t at[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int x = x0 + u * kThreads + tid;
          at[u] = x < hi && (FITS || x - lo < p.keys_cap) ? paged_row(p.src, r, x, g, 701) : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = at[u] >= 0 ? p.w[at[u]] : __int_as_float(0x7fffffff);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int x = x0 + u * kThreads + tid;
          if (x < hi && (FITS || x - lo < p.keys_cap)) keys[x - lo] = key_of(w[u]);
        }
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      if (need <= 0) break;                            // nothing to choose
      const int shift = 24 - 8 * pass;
      const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
      const int c0 = max(lo, m0), c1 = min(hi, m1);    // this CTA's share of the middle part
      for (int x0 = c0 + (tid & ~31); x0 < c1; x0 += 4 * kThreads) {
        uint32_t k[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int x = x0 + u * kThreads + lane;
          k[u] = x < c1 ? key(x) : 0;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bool in = x0 + u * kThreads + lane < c1 && (k[u] & mask) == prefix;
          if (in) atomicAdd(&hist[pass][(k[u] >> shift) & 255], 1);
        }
      }
      cluster_barrier();
      if (tid < 256) {                                 // bin tid from the top, over the cluster
        int t = 0;
#pragma unroll 4
        for (int c = 0; c < C; ++c) t += peer_word(&hist[pass][255 - tid], c);
        sums[tid] = t;
      }
      __syncthreads();
      if (tid < 32) {
        // bins 8*lane .. 8*lane+7 from the top: lane 0 holds the largest digits
        int b[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = sums[8 * lane + i];
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += b[i];
        int above = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, above, o);
          if (lane >= o) above += y;
        }
        above -= sum;                                  // tokens in larger digits than this lane's
        if (above < need && need <= above + sum) {     // one lane: the digit of the need-th largest key
          int i = 0;
#pragma unroll
          for (int u = 0; u < 7; ++u)
            if (i == u && above + b[u] < need) {
              above += b[u];
              i = u + 1;
            }
          s_prefix = prefix | (static_cast<uint32_t>(255 - (8 * lane + i)) << shift);
          s_need = need - above;
        }
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
      __syncthreads();
    }
    // Each warp takes a run of whole groups of 32 tokens: tokens kept for certain and ties are counted, then
    // numbered in order.
    const int warp = tid >> 5;
    const int run = (((hi - lo + 31) >> 5) + kThreads / 32 - 1) / (kThreads / 32) * 32;
    const int x0 = min(hi, lo + warp * run), x1 = min(hi, x0 + run);
    int sure = 0, ties = 0;
#pragma unroll 4
    for (int x = x0 + lane; x < x1; x += 32) {
      const bool mid = x >= m0 && x < m1;
      const uint32_t k = key(x);
      sure += !mid || k > prefix;
      ties += mid && k == prefix;
    }
    uint64_t all;
    const uint64_t earlier = block_scan(static_cast<uint64_t>(ties) << 32 | static_cast<uint32_t>(sure), warp_sums, all);
    if (tid == 0) {
      counts[0] = static_cast<int>(all);
      counts[1] = static_cast<int>(all >> 32);
    }
    cluster_barrier();
    const uint64_t warp_start = __shfl_sync(0xffffffffu, earlier, 0);
    int at = static_cast<int>(warp_start), tie = static_cast<int>(warp_start >> 32);   // before this warp, in the context
    for (int c = 0; c < rank; ++c) {
      at += peer_word(&counts[0], c);
      tie += peer_word(&counts[1], c);
    }
    at += min(tie, need);
    const unsigned below = (1u << lane) - 1;
    for (int xb = x0; xb < x1; xb += 32) {
      const int x = xb + lane;
      const bool mid = x >= m0 && x < m1;
      const uint32_t k = x < x1 ? key(x) : 0;
      const bool is_tie = x < x1 && mid && k == prefix;
      const unsigned tied = __ballot_sync(0xffffffffu, is_tie);
      const bool keeps = x < x1 && (!mid || k > prefix || (is_tie && tie + __popc(tied & below) < need));
      const unsigned kept_mask = __ballot_sync(0xffffffffu, keeps);
      if (keeps) kept[at + __popc(kept_mask & below)] = x;
      at += __popc(kept_mask);
      tie += __popc(tied);
    }
    cluster_barrier();                                 // kept is complete; no CTA reads another's memory any more
  }

  if (n_new == 0) return;
  // Pack in ascending batches of the whole cluster.  In place a batch is read whole before it is written: token j
  // comes from a place >= j, so no later batch reads what an earlier one wrote.
  const int rw = p.row_words, words = 2 * rw;
  const int sub = max(1, (kThreads * kInFlight) / words);   // tokens whose words the CTA holds at a time
  const int most = p.in_place ? min(kBatch, sub) : kBatch;
  const int batches = (n_new + C * most - 1) / (C * most), step = (n_new + C * batches - 1) / (C * batches);   // evenly
#pragma unroll 1
  for (int b0 = 0; b0 < n_new; b0 += C * step) {
    const int j0 = b0 + rank * step, nj = max(0, min(step, n_new - j0));
    float wt = 0.f;
    __syncthreads();
    if (tid < nj) {
      const int j = j0 + tid, vb = p.dst.by_V.div(j);
      const int64_t src = paged_row(p.src, r, __ldcg(&kept[j]), g, 701);
      int64_t dst = -1;
      if (vb < p.dst.max_vb) dst = paged_row(p.dst, r, j, g, 702);
      else ra_record_error(RA_ERR_DEVICE_BOUNDS, 703);
      row_src[tid] = src;
      row_dst[tid] = src == dst ? -1 : dst;
      if (src >= 0) wt = p.w[src];
    }
    __syncthreads();
    if (!p.in_place && tid < nj && row_dst[tid] >= 0) p.w[row_dst[tid]] = wt;
    for (int t0 = 0; t0 < step; t0 += sub) {           // once in place
      const int total = max(0, min(sub, nj - t0)) * words;
      uint4 v[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int e = u * kThreads + tid;
        v[u] = make_uint4(0, 0, 0, 0);
        if (e < total) {
          int c;
          const int j = t0 + p.by_words.div(e, c);
          const int64_t at = row_src[j];
          if (at >= 0 && row_dst[j] >= 0) v[u] = __ldcs(c < rw ? &p.kc[at * rw + c] : &p.vc[at * rw + c - rw]);
        }
      }
      if (p.in_place) {
        cluster_barrier();
        if (tid < nj && row_dst[tid] >= 0) p.w[row_dst[tid]] = wt;
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int e = u * kThreads + tid;
        if (e < total) {
          int c;
          const int j = t0 + p.by_words.div(e, c);
          const int64_t at = row_dst[j];
          if (at >= 0) __stcs(c < rw ? &p.kc[at * rw + c] : &p.vc[at * rw + c - rw], v[u]);
        }
      }
    }
  }
}

}  // namespace

extern "C" ra_status ra_cp_evict(void* k_cache, void* v_cache, float* weights, const int32_t* block_table,
                                 const int32_t* dst_block_table, const int32_t* ctx_lens, int32_t R, int32_t Hkv,
                                 int32_t d, ra_dtype dt, int32_t block_size, int32_t interleave, int32_t pcp,
                                 int32_t dcp, int32_t max_vblocks, int32_t dst_max_vblocks, int64_t num_blocks,
                                 int32_t keep, int32_t n_sink, int32_t n_recent, int32_t* kept, int32_t* new_lens,
                                 ra_stream stream) {
  ra::clear_error();
  ra_status st = check_paged(R, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks);
  if (st != RA_OK) return st;
  RA_REQUIRE(dt == RA_BF16 || dt == RA_F32, "unknown dtype");
  RA_REQUIRE(d >= 1, "d must be >= 1");
  RA_REQUIRE(keep <= (1 << 30), "keep must be at most 2^30");
  RA_REQUIRE(keep >= 1 && n_sink >= 0 && n_recent >= 0 && static_cast<int64_t>(n_sink) + n_recent <= keep,
             "keep >= 1 and 0 <= n_sink + n_recent <= keep required (keep %d, n_sink %d, n_recent %d)", keep, n_sink,
             n_recent);
  RA_REQUIRE(dst_block_table == nullptr || dst_max_vblocks >= 1, "dst_max_vblocks must be >= 1");
  RA_REQUIRE(static_cast<int64_t>(R) * Hkv <= 65535, "R*Hkv must be at most 65535");
  const int64_t row_bytes = static_cast<int64_t>(d) * (dt == RA_BF16 ? 2 : 4);
  if (row_bytes % 16 != 0 || row_bytes > 16384)
    return ra::fail(RA_ERR_UNSUPPORTED, "d*elem_size must be a multiple of 16, at most 16384");
  RA_REQUIRE(k_cache && v_cache && weights && block_table && ctx_lens && kept && new_lens, "NULL pointer");
  RA_REQUIRE(k_cache != v_cache, "k_cache and v_cache must be different buffers");
  RA_REQUIRE(ra::aligned16(k_cache) && ra::aligned16(v_cache) && reinterpret_cast<uintptr_t>(weights) % 4 == 0,
             "the caches must be 16-byte aligned, weights 4-byte aligned");
  RA_REQUIRE(new_lens + R <= ctx_lens || ctx_lens + R <= new_lens, "new_lens must not overlap ctx_lens");
  EvictParams p;
  p.kc = static_cast<uint4*>(k_cache);
  p.vc = static_cast<uint4*>(v_cache);
  p.w = weights;
  p.src = make_paged(block_table, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks);
  p.in_place = dst_block_table == nullptr || dst_block_table == block_table;
  p.dst = p.in_place ? p.src
                     : make_paged(dst_block_table, Hkv, block_size, interleave, pcp, dcp, dst_max_vblocks, num_blocks);
  p.ctx = ctx_lens;
  p.row_words = static_cast<int>(row_bytes / 16);
  p.keep = keep; p.n_sink = n_sink; p.n_recent = n_recent;
  p.kept = kept; p.new_lens = new_lens;
  p.by_words = fast_div(2 * p.row_words);
  // CTAs of a cluster: as many as fill the GPU once (2 per SM), so that few heads still use all of it
  int C = 1;
  while (C < kMaxCluster && static_cast<int64_t>(R) * Hkv * 2 * C <= 152 * 2) C *= 2;
  const int64_t most = ra::ceil_div(ra::ceil_div(static_cast<int64_t>(max_vblocks) * p.src.V, C), 4) * 4;
  p.by_four = interleave % 4 == 0 && ra::aligned16(weights);   // then rows of four tokens are 16-byte words
  p.keys_cap = static_cast<int>(std::min<int64_t>(kKeysCap, most));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, R * Hkv);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.keys_cap) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto* kernel = most <= kKeysCap ? evict_kernel<true> : evict_kernel<false>;
  RA_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysCap * 4));
  RA_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, p));
  return RA_OK;
}
