// Eviction from the sharded paged cache by accumulated attention weight, per
// K/V head, and the packing of what is kept.
//
// Mathematics.  The weights map to 32-bit keys in their order (NaN 0, -0 as
// +0), and a radix select finds the key of the m-th heaviest token of the
// middle part, m = keep - n_sink - n_recent, 8 bits at a time from the top:
// all larger keys are kept, and of the equal ones the first as many as are
// missing.  A scan over the tokens in order then numbers the kept ones.
#include <algorithm>

#include "ra_paged.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_evict)

namespace {

constexpr int kThreads = 1024;
constexpr int kRowWords = 16;  // 16-byte words of a batch that a thread holds

struct EvictParams {
  uint4 *kc, *vc;
  float* w;
  Paged src, dst;  // dst.table may be src.table
  const int32_t* ctx;
  int row_words, keep, n_sink, n_recent, in_place;
  int32_t *kept, *new_lens;
};

// Order-preserving key of a weight.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block of a 0/1 flag; total of the block in `sum`.
__device__ __forceinline__ int block_rank(bool flag, int* warp_sums, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned b = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 0) warp_sums[warp] = __popc(b);
  __syncthreads();
  int before = 0;
  sum = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    const int c = warp_sums[i];
    if (i < warp) before += c;
    sum += c;
  }
  return before + __popc(b & ((1u << lane) - 1));
}

__global__ void __launch_bounds__(kThreads) evict_simple_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sums[kThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int r = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
  const int N = paged_len(p.src, p.ctx[r], 700);
  const int n_new = min(N, p.keep);
  int32_t* kept = p.kept + (static_cast<int64_t>(r) * p.src.Hkv + g) * p.keep;
  if (g == 0 && tid == 0) p.new_lens[r] = n_new;
  for (int j = n_new + tid; j < p.keep; j += kThreads) kept[j] = -1;

  if (N <= p.keep) {
    for (int j = tid; j < N; j += kThreads) kept[j] = j;
  } else {
    const int m0 = p.n_sink, m1 = N - p.n_recent;  // the middle part [m0, m1)
    auto key = [&](int x) {
      const int64_t at = paged_row(p.src, r, x, g, 701);
      return at < 0 ? 0u : key_of(p.w[at]);
    };
    int need = p.keep - p.n_sink - p.n_recent;
    uint32_t prefix = 0;
    if (need > 0) {
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int x = m0 + tid; x < m1; x += kThreads) {
          const uint32_t k = key(x);
          if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
          int b = 255;
          for (; b > 0 && hist[b] < need; --b) need -= hist[b];
          s_prefix = prefix | (static_cast<uint32_t>(b) << shift);
          s_need = need;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        __syncthreads();
      }
    } else {
      prefix = 0xffffffffu;  // above every key of a number
    }
    // tokens with a larger key and the first `need` of the equal ones
    int out = 0, ties = 0;
    for (int x0 = 0; x0 < N; x0 += kThreads) {
      const int x = x0 + tid;
      const bool mid = x >= m0 && x < m1;
      const uint32_t k = mid ? key(x) : 0u;
      int sum;
      const bool tie = mid && k == prefix;
      const int tr = ties + block_rank(tie, warp_sums, sum);
      ties += sum;
      const bool sel = x < N && (!mid || k > prefix || (tie && tr < need));
      const int at = out + block_rank(sel, warp_sums, sum);
      out += sum;
      if (sel) kept[at] = x;
    }
  }
  __syncthreads();
  if (p.in_place && N <= p.keep) return;

  // Pack in ascending batches.  A batch is read whole before it is written,
  // and token j comes from a place >= j, so no later batch reads what an
  // earlier one wrote, in place or not.
  const int rw = p.row_words, words = 2 * rw;
  const int per = (kThreads * kRowWords) / words > 0 ? (kThreads * kRowWords) / words : 1;
  for (int j0 = 0; j0 < n_new; j0 += per) {
    const int nj = min(per, n_new - j0);
    uint4 v[kRowWords];
#pragma unroll
    for (int u = 0; u < kRowWords; ++u) {
      const int e = u * kThreads + tid, j = e / words, c = e % words;
      if (j < nj) {
        const int64_t at = paged_row(p.src, r, kept[j0 + j], g, 701);
        v[u] = at < 0 ? make_uint4(0, 0, 0, 0) : (c < rw ? p.kc[at * rw + c] : p.vc[at * rw + c - rw]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kRowWords; ++u) {
      const int e = u * kThreads + tid, j = e / words, c = e % words;
      if (j < nj) {
        const int vb = (j0 + j) / p.dst.V;
        const int64_t at = vb < p.dst.max_vb ? paged_row(p.dst, r, j0 + j, g, 702) : -1;
        if (vb >= p.dst.max_vb) ra_record_error(RA_ERR_DEVICE_BOUNDS, 703);
        if (at >= 0) (c < rw ? p.kc[at * rw + c] : p.vc[at * rw + c - rw]) = v[u];
      }
    }
  }
  for (int j0 = 0; j0 < n_new; j0 += kThreads) {
    const int j = j0 + tid;
    float w = 0.f;
    if (j < n_new) {
      const int64_t at = paged_row(p.src, r, kept[j], g, 701);
      if (at >= 0) w = p.w[at];
    }
    __syncthreads();
    if (j < n_new && j / p.dst.V < p.dst.max_vb) {
      const int64_t at = paged_row(p.dst, r, j, g, 702);
      if (at >= 0) p.w[at] = w;
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
  RA_REQUIRE(keep >= 1 && n_sink >= 0 && n_recent >= 0 && static_cast<int64_t>(n_sink) + n_recent <= keep,
             "keep >= 1 and 0 <= n_sink + n_recent <= keep required (keep %d, n_sink %d, n_recent %d)", keep, n_sink,
             n_recent);
  RA_REQUIRE(dst_block_table == nullptr || dst_max_vblocks >= 1, "dst_max_vblocks must be >= 1");
  RA_REQUIRE(R <= 65535 && Hkv <= 65535, "R and Hkv must be at most 65535");
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
  evict_simple_kernel<<<dim3(R, Hkv), kThreads, 0, stream>>>(p);
  RA_LAUNCH_CHECK("evict_simple_kernel");
  return RA_OK;
}
