// Attention of a chunk of new tokens per request over the sharded paged cache.
//
// Simple form: one warp per (query, head) runs the softmax over the visible
// tokens in one pass, with a running maximum and sum in fp32.
#include <math_constants.h>

#include <algorithm>

#include "ra_paged.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_chunk_attn)

namespace {

constexpr float kLn2 = 0.6931471805599453f;

struct ChunkParams {
  const __nv_bfloat16 *q, *kc, *vc;
  const int32_t *qsl, *ctx;
  Paged c;
  int64_t T;
  int R, Hq, G, causal;
  float scale_log2;
  void* o;
  float* lse;
};

// Largest r with qsl[r] <= t, of requests 0 .. R-1.
__device__ __forceinline__ int request_of(const int32_t* __restrict__ qsl, int R, int64_t t) {
  int lo = 0, hi = R - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(qsl[mid]) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int D, bool OUT_BF16>
__global__ void __launch_bounds__(256) chunk_simple_kernel(const ChunkParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (blockIdx.x == 0) {
    int a, b;
    for (int i = threadIdx.x; i < p.R; i += blockDim.x) query_range(p.qsl, i, p.T, a, b, 500);
  }
  if (row >= p.T * p.Hq) return;
  const int64_t t = row / p.Hq;
  const int h = static_cast<int>(row % p.Hq), g = h / p.G;
  const int r = request_of(p.qsl, p.R, t);
  int q0, n;
  query_range(p.qsl, r, p.T, q0, n, 500);
  if (t < q0 || t >= q0 + n) return;
  const int L = paged_len(p.c, p.ctx[r], 501);
  const int64_t last = p.causal ? static_cast<int64_t>(p.ctx[r]) - n + (t - q0) : L - 1;
  const int seen = static_cast<int>(last + 1 < L ? last + 1 : L);
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[row * D + lane + 32 * e]) * p.scale_log2;
    acc[e] = 0.f;
  }
  float m = -CUDART_INF_F, l = 0.f;
  for (int x = 0; x < seen; ++x) {
    const int64_t at = paged_row(p.c, r, x, g, 502);
    if (at < 0) continue;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * __bfloat162float(p.kc[at * D + lane + 32 * e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, s);
    if (mn == -CUDART_INF_F) continue;
    const float a = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * __bfloat162float(p.vc[at * D + lane + 32 * e]);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (OUT_BF16) static_cast<__nv_bfloat16*>(p.o)[row * D + lane + 32 * e] = __float2bfloat16_rn(acc[e] * inv);
    else static_cast<float*>(p.o)[row * D + lane + 32 * e] = acc[e] * inv;
  }
  if (p.lse && lane == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -CUDART_INF_F;
}

}  // namespace

extern "C" ra_status ra_cp_chunk_attn_workspace_size(int32_t Hq, int32_t Hkv, int32_t d, size_t* bytes) {
  ra::clear_error();
  RA_REQUIRE(bytes != nullptr, "bytes is NULL");
  RA_REQUIRE(Hq >= 1 && Hkv >= 1 && d >= 1, "sizes must be >= 1");
  *bytes = 16;
  return RA_OK;
}

extern "C" ra_status ra_cp_chunk_attn(const void* q, const void* k_cache, const void* v_cache,
                                      const int32_t* block_table, const int32_t* query_start_loc,
                                      const int32_t* ctx_lens, int64_t T, int32_t R, int32_t Hq, int32_t Hkv,
                                      int32_t d, int32_t block_size, int32_t interleave, int32_t pcp, int32_t dcp,
                                      int32_t max_vblocks, int64_t num_blocks, int32_t causal, float scale, void* o,
                                      ra_dtype out_dt, float* lse, void* workspace, size_t ws_bytes,
                                      ra_stream stream) {
  ra::clear_error();
  ra_status st = check_paged(R, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks);
  if (st != RA_OK) return st;
  RA_REQUIRE(out_dt == RA_F32 || out_dt == RA_BF16, "unknown out dtype");
  RA_REQUIRE(Hq >= 1 && Hq % Hkv == 0, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
  RA_REQUIRE(T >= 0 && T < (int64_t(1) << 31) / Hq, "T*Hq must be in [0, 2^31)");
  if (d != 64 && d != 128) return ra::fail(RA_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (Hq / Hkv > 64) return ra::fail(RA_ERR_UNSUPPORTED, "GQA group %d > 64 not supported", Hq / Hkv);
  if (block_size % 16 != 0) return ra::fail(RA_ERR_UNSUPPORTED, "block_size must be a multiple of 16");
  if (T == 0) return RA_OK;
  RA_REQUIRE(q && k_cache && v_cache && block_table && query_start_loc && ctx_lens && o && workspace, "NULL pointer");
  RA_REQUIRE(ra::aligned16(q) && ra::aligned16(k_cache) && ra::aligned16(v_cache) && ra::aligned16(o) &&
                 ra::aligned16(workspace),
             "q, the caches, o and workspace must be 16-byte aligned");
  size_t need = 0;
  if ((st = ra_cp_chunk_attn_workspace_size(Hq, Hkv, d, &need)) != RA_OK) return st;
  RA_REQUIRE(ws_bytes >= need, "workspace too small (%zu < %zu bytes)", ws_bytes, need);
  ChunkParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kc = static_cast<const __nv_bfloat16*>(k_cache);
  p.vc = static_cast<const __nv_bfloat16*>(v_cache);
  p.qsl = query_start_loc; p.ctx = ctx_lens;
  p.c = make_paged(block_table, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks);
  p.T = T; p.R = R; p.Hq = Hq; p.G = Hq / Hkv; p.causal = causal ? 1 : 0;
  p.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(d))) * 1.4426950408889634f;
  p.o = o; p.lse = lse;
  const unsigned blocks = static_cast<unsigned>(ra::ceil_div(T * Hq, 8));
  const bool bf = out_dt == RA_BF16;
  if (d == 128) {
    if (bf) chunk_simple_kernel<128, true><<<blocks, 256, 0, stream>>>(p);
    else chunk_simple_kernel<128, false><<<blocks, 256, 0, stream>>>(p);
  } else {
    if (bf) chunk_simple_kernel<64, true><<<blocks, 256, 0, stream>>>(p);
    else chunk_simple_kernel<64, false><<<blocks, 256, 0, stream>>>(p);
  }
  RA_LAUNCH_CHECK("chunk_simple_kernel");
  return RA_OK;
}
