// The attention weight that every cached token receives from a chunk of
// queries: the column sums of the softmax, from the scores and the rows' LSE.
//
// Simple form: one warp per (token, K/V head) runs over the queries.
#include <math_constants.h>

#include <algorithm>

#include "ra_paged.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_attn_weights)

namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct WeightParams {
  const __nv_bfloat16 *q, *kc;
  const float* lse;
  const int32_t *qsl, *ctx;
  Paged c;
  int64_t T;
  int R, Hq, G, causal;
  float scale_log2;
  const float* w_in;
  float* w_out;
};

template <int D>
__global__ void __launch_bounds__(256) weights_simple_kernel(const WeightParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y, g = blockIdx.z;
  int q0, n;
  query_range(p.qsl, r, p.T, q0, n, 600);
  const int L = paged_len(p.c, p.ctx[r], 601);
  const int64_t pos0 = p.causal ? static_cast<int64_t>(p.ctx[r]) - n : L;  // position of the first query
  for (int x = blockIdx.x * 8 + (threadIdx.x >> 5); x < L; x += gridDim.x * 8) {
    const int64_t at = paged_row(p.c, r, x, g, 602);
    if (at < 0) continue;
    float k[E];
#pragma unroll
    for (int e = 0; e < E; ++e) k[e] = __bfloat162float(p.kc[at * D + lane + 32 * e]) * p.scale_log2;
    float w = 0.f;
    for (int64_t i = pos0 >= x ? 0 : x - pos0; i < n; ++i)
      for (int h = g * p.G; h < (g + 1) * p.G; ++h) {
        const int64_t row = (q0 + i) * p.Hq + h;
        const float lse = p.lse[row];
        if (lse == -CUDART_INF_F) continue;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += k[e] * __bfloat162float(p.q[row * D + lane + 32 * e]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        w += exp2f(s - lse * kLog2e);
      }
    if (lane == 0) p.w_out[at] = (p.w_in && x < pos0 ? p.w_in[at] : 0.f) + w;
  }
}

}  // namespace

extern "C" ra_status ra_cp_attn_weights(const void* q, const float* lse, const void* k_cache,
                                        const int32_t* block_table, const int32_t* query_start_loc,
                                        const int32_t* ctx_lens, int64_t T, int32_t R, int32_t Hq, int32_t Hkv,
                                        int32_t d, int32_t block_size, int32_t interleave, int32_t pcp, int32_t dcp,
                                        int32_t max_vblocks, int64_t num_blocks, int32_t causal, float scale,
                                        const float* w_in, float* w_out, ra_stream stream) {
  ra::clear_error();
  ra_status st = check_paged(R, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks);
  if (st != RA_OK) return st;
  RA_REQUIRE(Hq >= 1 && Hq % Hkv == 0, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
  RA_REQUIRE(T >= 0 && T < (int64_t(1) << 31) / Hq, "T*Hq must be in [0, 2^31)");
  if (d != 64 && d != 128) return ra::fail(RA_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (Hq / Hkv > 64) return ra::fail(RA_ERR_UNSUPPORTED, "GQA group %d > 64 not supported", Hq / Hkv);
  if (block_size % 16 != 0) return ra::fail(RA_ERR_UNSUPPORTED, "block_size must be a multiple of 16");
  RA_REQUIRE((T == 0 || (q && lse)) && k_cache && block_table && query_start_loc && ctx_lens && w_out, "NULL pointer");
  RA_REQUIRE(ra::aligned16(q) && ra::aligned16(k_cache), "q and k_cache must be 16-byte aligned");
  RA_REQUIRE(reinterpret_cast<uintptr_t>(lse) % 4 == 0 && reinterpret_cast<uintptr_t>(w_in) % 4 == 0 &&
                 reinterpret_cast<uintptr_t>(w_out) % 4 == 0,
             "lse and the weights must be 4-byte aligned");
  RA_REQUIRE(R <= 65535 && Hkv <= 65535, "R and Hkv must be at most 65535");
  WeightParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.kc = static_cast<const __nv_bfloat16*>(k_cache);
  p.lse = lse; p.qsl = query_start_loc; p.ctx = ctx_lens;
  p.c = make_paged(block_table, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks);
  p.T = T; p.R = R; p.Hq = Hq; p.G = Hq / Hkv; p.causal = causal ? 1 : 0;
  p.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(d))) * kLog2e;
  p.w_in = w_in; p.w_out = w_out;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ra::ceil_div(static_cast<int64_t>(max_vblocks) * p.c.V, 8), 512)),
                  R, Hkv);
  if (d == 128) weights_simple_kernel<128><<<grid, 256, 0, stream>>>(p);
  else weights_simple_kernel<64><<<grid, 256, 0, stream>>>(p);
  RA_LAUNCH_CHECK("weights_simple_kernel");
  return RA_OK;
}
