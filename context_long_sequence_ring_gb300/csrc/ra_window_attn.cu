// Attention with a sliding window and first tokens that stay visible, over the
// sharded paged cache and on packed sequences, and the gradient of the latter.
//
// Mathematics.  The query at position p sees token x iff x <= p and (x > p - window
// or x < n_sink).  O = sum_x e^{s_x - lse} v_x with lse = ln sum_x e^{s_x}, s_x = scale q.k_x.
// Backward, with P = e^{s - lse} and delta = sum dO O of each row:
//   dV = P^T dO,  dS = P (dO V^T - delta),  dQ = scale dS K,  dK = scale dS^T Q.
#include "ra_chunk_attn.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_window_attn)

namespace {

constexpr int kRowThreads = 256;

struct WindowArgs {
  Paged c;                       // of the paged form
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_rs, k_rs, v_rs;      // row strides; paged: q_rs only
  const int32_t *qsl, *ctx;      // ctx NULL: packed sequences
  int64_t T;
  int R, Hq, Hkv, window, n_sink, out_bf16;
  float scale;
  void* o;                       // [T, Hq, D]
  float* lse;
  const __nv_bfloat16 *o_in, *d_o;
  float* delta;                  // [T, Hq]
  void *dq, *dk, *dv;
  int64_t dq_rs, dk_rs, dv_rs;
};

// Request of row t; false for a row of no request.
__device__ __forceinline__ bool find_row(const WindowArgs& a, int64_t t, int& r, int& q0, int& n, int& L) {
  if (t == 0)                    // every range is looked at, by the first row's warps
    for (int i = threadIdx.x & 31; i < a.R; i += 32) query_range(load_lens(a.qsl, a.qsl, i, a.R), a.T, q0, n, 800);
  int lo = 0, hi = a.R - 1;      // first request that ends past t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.qsl[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  r = lo;
  query_range(load_lens(a.qsl, a.ctx ? a.ctx : a.qsl, r, a.R), a.T, q0, n, 800);
  if (t < q0 || t >= q0 + n) return false;
  L = a.ctx ? paged_len(a.c, a.ctx[r], 801) : n;
  return true;
}

template <int D>
__device__ __forceinline__ float dot(const float (&x)[D / 32], const __nv_bfloat16* y) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) s += x[e] * __bfloat162float(y[e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
__device__ __forceinline__ void store_out(void* out, bool bf, int64_t at, float x) {
  if (bf) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
  else static_cast<float*>(out)[at] = x;
}

// dQ of a row and head by a warp, and the row's delta.
template <int D>
__global__ void __launch_bounds__(kRowThreads) window_dq_kernel(const __grid_constant__ WindowArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (w >= a.T * a.Hq) return;
  const int64_t t = w / a.Hq;
  const int h = static_cast<int>(w - t * a.Hq), g = h / (a.Hq / a.Hkv);
  int r, q0, n, L;
  if (!find_row(a, t, r, q0, n, L)) return;
  const int p = static_cast<int>(t - q0), lo = max(0, p - a.window + 1);
  float x[E], y[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = __bfloat162float(a.q[t * a.q_rs + h * D + lane * E + e]) * a.scale;
    y[e] = __bfloat162float(a.d_o[w * D + lane * E + e]);
    acc[e] = 0.f;
  }
  const float delta = dot<D>(y, a.o_in + w * D + lane * E), lse = a.lse[w];
  if (lane == 0) a.delta[w] = delta;
  for (int j = 0; j <= p; ++j) {
    if (j >= a.n_sink && j < lo) j = lo;
    const __nv_bfloat16* k = a.k + (q0 + j) * a.k_rs + g * D + lane * E;
    const float pr = expf(dot<D>(x, k) - lse), ds = pr * (dot<D>(y, a.v + (q0 + j) * a.v_rs + g * D + lane * E) - delta);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += ds * __bfloat162float(k[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) store_out(a.dq, a.out_bf16, t * a.dq_rs + h * D + lane * E + e, acc[e] * a.scale);
}

// dK and dV of a key and K/V head by a warp.
template <int D>
__global__ void __launch_bounds__(kRowThreads) window_dkv_kernel(const __grid_constant__ WindowArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, G = a.Hq / a.Hkv;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (w >= a.T * a.Hkv) return;
  const int64_t t = w / a.Hkv;
  const int g = static_cast<int>(w - t * a.Hkv);
  int r, q0, n, L;
  if (!find_row(a, t, r, q0, n, L)) return;
  const int j = static_cast<int>(t - q0);
  float x[E], y[E], dk[E], dv[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = __bfloat162float(a.k[t * a.k_rs + g * D + lane * E + e]);
    y[e] = __bfloat162float(a.v[t * a.v_rs + g * D + lane * E + e]);
    dk[e] = dv[e] = 0.f;
  }
  const int64_t far = static_cast<int64_t>(j) + a.window;
  const int end = j < a.n_sink || far > n ? n : static_cast<int>(far);
  for (int i = j; i < end; ++i)
    for (int h = g * G; h < (g + 1) * G; ++h) {
      const int64_t at = (q0 + i) * static_cast<int64_t>(a.Hq) + h;
      const __nv_bfloat16 *q = a.q + (q0 + i) * a.q_rs + h * D + lane * E, *d_o = a.d_o + at * D + lane * E;
      const float pr = expf(dot<D>(x, q) * a.scale - a.lse[at]), ds = pr * (dot<D>(y, d_o) - a.delta[at]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        dk[e] += ds * __bfloat162float(q[e]);
        dv[e] += pr * __bfloat162float(d_o[e]);
      }
    }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    store_out(a.dk, a.out_bf16, t * a.dk_rs + g * D + lane * E + e, dk[e] * a.scale);
    store_out(a.dv, a.out_bf16, t * a.dv_rs + g * D + lane * E + e, dv[e]);
  }
}

ra_status check_heads(int64_t T, int32_t R, int32_t Hq, int32_t Hkv, int32_t d, int32_t window, int32_t n_sink, ra_dtype out_dt) {
  RA_REQUIRE(out_dt == RA_F32 || out_dt == RA_BF16, "unknown out dtype");
  RA_REQUIRE(R >= 1 && Hkv >= 1 && Hq >= 1 && Hq % Hkv == 0, "R >= 1 and Hq (%d) a multiple of Hkv (%d) required", Hq, Hkv);
  RA_REQUIRE(T >= 0 && T < (int64_t(1) << 31) / Hq && T < (1 << 30), "T must be in [0, 2^30), T*Hq below 2^31");
  RA_REQUIRE(window >= 1 && n_sink >= 0, "window >= 1 and n_sink >= 0 required");
  if (d != 64 && d != 128) return ra::fail(RA_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (Hq / Hkv > 64) return ra::fail(RA_ERR_UNSUPPORTED, "GQA group %d > 64 not supported", Hq / Hkv);
  return RA_OK;
}

unsigned row_blocks(int64_t rows) { return static_cast<unsigned>(ra::ceil_div(rows, kRowThreads / 32)); }

}  // namespace

// The map of [T, heads, D] rows `stride` elements apart: boxes of 64 columns, box_heads heads, box_rows rows.
namespace {
ra_status row_map(CUtensorMap* map, const void* base, int D, int heads, int64_t rows, int64_t stride, uint32_t box_heads,
                  uint32_t box_rows) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return ra::fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {64, box_heads, box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return ra::fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return RA_OK;
}

constexpr int kFar = 1 << 30;    // no position is further: contexts and sequences are shorter
}  // namespace

extern "C" ra_status ra_cp_window_attn_workspace_size(int32_t Hq, int32_t Hkv, int32_t d, size_t* bytes) {
  ra::clear_error();
  RA_REQUIRE(bytes != nullptr, "bytes is NULL");
  RA_REQUIRE(Hq >= 1 && Hkv >= 1 && d >= 1, "sizes must be >= 1");
  *bytes = chunk_workspace<WindowPaged>(d);
  return RA_OK;
}

extern "C" ra_status ra_cp_window_attn(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                       const int32_t* query_start_loc, const int32_t* ctx_lens, int64_t T, int32_t R,
                                       int32_t Hq, int32_t Hkv, int32_t d, int32_t block_size, int32_t interleave,
                                       int32_t pcp, int32_t dcp, int32_t max_vblocks, int64_t num_blocks, int32_t window,
                                       int32_t n_sink, float scale, void* o, ra_dtype out_dt, float* lse, void* workspace,
                                       size_t ws_bytes, ra_stream stream) {
  ra::clear_error();
  RA_REQUIRE(window >= 1 && n_sink >= 0, "window >= 1 and n_sink >= 0 required");
  const ra_status st = check_chunk_paged(q, k_cache, v_cache, block_table, query_start_loc, ctx_lens, T, R, Hq, Hkv, d,
                                         block_size, interleave, pcp, dcp, max_vblocks, num_blocks, o, out_dt, workspace,
                                         ws_bytes, chunk_workspace<WindowPaged>(d));
  if (st != RA_OK || T == 0) return st;
  ChunkArgs a;
  static_cast<KeyUnits&>(a) =
      make_units(make_paged(block_table, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks));
  set_chunk_args(a, query_start_loc, ctx_lens, T, R, Hq, Hkv, d, scale, o, out_dt, lse, workspace);
  a.window = std::min(window, kFar);
  a.n_sink = std::min(n_sink, kFar);
  return d == 128 ? launch_chunk_paged<128, WindowPaged>(q, k_cache, v_cache, a, stream)
                  : launch_chunk_paged<64, WindowPaged>(q, k_cache, v_cache, a, stream);
}

extern "C" ra_status ra_window_attn_workspace_size(int64_t T, int32_t R, int32_t Hq, int32_t Hkv, int32_t d,
                                                   size_t* bytes) {
  ra::clear_error();
  RA_REQUIRE(bytes != nullptr, "bytes is NULL");
  RA_REQUIRE(T >= 0 && R >= 1 && Hq >= 1 && Hkv >= 1 && d >= 1 && T < kFar && T < (int64_t(1) << 31) / Hq, "bad sizes");
  *bytes = std::max(chunk_workspace<WindowPacked>(d), static_cast<size_t>(T * Hq * 8 + 256));
  return RA_OK;
}

namespace {
ra_status packed_args(WindowArgs& a, const void* q, int64_t q_rs, const void* k, int64_t k_rs, const void* v, int64_t v_rs,
                      const int32_t* qsl, int64_t T, int32_t R, int32_t Hq, int32_t Hkv, int32_t d, int32_t window,
                      int32_t n_sink, float scale, ra_dtype out_dt, void* workspace, size_t ws_bytes) {
  ra_status st = check_heads(T, R, Hq, Hkv, d, window, n_sink, out_dt);
  if (st != RA_OK) return st;
  const int64_t lim = int64_t(1) << 31;
  RA_REQUIRE(q_rs >= static_cast<int64_t>(Hq) * d && k_rs >= static_cast<int64_t>(Hkv) * d &&
                 v_rs >= static_cast<int64_t>(Hkv) * d && q_rs < lim && k_rs < lim && v_rs < lim,
             "row strides must be at least heads * d, below 2^31");
  RA_REQUIRE(q_rs % 8 == 0 && k_rs % 8 == 0 && v_rs % 8 == 0, "row strides must be multiples of 8 elements");
  if (T == 0) return RA_OK;
  RA_REQUIRE(q && k && v && qsl && workspace, "NULL pointer");
  RA_REQUIRE(ra::aligned16(q) && ra::aligned16(k) && ra::aligned16(v) && ra::aligned16(workspace),
             "q, k, v and workspace must be 16-byte aligned");
  size_t need = 0;
  if ((st = ra_window_attn_workspace_size(T, R, Hq, Hkv, d, &need)) != RA_OK) return st;
  RA_REQUIRE(ws_bytes >= need, "workspace too small (%zu < %zu bytes)", ws_bytes, need);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_rs = q_rs; a.k_rs = k_rs; a.v_rs = v_rs;
  a.qsl = qsl; a.ctx = nullptr; a.T = T; a.R = R; a.Hq = Hq; a.Hkv = Hkv;
  a.window = window; a.n_sink = n_sink; a.out_bf16 = out_dt == RA_BF16;
  a.scale = scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(d));
  return RA_OK;
}
}  // namespace

extern "C" ra_status ra_window_attn_fwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                        const void* v, int64_t v_row_stride, const int32_t* query_start_loc, int64_t T,
                                        int32_t R, int32_t Hq, int32_t Hkv, int32_t d, int32_t window, int32_t n_sink,
                                        float scale, void* o, ra_dtype out_dt, float* lse, void* workspace, size_t ws_bytes,
                                        ra_stream stream) {
  ra::clear_error();
  WindowArgs a = {};
  const ra_status st = packed_args(a, q, q_row_stride, k, k_row_stride, v, v_row_stride, query_start_loc, T, R, Hq, Hkv, d,
                                   window, n_sink, scale, out_dt, workspace, ws_bytes);
  if (st != RA_OK) return st;
  if (T == 0) return RA_OK;
  RA_REQUIRE(o != nullptr && ra::aligned16(o), "o must be given and 16-byte aligned");
  ChunkArgs c;
  c.c = Paged{};
  c.c.Hkv = Hkv;
  c.lu = 5; c.lupt = 2; c.nsub = 1;
  c.by_vbu = fast_div(1);
  set_chunk_args(c, query_start_loc, nullptr, T, R, Hq, Hkv, d, scale, o, out_dt, lse, workspace);
  c.window = std::min(window, kFar);
  c.n_sink = std::min(n_sink, kFar);
  CUtensorMap mq, mk, mv;
  ra_status s;
  if ((s = row_map(&mq, q, d, Hq, T, q_row_stride, c.G, c.tpt)) != RA_OK) return s;
  if ((s = row_map(&mk, k, d, Hkv, T, k_row_stride, 1, 32)) != RA_OK) return s;
  if ((s = row_map(&mv, v, d, Hkv, T, v_row_stride, 1, 32)) != RA_OK) return s;
  return d == 128 ? launch_chunk<128, WindowPacked>(mq, mk, mv, c, stream)
                  : launch_chunk<64, WindowPacked>(mq, mk, mv, c, stream);
}

extern "C" ra_status ra_window_attn_bwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                        const void* v, int64_t v_row_stride, const void* o, const float* lse,
                                        const void* d_o, const int32_t* query_start_loc, int64_t T, int32_t R, int32_t Hq,
                                        int32_t Hkv, int32_t d, int32_t window, int32_t n_sink, float scale, void* dq,
                                        int64_t dq_row_stride, void* dk, int64_t dk_row_stride, void* dv,
                                        int64_t dv_row_stride, ra_dtype out_dt, void* workspace, size_t ws_bytes,
                                        ra_stream stream) {
  ra::clear_error();
  WindowArgs a = {};
  const ra_status st = packed_args(a, q, q_row_stride, k, k_row_stride, v, v_row_stride, query_start_loc, T, R, Hq, Hkv, d,
                                   window, n_sink, scale, out_dt, workspace, ws_bytes);
  if (st != RA_OK) return st;
  const int64_t lim = int64_t(1) << 31, out_words = out_dt == RA_BF16 ? 8 : 4;
  RA_REQUIRE(dq_row_stride >= static_cast<int64_t>(Hq) * d && dk_row_stride >= static_cast<int64_t>(Hkv) * d &&
                 dv_row_stride >= static_cast<int64_t>(Hkv) * d && dq_row_stride < lim && dk_row_stride < lim &&
                 dv_row_stride < lim,
             "row strides must be at least heads * d, below 2^31");
  RA_REQUIRE(dq_row_stride % out_words == 0 && dk_row_stride % out_words == 0 && dv_row_stride % out_words == 0,
             "row strides must be multiples of 16 bytes");
  if (T == 0) return RA_OK;
  RA_REQUIRE(o && lse && d_o && dq && dk && dv, "NULL pointer");
  RA_REQUIRE(ra::aligned16(o) && ra::aligned16(d_o) && ra::aligned16(dq) && ra::aligned16(dk) && ra::aligned16(dv),
             "o, d_o, dq, dk and dv must be 16-byte aligned");
  a.o_in = static_cast<const __nv_bfloat16*>(o);
  a.d_o = static_cast<const __nv_bfloat16*>(d_o);
  a.lse = const_cast<float*>(lse);
  a.delta = static_cast<float*>(workspace);
  a.dq = dq; a.dk = dk; a.dv = dv; a.dq_rs = dq_row_stride; a.dk_rs = dk_row_stride; a.dv_rs = dv_row_stride;
  auto launch = [&](auto dim) -> ra_status {
    constexpr int D = decltype(dim)::value;
    window_dq_kernel<D><<<row_blocks(T * Hq), kRowThreads, 0, stream>>>(a);
    RA_LAUNCH_CHECK("window_dq_kernel");
    window_dkv_kernel<D><<<row_blocks(T * Hkv), kRowThreads, 0, stream>>>(a);
    RA_LAUNCH_CHECK("window_dkv_kernel");
    return RA_OK;
  };
  return d == 128 ? launch(std::integral_constant<int, 128>{}) : launch(std::integral_constant<int, 64>{});
}
