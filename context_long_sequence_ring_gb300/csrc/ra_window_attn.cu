// Attention with a sliding window and first tokens that stay visible, over the
// sharded paged cache and on packed sequences: two forms of the kernel in
// ra_chunk_attn.cuh.  The gradient of the latter: ra_window_grad.cu.
#include "ra_chunk_attn.cuh"
#include "ra_window.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_window_attn)

namespace ra {
size_t window_forward_workspace(int d) { return chunk_workspace<WindowPacked>(d); }
}  // namespace ra

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
                                         block_size, interleave, pcp, dcp, max_vblocks, num_blocks, o, out_dt, lse, workspace,
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
  RA_REQUIRE(T >= 0 && R >= 1 && Hq >= 1 && Hkv >= 1 && d >= 1 && T < kFar && T < (int64_t(1) << 31) / Hq &&
                 Hq % Hkv == 0 && Hq / Hkv <= BM,
             "bad sizes");
  *bytes = std::max(ra::window_forward_workspace(d), ra::window_backward_workspace(T, R, Hq, Hkv, d));
  return RA_OK;
}

extern "C" ra_status ra_window_attn_fwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                        const void* v, int64_t v_row_stride, const int32_t* query_start_loc, int64_t T,
                                        int32_t R, int32_t Hq, int32_t Hkv, int32_t d, int32_t window, int32_t n_sink,
                                        float scale, void* o, ra_dtype out_dt, float* lse, void* workspace, size_t ws_bytes,
                                        ra_stream stream) {
  ra::clear_error();
  size_t need = 0;
  ra_status st = check_packed(q, q_row_stride, k, k_row_stride, v, v_row_stride, query_start_loc, T, R, Hq, Hkv, d, window,
                              n_sink, out_dt, workspace, ws_bytes, need);
  if (st != RA_OK || T == 0) return st;
  RA_REQUIRE(o != nullptr && ra::aligned16(o), "o must be given and 16-byte aligned");
  const uint64_t rows = static_cast<uint64_t>(T) * Hq;
  if ((st = ra::check_workspace_apart(ra::Span{workspace, need}, ra::Span{o, rows * d * (out_dt == RA_BF16 ? 2 : 4)},
                                      ra::Span{lse, rows * 4})) != RA_OK)
    return st;
  ChunkArgs a;
  a.c = Paged{};
  a.c.Hkv = Hkv;
  a.lu = 5; a.lupt = 2; a.nsub = 1;
  a.by_vbu = fast_div(1);
  set_chunk_args(a, query_start_loc, nullptr, T, R, Hq, Hkv, d, scale, o, out_dt, lse, workspace);
  a.window = std::min(window, kFar);
  a.n_sink = std::min(n_sink, kFar);
  CUtensorMap mq, mk, mv;
  if ((st = row_map(&mq, q, d, Hq, T, q_row_stride, a.G, a.tpt)) != RA_OK) return st;
  if ((st = row_map(&mk, k, d, Hkv, T, k_row_stride, 1, 32)) != RA_OK) return st;
  if ((st = row_map(&mv, v, d, Hkv, T, v_row_stride, 1, 32)) != RA_OK) return st;
  return d == 128 ? launch_chunk<128, WindowPacked>(mq, mk, mv, a, stream)
                  : launch_chunk<64, WindowPacked>(mq, mk, mv, a, stream);
}
