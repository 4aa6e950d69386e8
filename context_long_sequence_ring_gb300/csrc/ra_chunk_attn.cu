// Attention of a chunk of new tokens per request over the sharded paged cache:
// the causal form of the kernel in ra_chunk_attn.cuh.
#include "ra_chunk_attn.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_chunk_attn)

extern "C" ra_status ra_cp_chunk_attn_workspace_size(int32_t Hq, int32_t Hkv, int32_t d, size_t* bytes) {
  ra::clear_error();
  RA_REQUIRE(bytes != nullptr, "bytes is NULL");
  RA_REQUIRE(Hq >= 1 && Hkv >= 1 && d >= 1, "sizes must be >= 1");
  *bytes = chunk_workspace<CausalPaged>(d);
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
  const ra_status st = check_chunk_paged(q, k_cache, v_cache, block_table, query_start_loc, ctx_lens, T, R, Hq, Hkv, d,
                                         block_size, interleave, pcp, dcp, max_vblocks, num_blocks, o, out_dt, lse, workspace,
                                         ws_bytes, chunk_workspace<CausalPaged>(d));
  if (st != RA_OK || T == 0) return st;
  ChunkArgs a;
  static_cast<KeyUnits&>(a) =
      make_units(make_paged(block_table, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks));
  set_chunk_args(a, query_start_loc, ctx_lens, T, R, Hq, Hkv, d, scale, o, out_dt, lse, workspace);
  a.causal = causal ? 1 : 0;
  return d == 128 ? launch_chunk_paged<128, CausalPaged>(q, k_cache, v_cache, a, stream)
                  : launch_chunk_paged<64, CausalPaged>(q, k_cache, v_cache, a, stream);
}
