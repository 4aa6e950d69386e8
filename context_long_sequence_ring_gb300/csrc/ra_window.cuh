// Shared host pieces of the window attention on packed sequences, forward and backward.
#pragma once

#include <algorithm>

#include "ra_attn_tc.cuh"
#include "ra_paged.cuh"

namespace {

constexpr int kFar = 1 << 30;    // no position is further: contexts and sequences are shorter

// The map of [rows, heads, D] rows `stride` elements apart: boxes of 64 columns, box_heads heads, box_rows rows.
inline ra_status row_map(CUtensorMap* map, const void* base, int D, int heads, int64_t rows, int64_t stride,
                         uint32_t box_heads, uint32_t box_rows) {
  return bf16_map(map, base, D, heads, rows, D, stride, box_heads, box_rows);
}

// What both directions require of their arguments; `need`: bytes of workspace.
inline ra_status check_packed(const void* q, int64_t q_rs, const void* k, int64_t k_rs, const void* v, int64_t v_rs,
                              const int32_t* qsl, int64_t T, int32_t R, int32_t Hq, int32_t Hkv, int32_t d, int32_t window,
                              int32_t n_sink, ra_dtype out_dt, const void* workspace, size_t ws_bytes, size_t& need) {
  RA_REQUIRE(out_dt == RA_F32 || out_dt == RA_BF16, "unknown out dtype");
  RA_REQUIRE(R >= 1 && Hkv >= 1 && Hq >= 1 && Hq % Hkv == 0, "R >= 1 and Hq (%d) a multiple of Hkv (%d) required", Hq, Hkv);
  RA_REQUIRE(T >= 0 && T < kFar && T < (int64_t(1) << 31) / Hq, "T must be in [0, 2^30), T*Hq below 2^31");
  RA_REQUIRE(window >= 1 && n_sink >= 0, "window >= 1 and n_sink >= 0 required");
  if (d != 64 && d != 128) return ra::fail(RA_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", d);
  if (Hq / Hkv > 64) return ra::fail(RA_ERR_UNSUPPORTED, "GQA group %d > 64 not supported", Hq / Hkv);
  const int64_t lim = int64_t(1) << 31;
  RA_REQUIRE(q_rs >= static_cast<int64_t>(Hq) * d && k_rs >= static_cast<int64_t>(Hkv) * d &&
                 v_rs >= static_cast<int64_t>(Hkv) * d && q_rs < lim && k_rs < lim && v_rs < lim,
             "row strides must be at least heads * d, below 2^31");
  RA_REQUIRE(q_rs % 8 == 0 && k_rs % 8 == 0 && v_rs % 8 == 0, "row strides must be multiples of 8 elements");
  if (T == 0) return RA_OK;
  RA_REQUIRE(q && k && v && qsl && workspace, "NULL pointer");
  RA_REQUIRE(ra::aligned16(q) && ra::aligned16(k) && ra::aligned16(v) && ra::aligned16(workspace),
             "q, k, v and workspace must be 16-byte aligned");
  const ra_status st = ra_window_attn_workspace_size(T, R, Hq, Hkv, d, &need);
  if (st != RA_OK) return st;
  RA_REQUIRE(ws_bytes >= need, "workspace too small (%zu < %zu bytes)", ws_bytes, need);
  const int64_t qw = static_cast<int64_t>(Hq) * d * 2, kw = static_cast<int64_t>(Hkv) * d * 2;
  return ra::check_workspace_apart(ra::Span{workspace, need}, ra::row_span(q, T, 2 * q_rs, qw), ra::row_span(k, T, 2 * k_rs, kw),
                                   ra::row_span(v, T, 2 * v_rs, kw), ra::Span{qsl, (R + 1ull) * 4});
}

}  // namespace

namespace ra {
size_t window_forward_workspace(int d);                                              // in ra_window_attn.cu
size_t window_backward_workspace(int64_t T, int32_t R, int32_t Hq, int32_t Hkv, int32_t d);   // in ra_window_grad.cu
}  // namespace ra
