// Shared host and device helpers of libringattn (no attention arithmetic).
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "ringattn.h"

namespace ra {

// ---------------------------------------------------------------- host side

// Record the thread-local error text (printf-style) and return `s`.
ra_status fail(ra_status s, const char* fmt, ...);
// Map a CUDA error to RA_ERR_CUDA with context; RA_OK on cudaSuccess.
ra_status cuda_status(cudaError_t e, const char* what);
// Clears the thread-local error text at the start of an entry point.
void clear_error();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether rows of a (`wa` bytes, `sa` apart) and of b share bytes: rows at the same distance lie side by side or not at
// all; at different ones, nothing is said of rows whose spans meet.
inline bool rows_meet(const void* pa, int64_t sa, int64_t wa, const void* pb, int64_t sb, int64_t wb, int64_t T) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(pa), b0 = reinterpret_cast<uintptr_t>(pb);
  const uintptr_t a1 = a0 + (T - 1) * sa + wa, b1 = b0 + (T - 1) * sb + wb;
  if (a1 <= b0 || b1 <= a0) return false;
  if (T == 1 || sa != sb || sa <= 0) return true;
  const int64_t off = b0 >= a0 ? static_cast<int64_t>((b0 - a0) % sa) : sa - 1 - static_cast<int64_t>((a0 - b0 - 1) % sa);
  return off < wa || off + wb > sa;
}

// Bytes [p, p + n); of [T, w] rows s apart, from the first to the last.
struct Span {
  const void* p;
  uint64_t n;
};
inline Span row_span(const void* p, int64_t T, int64_t s, int64_t w) { return Span{p, static_cast<uint64_t>((T - 1) * s + w)}; }
inline bool spans_meet(const Span& a, const Span& b) {
  const uint64_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && x < y + b.n && y < x + a.n;
}
// A workspace lies over none of what a call reads and writes.
template <class... S>
ra_status check_workspace_apart(const Span& workspace, const S&... others) {
  if ((spans_meet(workspace, others) || ...))
    return fail(RA_ERR_INVALID_ARG, "the workspace must not overlap what the call reads and writes");
  return RA_OK;
}

// Per-module device error words are fetched (and cleared) through these.
int fetch_error_api(int* where);
int fetch_error_cache(int* where);
int fetch_error_decode(int* where);
int fetch_error_attn_f32(int* where);
int fetch_error_attn_bf16(int* where);
int fetch_error_attn_block(int* where);
int fetch_error_rope(int* where);
int fetch_error_ring_step(int* where);
int fetch_error_rope_apply(int* where);
int fetch_error_chunk_attn(int* where);
int fetch_error_attn_weights(int* where);
int fetch_error_evict(int* where);
int fetch_error_rope_append(int* where);
int fetch_error_window_attn(int* where);
int fetch_error_window_grad(int* where);

}  // namespace ra

#define RA_REQUIRE(cond, ...)                                 \
  do {                                                        \
    if (!(cond)) return ra::fail(RA_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)

#define RA_CUDA_TRY(expr)                                     \
  do {                                                        \
    cudaError_t e_ = (expr);                                  \
    if (e_ != cudaSuccess) return ra::cuda_status(e_, #expr); \
  } while (0)

// Launch-error check after a <<<>>> launch.
#define RA_LAUNCH_CHECK(name) RA_CUDA_TRY(cudaGetLastError())

// ---------------------------------------------------------------- device side
// Each translation unit that includes this header gets its own error word
// (no relocatable device code is needed); the module's fetch function reads
// and clears it.
static __device__ int ra_err_word[2];

#define RA_DEFINE_ERROR_FETCH(fn)                                                  \
  namespace ra {                                                                   \
  int fn(int* where) {                                                             \
    int w[2] = {0, 0};                                                             \
    if (cudaMemcpyFromSymbol(w, ra_err_word, sizeof(w)) != cudaSuccess) return -1; \
    if (w[0] != 0) {                                                               \
      int z[2] = {0, 0};                                                           \
      if (cudaMemcpyToSymbol(ra_err_word, z, sizeof(z)) != cudaSuccess) return -1; \
    }                                                                              \
    if (where) *where = w[1];                                                      \
    return w[0];                                                                   \
  }                                                                                \
  }

__device__ __forceinline__ void ra_record_error(int status, int where) {
  if (atomicCAS(&ra_err_word[0], 0, status) == 0) atomicExch(&ra_err_word[1], where);
}
