// Where the tokens of a request lie in the sharded paged cache
// [W, num_blocks, Hkv, bs, d] (vLLM-Ascend "Context Parallel (CP)", section
// "Block table"): token x is in virtual block x / V, V = bs*W, and there at
// o = x % V: device (o / I) % W, slot (o / I) / W * I + o % I.
#pragma once

#include "ra_common.cuh"

namespace {

// Division of n in [0, 2^31) by a fixed d >= 1: q = n * m >> (31 + l), m = ceil(2^(31+l) / d), l = ceil(log2 d)
// (exact because m * d - 2^(31+l) < d <= 2^l).
struct FastDiv {
  uint32_t m, d;
  int sh;
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * m) >> sh);
  }
  __device__ __forceinline__ int div(int n, int& rem) const {
    const int q = div(n);
    rem = n - q * static_cast<int>(d);
    return q;
  }
};

inline FastDiv fast_div(int64_t d) {
  int l = 0;
  while ((int64_t(1) << l) < d) ++l;
  FastDiv f;
  f.d = static_cast<uint32_t>(d);
  f.sh = 31 + l;
  f.m = static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + d - 1) / d);
  return f;
}

struct Paged {
  const int32_t* table;  // [R, max_vb]
  int max_vb, bs, I, W, V, Hkv;
  FastDiv by_V, by_I, by_W, by_WI;
  int64_t num_blocks;
};

// Tokens of a context that the block table can hold, at most 2^30; a longer one is cut.
__device__ __forceinline__ int paged_len(const Paged& c, int32_t ctx, int site) {
  const int64_t table = static_cast<int64_t>(c.max_vb) * c.V, cap = table < (1 << 30) ? table : 1 << 30;
  if (ctx > cap) {
    ra_record_error(RA_ERR_DEVICE_BOUNDS, site);
    return static_cast<int>(cap);
  }
  return ctx < 0 ? 0 : ctx;
}

// Physical block of a request's virtual block, -1 if its id is bad.
__device__ __forceinline__ int64_t paged_block(const Paged& c, int64_t r, int vb, int site) {
  const int32_t b = c.table[r * c.max_vb + vb];
  if (b < 0 || b >= c.num_blocks) {
    ra_record_error(RA_ERR_DEVICE_BOUNDS, site);
    return -1;
  }
  return b;
}

// Row (of d elements, or of one weight) of token x for K/V head g; -1 where its block is bad.
__device__ __forceinline__ int64_t paged_row(const Paged& c, int64_t r, int x, int g, int site) {
  int o;
  const int vb = c.by_V.div(x, o), lbi = c.by_I.div(o), q = c.by_W.div(lbi);
  const int64_t b = paged_block(c, r, vb, site);
  if (b < 0) return -1;
  return (((lbi - q * c.W) * c.num_blocks + b) * c.Hkv + g) * c.bs + q * c.I + (o - lbi * c.I);
}

// What the work division reads of a request.
struct Lens {
  int32_t q_begin, q_end, ctx;
};
__device__ __forceinline__ Lens load_lens(const int32_t* qsl, const int32_t* ctx, int r, int R) {
  if (r >= R) return Lens{0, 0, 0};
  return Lens{qsl[r], qsl[r + 1], ctx[r]};
}

// The request's queries [q0, q0 + n); n = 0 where the range is bad.
__device__ __forceinline__ void query_range(const Lens& x, int64_t T, int& q0, int& n, int site) {
  if (x.q_begin < 0 || x.q_end < x.q_begin || x.q_end > T) {
    ra_record_error(RA_ERR_DEVICE_BOUNDS, site);
    q0 = n = 0;
    return;
  }
  q0 = x.q_begin;
  n = x.q_end - x.q_begin;
}

// Host checks of the sizes that every paged operator shares.
inline ra_status check_paged(int32_t R, int32_t Hkv, int32_t block_size, int32_t interleave, int32_t pcp, int32_t dcp,
                             int32_t max_vblocks, int64_t num_blocks) {
  RA_REQUIRE(R >= 1 && Hkv >= 1 && block_size >= 1 && interleave >= 1 && pcp >= 1 && dcp >= 1 && max_vblocks >= 1 &&
                 num_blocks >= 1,
             "sizes must be >= 1");
  RA_REQUIRE(block_size % interleave == 0,
             "block_size %% cp_kv_cache_interleave_size must be 0 (block_size=%d, interleave=%d)", block_size,
             interleave);
  RA_REQUIRE(static_cast<int64_t>(pcp) * dcp <= 4096, "pcp*dcp too large");
  const int64_t W = static_cast<int64_t>(pcp) * dcp;
  RA_REQUIRE(W * block_size <= (int64_t(1) << 24), "a virtual block holds at most 2^24 tokens");
  RA_REQUIRE(num_blocks < (int64_t(1) << 31) && W * num_blocks < (int64_t(1) << 31) / Hkv,
             "pcp*dcp*num_blocks*Hkv must be below 2^31");
  return RA_OK;
}

inline Paged make_paged(const int32_t* table, int32_t Hkv, int32_t block_size, int32_t interleave, int32_t pcp,
                        int32_t dcp, int32_t max_vblocks, int64_t num_blocks) {
  Paged c;
  c.table = table; c.max_vb = max_vblocks; c.bs = block_size; c.I = interleave;
  c.W = pcp * dcp; c.V = block_size * c.W; c.Hkv = Hkv; c.num_blocks = num_blocks;
  c.by_V = fast_div(c.V); c.by_I = fast_div(c.I); c.by_W = fast_div(c.W);
  c.by_WI = fast_div(static_cast<int64_t>(c.W) * c.I);
  return c;
}

}  // namespace
