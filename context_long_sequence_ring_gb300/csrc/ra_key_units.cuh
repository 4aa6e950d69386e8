// Key tiles over the sharded paged cache, as the tensor-core kernels on it read
// them where they lie.
//
// A "unit" is u consecutive slots of a block on one device, one TMA box per 64
// columns.  Units are ordered by virtual block, slot, device, so that a prefix of
// the units covers a prefix of the context up to one interleave group; a tile is
// 128/u units.  Within a unit positions grow with the slot, so that every mask
// is a prefix per unit.  u = 32 where the block size allows, else 16: with u = 64
// and 128 the last virtual block of a sharded cache is read more coarsely
// (chunk attention of 48 requests of 2k-16k tokens on 8 devices: 283 us at 32, 294 at
// 64, 348 at 128, before the loads left L2 first; one long context is the same within 1 %).
#pragma once

#include "ra_attn_tc.cuh"
#include "ra_paged.cuh"

namespace {

struct KeyUnits {
  Paged c;
  int lu, lupt, nsub;   // log2 slots of a unit, log2 units of a tile, units of a block
  FastDiv by_vbu;       // by the units of a virtual block
};

inline KeyUnits make_units(const Paged& c) {
  KeyUnits a;
  a.c = c;
  a.lu = c.bs % 32 == 0 ? 5 : 4;
  a.lupt = 7 - a.lu;
  a.nsub = c.bs >> a.lu;
  a.by_vbu = fast_div(static_cast<int64_t>(a.nsub) * c.W);
  return a;
}

// Units that hold a token below lim: a prefix of the units.
__device__ __forceinline__ int units_below(const KeyUnits& a, int lim) {
  if (lim <= 0) return 0;
  int o, rem;
  int k = a.c.by_V.div(lim, o) * a.nsub * a.c.W;
  if (o > 0) {
    const int q = a.c.by_WI.div(o - 1, rem);
    const int sub = (q * a.c.I + min(rem, a.c.I - 1)) >> a.lu;   // last unit row with a token below
    int off;
    const int first = a.c.by_I.div(sub << a.lu, off) * a.c.W * a.c.I + off;
    k += sub * a.c.W + min(a.c.W, a.c.by_I.div(o - first + a.c.I - 1));
  }
  return k;
}

// Units from the start all of whose tokens are below lim.
__device__ __forceinline__ int units_within(const KeyUnits& a, int lim) {
  int o;
  const int vb = a.c.by_V.div(lim, o);
  return (vb * a.nsub + ((a.c.by_WI.div(o) * a.c.I) >> a.lu)) * a.c.W;
}

// Visible slots (a prefix, 0..u) of unit (vb, sub, w) for a row that sees positions below lim.
__device__ __forceinline__ int unit_visible(const KeyUnits& a, int vb, int sub, int w, int lim) {
  const int y = lim - vb * a.c.V - w * a.c.I;
  if (y <= 0) return 0;
  int part;
  const int q = a.c.by_WI.div(y, part);
  return max(0, min(1 << a.lu, q * a.c.I + min(part, a.c.I) - (sub << a.lu)));
}

// Visible slots of unit `unit` of request r.  `check`: some block of this CTA's work was bad, leave out the tokens
// of such blocks.
__device__ __forceinline__ int visible_in(const KeyUnits& a, int r, bool check, int unit, int lim) {
  int rem, w;
  const int vb = a.by_vbu.div(unit, rem), sub = a.c.by_W.div(rem, w);
  const int v = unit_visible(a, vb, sub, w, lim);
  if (!check || v == 0) return v;
  const int32_t b = vb < a.c.max_vb ? a.c.table[static_cast<int64_t>(r) * a.c.max_vb + vb] : -1;
  return b < 0 || b >= a.c.num_blocks ? 0 : v;
}

// Visible columns (a prefix, 0..16) of each 16 columns of a tile, 8 bits each, for a row that sees positions below
// lim.  By a whole warp: where all lanes have the same lim (the rows of one token) each computes one of the eight.
__device__ __forceinline__ uint64_t tile_limits(const KeyUnits& a, int r, bool check, int tile, int lim) {
  const int units = tile << a.lupt, per = a.lu - 4;   // 16-column groups of a unit: 2^per
  if (__all_sync(0xffffffffu, lim == __shfl_sync(0xffffffffu, lim, 0))) {
    const int i = threadIdx.x & 7;
    const int v = visible_in(a, r, check, units + (i >> per), lim) - 16 * (i & ((1 << per) - 1));
    const uint32_t byte = static_cast<uint32_t>(max(0, min(v, 16))) << (8 * (i & 3));
    const uint32_t lo = __reduce_or_sync(0xffffffffu, i < 4 ? byte : 0u), hi = __reduce_or_sync(0xffffffffu, i < 4 ? 0u : byte);
    return static_cast<uint64_t>(hi) << 32 | lo;
  }
  uint64_t lm = 0;
  int v = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    if ((i & ((1 << per) - 1)) == 0) v = visible_in(a, r, check, units + (i >> per), lim);   // the next unit
    lm |= static_cast<uint64_t>(min(v, 16)) << (8 * i);
    v = max(v - 16, 0);
  }
  return lm;
}

// ------------------------------------------------------------------ pipeline pieces
// The tiled load for data that is read once: its L2 lines go first, so that a long context does not push out
// what is used again (tables, queries, partial results and the kernels' own code).
__device__ __forceinline__ uint64_t policy_once() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_3d_once(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                                 int32_t c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// mbar_wait by a whole warp with one outcome for all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, long long limit, int site) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, limit, site));
}

template <int NS>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ void advance() {
    if (++st == NS) {
      st = 0;
      ph ^= 1;
    }
  }
};

// ------------------------------------------------------------------ host side
// Three-dimensional bf16 map with 64-column boxes in the 128-byte swizzle the MMA descriptors expect.
inline ra_status box_map(CUtensorMap* map, const void* base, int D, int64_t n1, int64_t n2, uint32_t box1, uint32_t box2) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return ra::fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(n1) * D * 2};
  cuuint32_t box[3] = {64, box1, box2};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return ra::fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return RA_OK;
}

}  // namespace
