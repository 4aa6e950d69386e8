// The attention weight that every cached token receives from a chunk of
// queries: the column sums of the softmax, from the scores and the rows' LSE.
//
// Mathematics.  w[x, g] += sum_{i, h in g} 2^(s_ihx * scale log2 e - lse_ih log2 e)
// over the queries i that see token x.  The rows' LSE is known, so that nothing
// is rescaled and one pass over K suffices.
//
// The score tile is computed transposed, S^T = K Q^T (128 keys x up to 128 query
// rows): a key is a lane of tensor memory, a thread sums its key's row, and no sum
// crosses threads.  A CTA holds two key tiles ("slots") and lets the
// request's query tiles pass by: each Q tile that TMA brings in serves both.
// Scores are double buffered per slot in tensor memory (2 x 2 x 128 columns),
// so that the exps never wait for the tensor core.
//
// What bounds it: for single tokens (few query rows; the columns are trimmed to the
// rows there are) HBM: K is read once, the pairs of tiles of one head follow one
// another on a CTA while the Q tile stays, and K leaves L2 first.  32 single tokens
// over 2048-16384 (32/8 heads of 128): 99 us, 6.65 TB/s, 98 % of the copy rate.
// For more queries one exp per (query row, key), 32 a cycle and SM: 512 cycles for a
// 128 x 128 tile, as many as its score product.  With two warps to an SM quarter a
// tile takes 1650-1900 instead, two slots side by side, and the MMA thread's turn over
// two tiles of each slot 4600; the last 64 queries of 4 prompts of 8192-16384 take
// 38 us (floor 15).  Four slots with 16 warps of exps: 44 us (registers, latency
// between tiles); an MMA thread for each slot: 38.9.
//
// Work.  The key tile pairs of all requests and heads lie on one axis of cost,
// which is cut into 152 equal parts; a part ends at the border of a pair, whose sum
// is made by one CTA in a fixed order.  So the least that a CTA takes is 256 keys
// against all queries that see them: where many queries meet few keys (a whole
// prompt) the parts are not equal.  4096 queries of a context of 4096, 32/8
// heads of 128: the busiest CTA has three times the mean, 242 us on a floor of 36 (products);
// with 8/1 heads 16 of the 152 CTAs have work, 322 us on 9; 4096 of 32768: 1141 on 540.
//
// Roles (384 threads): warp 0 TMA, warp 1 MMA issue, warp 2 LSE rows, warp 3
// schedule, warps 4-7 and 8-11 exps and sums of slots 0 and 1.
#include <algorithm>

#include "ra_key_units.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_attn_weights)

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kCtas = 152;
constexpr int kWeightThreads = 384;
constexpr int kSegs = 4, kSegReaders = 11;
template <int D>
constexpr int kLseStagesOf = D == 128 ? 2 : 4;   // not below the query tiles that stay

struct WeightArgs : KeyUnits {
  const int32_t *qsl, *ctx;
  const float* lse;
  int64_t T;
  int R, Hq, G, causal;
  int tpt, pair_q;        // tokens of a query tile; query tiles that a pair of key tiles spans under the causal mask
  int q_stages;           // query tiles that fit in shared memory
  FastDiv by_tpt, by_G, by_pair_q;
  float scale_log2;
  const float* w_in;
  float* w_out;
  long long wait_limit;
  long long drain_limit;  // of the last wait for products in flight: not below 2^22 cycles
};

// ------------------------------------------------------------------ work
struct Req {
  int r, q0, n, L, tiles, nq;   // request, first query row, queries, context, key tiles, query tiles
  long long pos0;               // position of query 0
  int k0;                       // pairs before it: the later ones meet fewer and fewer query tiles
  __device__ int pairs() const { return (tiles + 1) >> 1; }
};

__device__ __forceinline__ Req make_req(const WeightArgs& a, int r, const Lens& x) {
  Req q;
  q.r = r;
  query_range(x, a.T, q.q0, q.n, 600);
  q.L = paged_len(a.c, x.ctx, 601);
  q.pos0 = static_cast<long long>(x.ctx) - q.n;
  q.tiles = (units_below(a, q.L) + (1 << a.lupt) - 1) >> a.lupt;
  q.nq = a.by_tpt.div(q.n + a.tpt - 1);
  q.k0 = a.causal ? (q.pos0 <= 0 ? 0 : static_cast<int>(min(q.pos0 >> 8, 1ll << 30))) : 1 << 30;
  return q;
}

__device__ __forceinline__ Req load_req(const WeightArgs& a, int r) { return make_req(a, r, load_lens(a.qsl, a.ctx, r, a.R)); }

// Cost of pairs 0 .. k-1: each 5 for its loads and 4 for each query tile it meets.
__device__ __forceinline__ long long prefix(const WeightArgs& a, const Req& q, int k) {
  const long long full = min(k, q.k0 + 1);               // pairs that meet all query tiles
  const long long m = min(k - static_cast<int>(full), a.pair_q > 0 ? a.by_pair_q.div(q.nq) : 1 << 30);
  return 5ll * k + 4 * (full * q.nq + m * q.nq - a.pair_q * (m * (m + 1) / 2));
}

// Key tiles of one head.  Where the request's query tiles all stay in shared memory (nqt > 0) an item is a run
// of pairs, else it is one pair and the query tiles qf .. qf + nq - 1 pass by.
struct Item {
  int r, g, q0, n, L, pos0;     // as in Req; pos0 cut below at -n
  int tile0, tiles;             // first key tile, key tiles
  int nqt, qf, nq;
  int more;                     // 0: end of the part
};

// First query tile that can see a key of tile `tile` or of a later one.
__device__ __forceinline__ int first_query_tile(const WeightArgs& a, int tile, int pos0) {
  if (!a.causal) return 0;
  int rem, off;
  const int vb = a.by_vbu.div(tile << a.lupt, rem), s0 = a.c.by_W.div(rem) << a.lu;
  const int first = vb * a.c.V + a.c.by_I.div(s0, off) * a.c.W * a.c.I + off;   // no key of them is before it
  return first <= pos0 ? 0 : a.by_tpt.div(first - pos0);
}

__device__ __forceinline__ long long warp_scan(long long v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += y;
  }
  return v;
}

// Walks the pairs whose start lies in part [lo, hi) of the cost axis.
struct ItemIter {
  const WeightArgs& a;
  long long lo, hi, at;
  Req q;
  int g, k, pairs;
  bool live;
  __device__ ItemIter(const WeightArgs& args) : a(args), live(false) {}
  // f(request) for all requests in order, as in the chunk attention's plan.
  template <class F>
  __device__ __forceinline__ bool for_requests(const F& f) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int base = 0; base < a.R; base += 128) {
      Lens x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = load_lens(a.qsl, a.ctx, base + 32 * j + lane, a.R);
#pragma unroll 1
      for (int j = 0; j < 4 && base + 32 * j < a.R; ++j) {
        const Lens y = j == 0 ? x[0] : j == 1 ? x[1] : j == 2 ? x[2] : x[3];
        if (f(make_req(a, base + 32 * j + lane, y))) return true;
      }
    }
    return false;
  }
  // The request with the first cost at or past the part's start, found by the whole warp; the lane that gets true
  // walks.
  __device__ bool find(int part) {
    const int lane = threadIdx.x & 31;
    const bool few = a.R <= 32;            // then each lane keeps its request
    long long total = 0;
    auto add = [&](const Req& x) {
      total += a.c.Hkv * prefix(a, x, x.pairs());
      return false;
    };
    if (few) {
      q = load_req(a, lane);
      add(q);
    } else {
      for_requests(add);
    }
    total = __shfl_sync(0xffffffffu, warp_scan(total), 31);
    const long long share = (total + kCtas - 1) / kCtas;
    lo = min(total, share * part);
    hi = min(total, share * (part + 1));
    if (lo >= hi) return false;
    long long before = 0, pre = 0;
    auto look = [&](const Req& x) {
      const long long c = a.c.Hkv * prefix(a, x, x.pairs()), s = warp_scan(c);
      pre = before + s - c;
      before += __shfl_sync(0xffffffffu, s, 31);
      if (before <= lo) return false;
      live = pre <= lo && lo < pre + c;
      if (live) q = x;
      return true;
    };
    if (few) look(q); else for_requests(look);
    if (!live) return false;
    pairs = q.pairs();
    const long long per_head = prefix(a, q, pairs);
    g = 0;
    while (g + 1 < a.c.Hkv && (g + 1) * per_head <= lo - pre) ++g;
    const long long off = lo - pre - g * per_head;
    int u = 0, v = pairs;               // first pair with prefix >= off (pairs: the next head's first)
    while (u < v) {
      const int mid = (u + v) >> 1;
      if (prefix(a, q, mid) >= off) v = mid; else u = mid + 1;
    }
    k = u;
    at = pre + g * per_head + prefix(a, q, k);
    skip();
    return true;
  }
  // Past the last pair of a head: on to the next head, the next request that has any.
  __device__ void skip() {
    while (live && k >= pairs) {
      k = 0;
      if (++g < a.c.Hkv) continue;
      g = 0;
      do {
        if (++q.r >= a.R) { live = false; return; }
        q = load_req(a, q.r);
        pairs = q.pairs();
      } while (pairs == 0);
    }
  }
  __device__ bool next(Item& s) {
    if (!live || at >= hi) return false;
    s.r = q.r; s.g = g; s.q0 = q.q0; s.n = q.n; s.L = q.L;
    s.pos0 = static_cast<int>(q.pos0 < -q.n ? -q.n : q.pos0);
    s.tile0 = 2 * k;
    s.nqt = q.nq <= a.q_stages ? q.nq : 0;
    s.qf = s.nqt ? 0 : min(q.nq, first_query_tile(a, s.tile0, s.pos0));
    s.nq = q.nq - s.qf;
    const long long here = prefix(a, q, k);
    int u = k + 1, v = s.nqt || q.nq == 0 ? pairs : k + 1;   // past the last pair of the item: its start is below hi
    while (u < v) {
      const int mid = (u + v + 1) >> 1;
      if (at + prefix(a, q, mid - 1) - here < hi) u = mid; else v = mid - 1;
    }
    at += prefix(a, q, u) - here;
    s.tiles = min(2 * u, q.tiles) - 2 * k;
    k = u;
    s.more = 1;
    skip();
    return true;
  }
};

// ------------------------------------------------------------------ the kernel
template <int D>
constexpr int kKStages = D == 128 ? 5 : 9;
template <int D>
constexpr int kQStages = D == 128 ? 2 : 4;

template <int D>
struct __align__(1024) WeightSmem {
  uint8_t k[kKStages<D>][BN * D * 2];
  uint8_t q[kQStages<D>][BM * D * 2];
  uint64_t k_full[kKStages<D>], k_empty[kKStages<D>], q_full[kQStages<D>], q_empty[kQStages<D>];
  static constexpr int kLseStages = kLseStagesOf<D>;
  uint64_t l_full[kLseStages], l_empty[kLseStages], seg_full[kSegs], seg_empty[kSegs];
  uint64_t s_full[2][2], s_empty[2][2], drain;
  __align__(16) float neg_lse[kLseStages][BM];   // -lse * log2 e; -inf: the row adds nothing (also where there is none)
  int all_count[kLseStages];                     // all 128 rows add
  Item item[kSegs];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(WeightSmem<128>) + 1024 <= 232448 && sizeof(WeightSmem<64>) + 1024 <= 232448, "227 KB of shared memory");

struct ItemReader {
  uint32_t at = 0;
  bool ok = true;   // false: a wait expired, the part has not ended
  template <class Smem>
  __device__ bool next(Smem& sm, Item& s, volatile int* abort_flag, long long limit, bool whole_warp) {
    const int i = at & (kSegs - 1);
    const uint32_t bar = smem_u32(&sm.seg_full[i]), ph = (at / kSegs) & 1;
    ok = whole_warp ? warp_wait(bar, ph, abort_flag, limit, 670) : mbar_wait(bar, ph, abort_flag, limit, 671);
    if (!ok) return false;
    s = sm.item[i];
    if (whole_warp) __syncwarp();
    if (!whole_warp || (threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sm.seg_empty[i]));
    ++at;
    return s.more != 0;
  }
};

// Valid columns of a query tile.
__device__ __forceinline__ int columns(const WeightArgs& a, const Item& s, int t) {
  return min(s.n - t * a.tpt, a.tpt) * a.G;
}

// Sum of 2^(x * scale - lse) over N columns; MASK: over those from lo on that count (neg_lse above -inf) alone.
// Columns are left out after their exponent is formed, so that what a row that does not count, or does not see the
// token, holds (NaN in its score or its LSE) stays outside.
template <bool MASK, int N>
__device__ __forceinline__ float chunk_sum(const uint32_t (&x)[N], uint64_t sc2, const float* neg_lse, int lo) {
  uint64_t acc[4];
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const ulonglong2 nl = *reinterpret_cast<const ulonglong2*>(neg_lse + i);
    float e[4], l[4];
    f2unpack(ffma2(f2pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), sc2, nl.x), e[0], e[1]);
    f2unpack(ffma2(f2pack(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), sc2, nl.y), e[2], e[3]);
    if (MASK) {
      f2unpack(nl.x, l[0], l[1]);
      f2unpack(nl.y, l[2], l[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < lo || l[j] == -CUDART_INF_F) e[j] = -CUDART_INF_F;
    }
    const uint64_t u = f2pack(ex2(e[0]), ex2(e[1])), v = f2pack(ex2(e[2]), ex2(e[3]));
    const int k = (i >> 2) & 1;
    acc[k] = i < 8 ? u : fadd2(acc[k], u);
    acc[2 + k] = i < 8 ? v : fadd2(acc[2 + k], v);
  }
  float p0, p1;
  f2unpack(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), p0, p1);
  return p0 + p1;
}

template <int D>
__global__ void __launch_bounds__(kWeightThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ1,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ WeightArgs a) {
  constexpr int SLABS = D / 64, NK = kKStages<D>, NQ = kQStages<D>, kLseStages = kLseStagesOf<D>;
  static_assert(kLseStages >= NQ);
  constexpr uint32_t kTileBytes = BM * D * 2;
  extern __shared__ uint8_t smem_raw[];
  WeightSmem<D>& sm = *reinterpret_cast<WeightSmem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const long long lim = a.wait_limit;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NK; ++s) {
      mbar_init(smem_u32(&sm.k_full[s]), 1);
      mbar_init(smem_u32(&sm.k_empty[s]), 1);
    }
    for (int s = 0; s < NQ; ++s) {
      mbar_init(smem_u32(&sm.q_full[s]), 1);
      mbar_init(smem_u32(&sm.q_empty[s]), 1);
    }
    for (int s = 0; s < kLseStages; ++s) {
      mbar_init(smem_u32(&sm.l_full[s]), 1);
      mbar_init(smem_u32(&sm.l_empty[s]), 8);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(smem_u32(&sm.seg_full[s]), 1);
      mbar_init(smem_u32(&sm.seg_empty[s]), kSegReaders);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&sm.s_full[i >> 1][i & 1]), 1);
      mbar_init(smem_u32(&sm.s_empty[i >> 1][i & 1]), 128);
    }
    mbar_init(smem_u32(&sm.drain), 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  ItemIter it(a);
  bool mine = false;
  if (warp == 3) mine = it.find(blockIdx.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  ItemReader items;
  Item s = {};

  if (warp == 0) {
    // ============================================================ TMA producer (whole warp: a unit or a token per lane)
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmQ1);
      tma_prefetch_desc(&tmK);
    }
    Ring<NK> kr;
    Ring<NQ> qr;
    uint32_t k_issued = 0, q_issued = 0;
    bool ok = true;
    const uint64_t once = policy_once();      // a key tile is read by one CTA, once
    const int oob = static_cast<int>(a.c.W * a.c.num_blocks * a.c.Hkv);   // past the last block: zero fill
    // the lane's unit of a key tile; its block is looked up a tile ahead
    struct Unit {
      int s0, w, blk;
    };
    auto locate = [&](int tile) {
      Unit x;
      int rem;
      const int vb = a.by_vbu.div((tile << a.lupt) + lane, rem);
      x.s0 = a.c.by_W.div(rem, x.w) << a.lu;
      x.blk = -1;
      if (tile < s.tile0 + s.tiles && lane >> a.lupt == 0 && static_cast<int64_t>(vb) * a.c.V < s.L)
        x.blk = a.c.table[static_cast<int64_t>(s.r) * a.c.max_vb + vb];
      return x;
    };
    auto load_k = [&](const Unit& x) -> bool {
      if (!warp_wait(smem_u32(&sm.k_empty[kr.st]), kr.ph ^ 1, abort_flag, lim, 620)) return false;
      const uint32_t bar = smem_u32(&sm.k_full[kr.st]);
      if (lane == 0) mbar_arrive_expect_tx(bar, kTileBytes);
      __syncwarp();
      if (lane >> a.lupt == 0) {
        const int hb = x.blk < 0 || x.blk >= a.c.num_blocks ? oob : static_cast<int>((x.w * a.c.num_blocks + x.blk) * a.c.Hkv + s.g);
        for (int sl = 0; sl < SLABS; ++sl)
          tma_load_3d_once(smem_u32(sm.k[kr.st] + sl * BN * 128 + (lane << a.lu) * 128), &tmK, bar, 64 * sl, x.s0, hb, once);
      }
      ++k_issued;
      kr.advance();
      return true;
    };
    auto load_q = [&](int t) -> bool {
      if (!warp_wait(smem_u32(&sm.q_empty[qr.st]), qr.ph ^ 1, abort_flag, lim, 621)) return false;
      const uint32_t bar = smem_u32(&sm.q_full[qr.st]);
      const int tokens = min(s.n - t * a.tpt, a.tpt), row = s.q0 + t * a.tpt;
      if (lane == 0) mbar_arrive_expect_tx(bar, SLABS * tokens * a.G * 128);
      __syncwarp();
      if (tokens == a.tpt) {
        if (lane < SLABS)
          tma_load_3d(smem_u32(sm.q[qr.st] + lane * BM * 128), &tmQ, bar, 64 * lane, s.g * a.G, row);
      } else {   // a token's heads at a time: no rows of other requests
        for (int i = lane; i < tokens; i += 32)
          for (int sl = 0; sl < SLABS; ++sl)
            tma_load_3d(smem_u32(sm.q[qr.st] + sl * BM * 128 + i * a.G * 128), &tmQ1, bar, 64 * sl, s.g * a.G, row + i);
      }
      ++q_issued;
      qr.advance();
      return true;
    };
    while (ok && items.next(sm, s, abort_flag, lim, true)) {
      if (s.nq <= 0) continue;
      Unit x = locate(s.tile0), y = locate(s.tile0 + 1);
      ok = load_k(x);
      for (int t = 0; t < s.nqt && ok; ++t) ok = load_q(t);
      for (int i = 1; i < s.tiles && ok; ++i) {
        x = y;
        y = locate(s.tile0 + i + 1);
        ok = load_k(x);
      }
      if (s.nqt == 0)
        for (int t = s.qf; t < s.qf + s.nq && ok; ++t) ok = load_q(t);
    }
    if (lane == 0) {
      // The last load of each buffer lands before the CTA exits, also where another role has given up, or gives up
      // from here on (else each has been waited for by its reader).
      for (int i = 0; i < NK; ++i) {
        const uint32_t n = k_issued / NK + (static_cast<uint32_t>(i) < k_issued % NK ? 1 : 0);
        if (n) mbar_wait_quiesce(smem_u32(&sm.k_full[i]), (n - 1) & 1, 1 << 22);
      }
      for (int i = 0; i < NQ; ++i) {
        const uint32_t n = q_issued / NQ + (static_cast<uint32_t>(i) < q_issued % NQ ? 1 : 0);
        if (n) mbar_wait_quiesce(smem_u32(&sm.q_full[i]), (n - 1) & 1, 1 << 22);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    if (lane == 0) {
      Ring<NK> kr;
      Ring<NQ> qr;
      uint32_t cnt0 = 0, cnt1 = 0;   // score tiles of each slot so far
      bool ok = true;
      const uint64_t dk = desc_sw128(smem_u32(sm.k[0]), 16, 1024), dq = desc_sw128(smem_u32(sm.q[0]), 16, 1024);
      // A wait that passes at once still takes its 130 cycles or so, with the tensor core idle: the barriers of the
      // next product (its score buffer, its key tile) are looked at while the last products of this one are
      // queued.
      bool s_ready = false, k_ready = false;
      // S_h of the key tile at stage ks and the query tile t at stage qs; slot h_next is next, and its key tile at
      // stage k_next (-1: this one, or none)
      auto issue = [&](int h, int ks, int qs, int t, int h_next, int k_next, uint32_t k_next_ph) -> bool {
        const uint32_t c = h ? cnt1 : cnt0, b = 2 * h + (c & 1);
        if (!s_ready && !mbar_wait(smem_u32(&sm.s_empty[0][0] + b), ((c >> 1) & 1) ^ 1, abort_flag, lim, 632)) return false;
        if (h) ++cnt1; else ++cnt0;
        tc_fence_after();
        const uint32_t idesc = idesc_bf16_f32(BM, (columns(a, s, t) + 15) & ~15, 0, 0);
        const uint64_t d0 = dk + ks * (kTileBytes >> 4), d1 = dq + qs * (kTileBytes >> 4);
        const uint32_t cn = h_next ? cnt1 : cnt0;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off16 = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
          mma_bf16_ss(tmem + b * BN, d0 + off16, d1 + off16, idesc, kk > 0 ? 1u : 0u);
          if (kk == D / 16 - 3) {
            s_ready = mbar_test_wait(smem_u32(&sm.s_empty[0][0] + 2 * h_next + (cn & 1)), ((cn >> 1) & 1) ^ 1);
            k_ready = k_next >= 0 && mbar_test_wait(smem_u32(&sm.k_full[k_next]), k_next_ph);
          }
        }
        mma_commit(smem_u32(&sm.s_full[0][0] + b));
        return true;
      };
      while (ok && items.next(sm, s, abort_flag, lim, false)) {
        if (s.nq <= 0) continue;
        if (s.nqt) {
          const int q0 = qr.st;
          // The slots take turns, so that neither waits behind the other's score buffers.
#pragma unroll 1
          for (int i = 0; i < s.tiles && ok; i += 2) {
            const int qf = s.nqt > 1 ? first_query_tile(a, s.tile0 + i, s.pos0) : 0;
            const bool two = i + 1 < s.tiles, more = i + 2 < s.tiles;
            int ks[2];
            uint32_t kph[2];
            ks[0] = kr.st; kph[0] = kr.ph;
            kr.advance();
            ks[1] = kr.st; kph[1] = kr.ph;
            if (two) kr.advance();
            if (!k_ready && !(ok = mbar_wait(smem_u32(&sm.k_full[ks[0]]), kph[0], abort_flag, lim, 630))) break;
            if (i == 0)
              for (int t = 0; t < s.nqt && ok; ++t) {
                ok = mbar_wait(smem_u32(&sm.q_full[qr.st]), qr.ph, abort_flag, lim, 631);
                qr.advance();
              }
#pragma unroll 1
            for (int t = qf; t < s.nqt && ok; ++t) {
              const bool last = t + 1 == s.nqt;
              const int qs = q0 + t < NQ ? q0 + t : q0 + t - NQ;
              const int k_after = last && more ? kr.st : -1;
              if (!(ok = issue(0, ks[0], qs, t, two ? 1 : 0, two ? (t == qf ? ks[1] : -1) : k_after, two ? kph[1] : kr.ph))) break;
              if (last) mma_commit(smem_u32(&sm.k_empty[ks[0]]));
              if (!two) continue;
              if (t == qf && !k_ready && !(ok = mbar_wait(smem_u32(&sm.k_full[ks[1]]), kph[1], abort_flag, lim, 635))) break;
              if (!(ok = issue(1, ks[1], qs, t, 0, k_after, kr.ph))) break;
              if (last) mma_commit(smem_u32(&sm.k_empty[ks[1]]));
            }
          }
          s_ready = k_ready = false;   // the next item starts anew
          for (int t = 0; t < s.nqt && ok; ++t) mma_commit(smem_u32(&sm.q_empty[q0 + t < NQ ? q0 + t : q0 + t - NQ]));
        } else {
          int ks[2] = {0, 0};
          for (int h = 0; h < s.tiles && ok; ++h) {
            ok = mbar_wait(smem_u32(&sm.k_full[kr.st]), kr.ph, abort_flag, lim, 633);
            if (h) ks[1] = kr.st; else ks[0] = kr.st;
            kr.advance();
          }
#pragma unroll 1
          for (int t = s.qf; t < s.qf + s.nq && ok; ++t) {
            if (!(ok = mbar_wait(smem_u32(&sm.q_full[qr.st]), qr.ph, abort_flag, lim, 634))) break;
            ok = issue(0, ks[0], qr.st, t, s.tiles < 2 ? 0 : 1, -1, 0) && (s.tiles < 2 || issue(1, ks[1], qr.st, t, 0, -1, 0));
            if (!ok) break;
            mma_commit(smem_u32(&sm.q_empty[qr.st]));
            qr.advance();
          }
          s_ready = k_ready = false;
          if (ok) mma_commit(smem_u32(&sm.k_empty[ks[0]]));
          if (ok && s.tiles > 1) mma_commit(smem_u32(&sm.k_empty[ks[1]]));
        }
      }
      mma_commit(smem_u32(&sm.drain));
      if (!mbar_wait_quiesce(smem_u32(&sm.drain), 0, a.drain_limit) && ok && items.ok) {
        *abort_flag = 1;
        ra_record_error(RA_ERR_TIMEOUT, 639);
      }
    }
  } else if (warp == 2) {
    // ============================================================ LSE of the query rows
    uint32_t n = 0;
    bool ok = true;
    while (ok && items.next(sm, s, abort_flag, lim, true)) {
      for (int t = s.qf; t < s.qf + s.nq && ok; ++t, ++n) {
        const int cols = columns(a, s, t);
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 32 * j + lane;
          int head;
          const int tok = a.by_G.div(i, head);
          const float x = i < cols ? a.lse[static_cast<int64_t>(s.q0 + t * a.tpt + tok) * a.Hq + s.g * a.G + head] : -CUDART_INF_F;
          v[j] = x == -CUDART_INF_F ? x : -x * kLog2e;
        }
        const bool all_count = __all_sync(0xffffffffu, v[0] != -CUDART_INF_F && v[1] != -CUDART_INF_F &&
                                                           v[2] != -CUDART_INF_F && v[3] != -CUDART_INF_F);
        const int b = n % kLseStages;
        if (!(ok = warp_wait(smem_u32(&sm.l_empty[b]), ((n / kLseStages) & 1) ^ 1, abort_flag, lim, 640))) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) sm.neg_lse[b][32 * j + lane] = v[j];
        if (lane == 0) sm.all_count[b] = all_count;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.l_full[b]));
      }
    }
  } else if (warp == 3) {
    // ============================================================ items of this part, announced to the other roles
    const unsigned owner = __ballot_sync(0xffffffffu, mine);
    if (mine || (owner == 0 && lane == 0)) {
      bool more = true;
      for (uint32_t i = 0; more; ++i) {
        more = mine && it.next(s);
        if (!more) s.more = 0;
        const int b = i & (kSegs - 1);
        if (!mbar_wait(smem_u32(&sm.seg_empty[b]), ((i / kSegs) & 1) ^ 1, abort_flag, lim, 672)) break;
        sm.item[b] = s;
        mbar_arrive(smem_u32(&sm.seg_full[b]));
      }
    }
    __syncwarp();
  } else {
    // ============================================================ exps and sums (slot h): a key per thread
    const int h = (warp - 4) >> 2;
    const int quarter = warp & 3, key = quarter * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint64_t sc2 = f2pack(a.scale_log2, a.scale_log2);
    uint32_t n = 0, cnt = 0;   // LSE tiles, score tiles so far
    bool ok = true;
    // adds the score tile of query tile t; `first`: first query that sees this thread's token
    float sum = 0.f;
    auto add_tile = [&](int t, int first) -> bool {
      const uint32_t b = cnt & 1;
      if (!warp_wait(smem_u32(&sm.s_full[h][b]), (cnt >> 1) & 1, abort_flag, lim, 651)) return false;
      ++cnt;
      tc_fence_after();
      const int hi = columns(a, s, t), lo = min(BN, max(0, first - t * a.tpt) * a.G);
      const int lb = (s.nqt ? n + t : n) % kLseStages;
      const float* nlse = sm.neg_lse[lb];
      const uint32_t addr = t_lane + (2 * h + b) * BN;
      if (sm.all_count[lb] && !__any_sync(0xffffffffu, lo > 0)) {
        // all columns count: two chunks a turn, the next one's load in flight (a rolled loop, that its code
        // stays in the instruction cache)
        uint32_t xa[32], xb[32];
        tmem_ld32(addr, xa);
        tmem_wait_ld();
#pragma unroll 1
        for (int c = 0; c < BN; c += 64) {
          tmem_ld32(addr + c + 32, xb);
          sum += chunk_sum<false>(xa, sc2, nlse + c, 0);
          tmem_wait_ld();
          if (c == 0) tmem_ld32(addr + 64, xa);
          sum += chunk_sum<false>(xb, sc2, nlse + c + 32, 0);
          if (c == 0) tmem_wait_ld();
        }
      } else if (hi <= 16) {   // a token or a few: half a chunk
        uint32_t x[16];
        tmem_ld16(addr, x);
        tmem_wait_ld();
        sum += chunk_sum<true>(x, sc2, nlse, lo);
      } else {
#pragma unroll 1
        for (int c = 0; c < hi; c += 32) {
          uint32_t x[32];
          tmem_ld32(addr + c, x);
          tmem_wait_ld();
          sum += chunk_sum<true>(x, sc2, nlse + c, lo - c);
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&sm.s_empty[h][b]));
      return true;
    };
    // This thread's token of a key tile: position, row of the weights but for the block, and the block's id, looked
    // up a pair ahead.
    struct Token {
      int x, slot, w, blk;
    };
    auto locate = [&](int tile) {
      Token k;
      int rem, off;
      const int vb = a.by_vbu.div((tile << a.lupt) + (key >> a.lu), rem);
      k.slot = (a.c.by_W.div(rem, k.w) << a.lu) + (key & ((1 << a.lu) - 1));
      k.x = vb * a.c.V + (a.c.by_I.div(k.slot, off) * a.c.W + k.w) * a.c.I + off;
      k.blk = tile < s.tile0 + s.tiles && k.x < s.L ? a.c.table[static_cast<int64_t>(s.r) * a.c.max_vb + vb] : INT32_MIN;
      return k;
    };
    while (ok && items.next(sm, s, abort_flag, lim, true)) {
      Token ahead = locate(s.tile0 + h);
      const uint32_t n_lse = s.nqt;   // tiles of LSE that stay for the item
      for (uint32_t t = 0; t < n_lse && ok; ++t)
        ok = warp_wait(smem_u32(&sm.l_full[(n + t) % kLseStages]), ((n + t) / kLseStages) & 1, abort_flag, lim, 650);
#pragma unroll 1
      for (int i = h; i < max(s.tiles, 2) && ok; i += 2) {
        const bool active = i < s.tiles;   // false: slot 1 of an item of one tile, or past the last
        const Token tk = ahead;
        ahead = locate(s.tile0 + i + 2);
        int64_t at = -1;
        float old = 0.f;
        if (tk.blk != INT32_MIN) {
          if (tk.blk >= 0 && tk.blk < a.c.num_blocks) {
            at = ((tk.w * a.c.num_blocks + tk.blk) * a.c.Hkv + s.g) * a.c.bs + tk.slot;
            if (a.w_in && (!a.causal || tk.x < s.pos0)) old = a.w_in[at];
          } else {
            ra_record_error(RA_ERR_DEVICE_BOUNDS, 602);
          }
        }
        const int first = a.causal ? max(0, tk.x - s.pos0) : 0;
        sum = 0.f;
        if (s.nqt) {
          if (active) {
            const int qf = s.nqt > 1 ? first_query_tile(a, s.tile0 + (i & ~1), s.pos0) : 0;
#pragma unroll 1
            for (int t = qf; t < s.nqt && ok; ++t) ok = add_tile(t, first);
          }
        } else {
#pragma unroll 1
          for (int t = s.qf; t < s.qf + s.nq && ok; ++t, ++n) {
            const int lb = n % kLseStages;
            if (!(ok = warp_wait(smem_u32(&sm.l_full[lb]), (n / kLseStages) & 1, abort_flag, lim, 652))) break;
            if (active) ok = add_tile(t, first);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.l_empty[lb]));
          }
        }
        if (ok && at >= 0) a.w_out[at] = old + sum;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0)
        for (uint32_t t = 0; t < n_lse; ++t) mbar_arrive(smem_u32(&sm.l_empty[(n + t) % kLseStages]));
      n += n_lse;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <int D>
ra_status launch_weights(const void* q, const void* k, const WeightArgs& a, cudaStream_t stream) {
  CUtensorMap mq, mq1, mk;
  ra_status st;
  const int64_t T = std::max<int64_t>(a.T, 1);   // without queries Q is not read: any address serves the map
  const void* qb = a.T > 0 ? q : k;
  if ((st = box_map(&mq, qb, D, a.Hq, T, a.G, a.tpt)) != RA_OK) return st;
  if ((st = box_map(&mq1, qb, D, a.Hq, T, a.G, 1)) != RA_OK) return st;
  if ((st = box_map(&mk, k, D, a.c.bs, a.c.W * a.c.num_blocks * a.c.Hkv, 1 << a.lu, 1)) != RA_OK) return st;
  const size_t smem = sizeof(WeightSmem<D>) + 1024;
  RA_CUDA_TRY(cudaFuncSetAttribute(weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
  weights_kernel<D><<<kCtas, kWeightThreads, smem, stream>>>(mq, mq1, mk, a);
  RA_LAUNCH_CHECK("weights_kernel");
  return RA_OK;
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
  WeightArgs a;
  static_cast<KeyUnits&>(a) =
      make_units(make_paged(block_table, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks));
  a.qsl = query_start_loc; a.ctx = ctx_lens; a.lse = lse;
  a.T = T; a.R = R; a.Hq = Hq; a.G = Hq / Hkv; a.causal = causal ? 1 : 0;
  a.tpt = BM / a.G;
  a.pair_q = a.causal ? 2 * BN / a.tpt : 0;
  a.q_stages = d == 128 ? kQStages<128> : kQStages<64>;
  a.by_tpt = fast_div(a.tpt);
  a.by_G = fast_div(a.G);
  a.by_pair_q = fast_div(std::max(a.pair_q, 1));
  a.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(d))) * kLog2e;
  a.w_in = w_in; a.w_out = w_out;
  a.wait_limit = ra::wait_limit();
  a.drain_limit = std::max<long long>(a.wait_limit, 1ll << 22);
  return d == 128 ? launch_weights<128>(q, k_cache, a, stream) : launch_weights<64>(q, k_cache, a, stream);
}
