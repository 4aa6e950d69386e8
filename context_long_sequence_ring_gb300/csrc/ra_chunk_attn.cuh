// Attention of a chunk of new tokens per request over the sharded paged cache.
//
// Mathematics.  O_i = sum_x e^{s_ix} v_x / sum_x e^{s_ix} over the visible
// tokens x, in one pass with a running maximum m and sum l per row; a context
// that several CTAs share is joined from their (m, l, O) with weights 2^{m - M}.
//
// Rows.  The G query heads of a K/V head read the same keys, so a tile of 128
// rows holds floor(128/G) tokens with all their G heads (one TMA box of Q).
// Two score tiles ("slots") are in flight per CTA so that one slot's softmax
// runs while the tensor core serves the other:
//   pair   the request has more rows than one tile: the slots are two row
//          tiles, and every K/V tile feeds both (tensor-bound, 2 x 128 rows
//          per K/V byte);
//   split  one row tile (single tokens, drafts): the slots take alternate K/V
//          tiles, each with its own running (m, l, O), joined at the end from
//          tensor memory (HBM-bound: a K/V tile of 64 KB takes the SM's share of
//          HBM bandwidth about 1.45 us, one slot's chain of score product, softmax
//          and P.V about 1.3 us, two of them half of that).  Its tiles are read by
//          one CTA once and leave L2 first (drafts 286 -> 279 us, a token at 131072
//          92 -> 87 us; where requests share prefix blocks it makes no difference: 48
//          on one prefix of 16384, 384 us with it and 385 without).  At D = 64
//          the fixed work of a tile would take longer than HBM: see kScores and
//          kJoint.
//
// Keys.  The cache is read where it lies, in units of 16 or 32 slots
// (ra_key_units.cuh).  V rows of slots past the context
// (which may hold NaN) are zeroed in shared memory by a warp of their own in
// the tiles that have any; units of a bad block are read out of bounds, which
// TMA fills with zeros.
//
// Work.  The keys that all row tiles of all heads and requests meet are laid
// out on one axis of cost, cut into equal parts, one per CTA (152;
// ra_chunk_plan.cuh): long and short contexts, prompts and single tokens
// balance without any plan from the host.  A part starts or ends inside at most
// two row tiles; their partial (m, l, O) go to the workspace (at most two per
// CTA) and a second small kernel joins them.
//
// Measured (32/8 heads of 128, 8 devices; calls, joining included): 48 requests with 1-6 drafted
// tokens over 2048-16384: 279-284 us, 6.5 TB/s, 96 % of the copy rate; one token over
// 131072: 88-89 us, 6.1 TB/s; 4 single tokens over 200-2000: 22.4 us; 4096 tokens of a
// prompt of 32768: 1.39-1.42 ms, 1.28-1.30 in short runs (1580 TFLOP/s).  12 requests (24/8 heads of
// 64, blocks of 16), prompts of 300-511 new tokens among single ones: 45 us.
// With a window of 4096: 4096 tokens of a prompt 284-297 us (this kernel 272, joining 22), 64 single tokens 195 us, 5.8 TB/s,
// 32768 packed tokens 1.53-1.62 ms (this kernel alone 1.39; a sequence of 16384 under no window 1.34 ms, 1640 TFLOP/s).
// What a window costs is an item's start and end, 11-13 thousand cycles on packed sequences, and masked tiles at either end:
// over the cache 64 us of the prompt's piece, whose items have 5.2 of them among 34.8.
//
// Roles (384 threads): warp 0 TMA, warp 1 MMA issue, warp 2 zeroing of dead V
// rows, warp 3 schedule, warps 4-7 and 8-11 softmax of slots 0 and 1.  Warp 1 issues as a whole, with an elected thread as
// the instructions' predicate: in a branch of one thread their operands are moved to uniform registers one by one
// (about 70 cycles each; the prompt over 32768 1476 us instead of 1295).
// Tensor memory: two (D = 128) or three (D = 64) score tiles S_b = columns [128b, +128) with P (bf16)
// over the first 64 of each, then O_0 and O_1, D columns each.
//
// Forms.  The kernel is written once for the causal mask over the cache, for a
// sliding window with first tokens that stay visible over the cache, and for the
// latter on packed sequences, whose keys are rows of one tensor (units of 32
// rows).  With a window the units of an item are those that hold first tokens, if they end
// before the window starts, and from there on those from the first that any of its rows sees;
// its tiles are cut out of that row of units, so that few first tokens take up a unit, not a tile.
#pragma once

#include <algorithm>
#include <type_traits>

#include "ra_chunk_plan.cuh"
#include "ra_key_units.cuh"

namespace {

struct CausalPaged {
  static constexpr bool kWindow = false, kPacked = false;
};
struct WindowPaged {
  static constexpr bool kWindow = true, kPacked = false;
};
struct WindowPacked {
  static constexpr bool kWindow = true, kPacked = true;
};

constexpr int kChunkThreads = 384;
constexpr int kMergeThreads = 256;
constexpr int kMergeRowBlocks = 8;
constexpr int kFewRows = 32;       // rows of a tile that get a block each

struct ChunkArgs : KeyUnits {
  const int32_t *qsl, *ctx;
  int64_t T;
  int R, Hq, G, causal, out_bf16;
  int tpt;                        // tokens of a row tile
  Rates rates;
  FastDiv by_G, by_tpi;                // by the tokens of a pair of row tiles
  float scale_log2;
  void* o;                        // [T, Hq, D]
  float* lse;                     // [T, Hq] or NULL
  float* o_part;                  // [2 * kCtas][256][D]
  float2* ml_part;                // [2 * kCtas][256]
  void* join;                     // [kCtas] Join of the form
  long long wait_limit;
  long long drain_limit;          // of the last wait for products in flight: not below 2^22 cycles
  int window, n_sink;             // at most 2^30
};

// ------------------------------------------------------------------ work
// A request as the work division sees it.
template <class F>
struct Req : std::conditional_t<F::kWindow, WindowItems, Items> {
  int r, q0, n, L;                // request, first query row, queries, context
  long long pos0;                 // position of query 0
};

template <class F>
__device__ __forceinline__ Lens load_req_lens(const ChunkArgs& a, int r) {
  if (!F::kPacked) return load_lens(a.qsl, a.ctx, r, a.R);
  if (r >= a.R) return Lens{0, 0, 0};
  return Lens{a.qsl[r], a.qsl[r + 1], 0};
}

template <class F>
__device__ __forceinline__ Req<F> make_req(const ChunkArgs& a, int r, const Lens& x) {
  Req<F> q;
  q.r = r;
  query_range(x, a.T, q.q0, q.n, 510);
  if (F::kPacked) {
    q.L = q.n;
    q.pos0 = 0;
  } else {
    q.L = paged_len(a.c, x.ctx, 511);
    q.pos0 = static_cast<long long>(x.ctx) - q.n;
  }
  const int items = q.n > a.tpt ? a.by_tpi.div(q.n + 2 * a.tpt - 1) : (q.n > 0);
  if constexpr (F::kWindow) q.set(a.rates, q.n, items, a.tpt, q.pos0, q.L, a.window, a.n_sink);
  else q.set(a.rates, q.n, items, a.tpt, q.pos0, q.L, a.causal);
  return q;
}

template <class F>
__device__ __forceinline__ Req<F> load_req(const ChunkArgs& a, int r) { return make_req<F>(a, r, load_req_lens<F>(a, r)); }

// Visible tokens of query i: positions below the returned value.
template <class F>
__device__ __forceinline__ int limit_of(const ChunkArgs& a, const Req<F>& q, int i) {
  if (!F::kWindow && !a.causal) return q.L;
  const long long lim = q.pos0 + i + 1;
  return lim < 0 ? 0 : (lim < q.L ? static_cast<int>(lim) : q.L);
}

// First position of query i's window, at most L.
template <class F>
__device__ __forceinline__ int low_of(const ChunkArgs& a, const Req<F>& q, int i) {
  const long long lo = q.pos0 + i + 1 - a.window;
  return lo < 0 ? 0 : (lo < q.L ? static_cast<int>(lo) : q.L);
}

__device__ __forceinline__ int tiles_over(const ChunkArgs& a, int units) { return (units + (1 << a.lupt) - 1) >> a.lupt; }

// The units of an item: unit j is j of the context where j < first, and `skip` units (packed: tokens) further from there on.
struct Run {
  int first, skip;
};
// Units of the run that hold a token below lim, and units all of whose tokens are below lim (both as prefixes; first
// tokens' units left aside, which are before the window).
template <class F>
__device__ __forceinline__ int run_to(const ChunkArgs& a, const Run& u, int lim) {
  if (F::kPacked) return (max(lim - u.skip, 0) + 31) >> 5;
  return units_below(a, lim) - u.skip;
}
template <class F>
__device__ __forceinline__ int run_inside(const ChunkArgs& a, const Run& u, int lim) {
  if (F::kPacked) return max(lim - u.skip, 0) >> 5;
  return units_within(a, lim) - u.skip;
}
template <class F>
__device__ __forceinline__ Run run_of(const ChunkArgs& a, const Req<F>& q, int k, int lim) {
  Run u{0, 0};
  if (F::kWindow) {
    const int low = low_of<F>(a, q, k * (q.pair ? 2 * a.tpt : a.tpt)), sinks = min(a.n_sink, lim);
    if (F::kPacked) {
      const int first = (sinks + 31) >> 5;
      if (low >= 32 * first) u = Run{first, low - 32 * first};
    } else {
      const int first = units_below(a, sinks), start = units_within(a, min(low, lim));
      if (start >= first) u = Run{first, start - first};
    }
  }
  return u;
}

// f(request) for all requests in order, each lane those at lane, lane + 32, ...; four loads in flight where there
// are many (f may stop the walk: it returns true in all lanes or in none).
template <class F, class Fn>
__device__ __forceinline__ bool for_requests(const ChunkArgs& a, const Fn& f) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int base = 0; base < a.R; base += 128) {
    Lens x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = load_req_lens<F>(a, base + 32 * j + lane);
#pragma unroll 1
    for (int j = 0; j < 4 && base + 32 * j < a.R; ++j) {
      const Lens y = j == 0 ? x[0] : j == 1 ? x[1] : j == 2 ? x[2] : x[3];
      if (f(make_req<F>(a, base + 32 * j + lane, y))) return true;
    }
  }
  return false;
}

// The plan and, in the lane that returns true, the request that holds the start of part `part` with the
// cost before it (none: the part is empty).  One warp, a request per lane.
template <class F>
__device__ __forceinline__ bool make_plan(const ChunkArgs& a, int part, Plan& plan, Req<F>& q, uint32_t& pre) {
  const int lane = threadIdx.x & 31;
  const bool few = a.R <= 32;            // then each lane keeps its request
  uint64_t sum = 0;
  uint32_t items = 0;
  auto add = [&](const Req<F>& x) {
    sum += a.c.Hkv * x.upto(x.items);
    items += a.c.Hkv * x.items;
    return false;
  };
  if (few) {
    q = load_req<F>(a, lane);
    add(q);
  } else {
    for_requests<F>(a, add);
  }
  constexpr uint32_t kPart = (1u << 26) - 1;   // 64 bits over the warp in three sums that fit in 32
  const uint32_t s0 = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(sum) & kPart);
  const uint32_t s1 = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(sum >> 26) & kPart);
  const uint32_t s2 = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(sum >> 52));
  items = __reduce_add_sync(0xffffffffu, items);
  sum = (static_cast<uint64_t>(s2) << 52) + (static_cast<uint64_t>(s1) << 26) + s0;
  plan.scale(sum);
  uint32_t total = 0;
  auto add_scaled = [&](const Req<F>& x) {
    total += a.c.Hkv * plan.prefix(x, x.items);
    return false;
  };
  auto sum_scaled = [&] {
    total = 0;
    if (few) add_scaled(q); else for_requests<F>(a, add_scaled);
    total = __reduce_add_sync(0xffffffffu, total);
  };
  if (plan.shift == 0) total = static_cast<uint32_t>(sum) + items;   // the same sum
  else sum_scaled();
  plan.divide(total, a.rates);
  if (plan.try_pieces(items, a.rates)) {
    sum_scaled();
    plan.use_pieces(total);
  }
  const uint32_t lo = plan.lo(part);
  if (lo >= plan.total) return false;
  uint32_t at = 0;
  bool mine = false;
  auto find = [&](const Req<F>& x) {
    const uint32_t cost = a.c.Hkv * plan.prefix(x, x.items);
    uint32_t s = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    pre = at + s - cost;
    at += __shfl_sync(0xffffffffu, s, 31);
    if (at <= lo) return false;
    mine = pre <= lo && lo < pre + cost;
    if (mine) q = x;
    return true;
  };
  if (few) find(q); else for_requests<F>(a, find);
  return mine;
}

// One row tile (pair) of a part, as the roles read it: K/V tiles [t0, t0 + nt) of `all`.
struct Segment {
  int r, g, q0, n, L, pos0;  // request, K/V head, its first query row, queries, context, position of query 0
  int tok0, t0, nt, all;     // first token of slot 0; tiles
  int dirty, clean0, clean1; // first tile (of this segment) with slots past the context; first tile of the item
                             // that rows of slot 0 / 1 see a part of only
  int pair;                  // 1 pair, 0 split, -1 end of the part
};

// With a window: t0 and nt count the item's tiles, and so do clean0 and clean1, low0 and low1.
struct WindowSegment : Segment {
  Run run;
  int low, border;           // first position of the item's windows; first unit of the context without a token below it
  int low0, low1;            // first tile from which the rows of slot 0 / 1 see all of a tile, as far as it goes down
};

template <class F>
using SegmentOf = std::conditional_t<F::kWindow, WindowSegment, Segment>;

// A row tile that several parts share, as its first part leaves it for the joining kernel.
template <class F>
struct Join {
  SegmentOf<F> s;
  uint32_t at, over, cost;
  Plan plan;
  int used;                  // 0: this part has none
};

// Walks the items of part [lo, hi) in order.
template <class F>
struct SegIter {
  const ChunkArgs& a;
  const Plan& plan;
  uint32_t lo, hi, at, cost;
  Req<F> q;
  int r, g, k;
  bool live, fresh;          // fresh: (r, g, k) has not been looked at yet
  __device__ SegIter(const ChunkArgs& args, const Plan& pl, int part, const Req<F>& first, uint32_t pre, bool any)
      : a(args), plan(pl), q(first) {
    live = any;
    if (!any) return;
    lo = plan.lo(part);
    hi = plan.lo(part + 1);
    r = q.r;
    fresh = true;
    const uint32_t per_head = plan.prefix(q, q.items), d = lo - pre;
    g = d / per_head;
    const uint32_t off = d - g * per_head;
    int x = 0, y = q.items - 1;   // largest k with prefix(k) <= off
    while (x < y) {
      const int mid = (x + y + 1) >> 1;
      if (plan.prefix(q, mid) <= off) x = mid; else y = mid - 1;
    }
    k = x;
    at = pre + g * per_head + plan.prefix(q, k);
  }
  __device__ void advance() {
    at += cost;
    if (++k < q.items) return;
    k = 0;
    if (++g < a.c.Hkv) return;
    g = 0;
    do {
      if (++r >= a.R) { live = false; return; }
      q = load_req<F>(a, r);
    } while (q.items == 0);
  }
  // The next segment of the part that has tiles, or an item that sees nothing; false at the end.
  __device__ bool next(SegmentOf<F>& s) {
    while (true) {
      if (!fresh) advance();
      fresh = false;
      if (!live || at >= hi) return false;
      cost = plan.cost(q, k);
      const int per = q.pair ? 2 * a.tpt : a.tpt, lim = limit_of<F>(a, q, min(q.n, (k + 1) * per) - 1);
      const Run run = run_of<F>(a, q, k, lim);
      s.all = tiles_over(a, run_to<F>(a, run, lim));
      int t1;
      cut(lo, hi, at, plan.over(q), cost, s.all, s.t0, t1);
      if (s.all == 0 ? lo > at : t1 <= s.t0) continue;
      s.r = r; s.g = g; s.q0 = q.q0; s.n = q.n; s.L = q.L;
      s.pos0 = static_cast<int>(q.pos0 < -q.n ? -q.n : q.pos0);   // below -n: nothing is visible either way
      s.pair = q.pair;
      s.tok0 = k * per;
      s.nt = t1 - s.t0;
      s.dirty = (run_inside<F>(a, run, q.L) >> a.lupt) - s.t0;
      s.clean0 = run_inside<F>(a, run, limit_of<F>(a, q, s.tok0)) >> a.lupt;
      s.clean1 = q.pair ? run_inside<F>(a, run, limit_of<F>(a, q, min(s.tok0 + a.tpt, q.n - 1))) >> a.lupt : s.clean0;
      if constexpr (F::kWindow) {
        s.run = run;
        s.low = low_of<F>(a, q, s.tok0);
        s.border = F::kPacked ? 0 : units_below(a, s.low);
        s.low0 = tiles_over(a, run_to<F>(a, run, low_of<F>(a, q, min(s.tok0 + a.tpt, q.n) - 1)));
        s.low1 = q.pair ? tiles_over(a, run_to<F>(a, run, low_of<F>(a, q, min(s.tok0 + 2 * a.tpt, q.n) - 1))) : s.low0;
      }
      return true;
    }
  }
};

// ------------------------------------------------------------------ softmax
// One online-softmax step of the row at tensor-memory address s_addr (BN fp32
// columns, raw Q.K^T): P in bf16 pairs goes over the first BN/2 columns, m
// (log2 units) and l are updated; returns the factor O must be scaled by.
// As in the ring kernel a tile is first taken in one pass against the running
// maximum (in a first tile: that of its first 32 columns), which stands while no
// chunk's sum of p exceeds 2^8; a tile in which it does and a masked one take two
// passes (maximum, then exps).  The two passes are rolled loops: they run once or
// twice per row tile, where fetching unrolled code took longer than running it.
// P is rounded to bf16, V's type: both operands of a product on the tensor cores have one, and fp32 or split
// operands would take two products and more for a gain below the rounding of a bf16 output.  l sums p as it is
// before the rounding, so that the LSE is fp32's.
// mask: visible columns of a masked tile.  Rows that are not in use may
// hold NaN scores: they are left out of the votes.
// A prefix of each 16 columns, 8 bits each.
struct PrefixMask {
  uint64_t lm;
  __device__ __forceinline__ uint32_t part(int c) const { return static_cast<uint32_t>(lm >> (16 * c)) & 0xffffu; }   // of columns [32c, +32)
  static constexpr uint32_t kWhole = 0x1010u;
  __device__ static __forceinline__ void apply(uint32_t (&x)[32], uint32_t f) {
    const int l0 = f & 255, l1 = f >> 8;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i >= l0) x[i] = __float_as_uint(-CUDART_INF_F);
      if (i >= l1) x[16 + i] = __float_as_uint(-CUDART_INF_F);
    }
  }
};
struct BitMask {
  static constexpr uint32_t kWhole = 0xffffffffu;
  __device__ static __forceinline__ void apply(uint32_t (&x)[32], uint32_t f) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!(f >> i & 1)) x[i] = __float_as_uint(-CUDART_INF_F);
  }
};

// Positions below `lim` and not below `low`, or below `sink`.  Packed: column i of unit j is position 32 j + i, `skip`
// further from unit `first` on.
struct PackedMask : BitMask {
  Run run;
  int lim, low, sink, unit;      // unit: first of the tile
  __device__ __forceinline__ uint32_t part(int c) const {
    const int j = unit + c, at = 32 * j + (j < run.first ? 0 : run.skip);
    return (low_bits(lim - at) & ~low_bits(low - at)) | low_bits(sink - at);
  }
};
// A position's place: its virtual block, and there the slots before it on device w: `full`, and I more on the devices
// below `w`, `rem` more on w itself.
struct Place {
  int vb, full, w, rem;
  __device__ __forceinline__ void set(const KeyUnits& a, int x) {
    int o, r;
    vb = a.c.by_V.div(x, o);
    full = a.c.by_WI.div(o, r) * a.c.I;
    w = a.c.by_I.div(r, rem);
  }
  // slots of unit (vb, sub, w) that hold tokens before it: unit_visible() without divisions
  __device__ __forceinline__ int before(const KeyUnits& a, int v, int sub, int dev) const {
    if (v != vb) return v < vb ? 1 << a.lu : 0;
    return full + (dev < w ? a.c.I : dev == w ? rem : 0) - (sub << a.lu);
  }
};
struct WindowMask : BitMask {
  const ChunkArgs& a;
  const Place &lim, &low, &sink;
  Run run;
  int unit, r;
  bool bad;
  __device__ __forceinline__ uint32_t one(int j) const {
    int rem, w;
    const int vb = a.by_vbu.div(j + (j < run.first ? 0 : run.skip), rem), sub = a.c.by_W.div(rem, w);
    const uint32_t all = low_bits(1 << a.lu);
    const uint32_t m = (low_bits(lim.before(a, vb, sub, w)) & ~low_bits(low.before(a, vb, sub, w))) |
                       low_bits(sink.before(a, vb, sub, w));
    if (!bad || m == 0) return m & all;
    const int32_t b = vb < a.c.max_vb ? a.c.table[static_cast<int64_t>(r) * a.c.max_vb + vb] : -1;
    return b < 0 || b >= a.c.num_blocks ? 0 : m & all;
  }
  __device__ __forceinline__ uint32_t part(int c) const {
    if (a.lu == 5) return one(unit + c);
    return one(unit + 2 * c) | one(unit + 2 * c + 1) << 16;
  }
};
template <class Mask>
__device__ __forceinline__ float softmax_step(uint32_t s_addr, bool first, bool masked, bool row_ok, const Mask& mask,
                                              float scale, float& m, float& l) {
  const uint64_t sc2 = f2pack(scale, scale);
  if (!masked) {
    uint32_t pk[BN / 2];
    float lsum = 0.f;
    uint32_t xa[32], xb[32];
    tmem_ld32(s_addr, xa);
    tmem_wait_ld();
    if (first) m = chunk_mask_max(xa, 0, false, 0) * scale;
    const uint64_t negm2 = f2pack(-m, -m);
    bool grow = __any_sync(0xffffffffu, row_ok && m == -CUDART_INF_F);
#pragma unroll
    for (int c = 0; c < BN / 32; ++c) {
      if (grow) break;
      uint32_t (&x)[32] = (c & 1) ? xb : xa;
      uint32_t (&y)[32] = (c & 1) ? xa : xb;
      if (c + 1 < BN / 32) tmem_ld32(s_addr + 32 * (c + 1), y);
      uint64_t acc0 = f2pack(0.f, 0.f), acc1 = acc0;
      chunk_exp_pack(x, sc2, negm2, acc0, acc1, &pk[16 * c]);
      float a0, a1, b0, b1;
      f2unpack(acc0, a0, a1);
      f2unpack(acc1, b0, b1);
      const float cs = (a0 + a1) + (b0 + b1);
      if (__any_sync(0xffffffffu, row_ok && !(cs <= kChunkSumLimit))) { grow = true; tmem_wait_ld(); break; }
      lsum += cs;
      if (c + 1 < BN / 32) tmem_wait_ld();
    }
    if (!grow) {
      l += lsum;
      tmem_st32(s_addr, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
      tmem_st32(s_addr + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
      return 1.f;
    }
  }
  // A chunk of a masked tile is whole for the warp, out of sight for all of it, or neither.
  auto load = [&](uint32_t (&x)[32], int c, uint32_t f) {
    tmem_ld32(s_addr + 32 * c, x);
    tmem_wait_ld();
    if (masked && !__all_sync(0xffffffffu, f == Mask::kWhole)) Mask::apply(x, f);
  };
  float mx = -CUDART_INF_F;
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    const uint32_t f = masked ? mask.part(c) : 0;
    if (masked && !__any_sync(0xffffffffu, f != 0)) continue;
    uint32_t x[32];
    load(x, c, f);
    mx = fmaxf(mx, chunk_mask_max(x, 0, false, 0));
  }
  const float m_tile = mx * scale;
  const bool need = first || (m_tile > m + 8.f);
  const float m_use = need ? fmaxf(m, m_tile) : m;
  const float m_ref = (m_use == -CUDART_INF_F) ? 0.f : m_use;
  const float alpha = first ? 0.f : ex2(m - m_ref);
  const uint64_t negm2 = f2pack(-m_ref, -m_ref);
  uint64_t acc0 = f2pack(0.f, 0.f), acc1 = acc0;
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {   // P of chunk c goes over scores that have been read
    const uint32_t f = masked ? mask.part(c) : 0;
    uint32_t x[32], pk[16];
    if (masked && !__any_sync(0xffffffffu, f != 0)) {
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[i] = 0;
    } else {
      load(x, c, f);
      chunk_exp_pack(x, sc2, negm2, acc0, acc1, pk);
    }
    tmem_st16(s_addr + 16 * c, pk);
  }
  float a0, a1, b0, b1;
  f2unpack(acc0, a0, a1);
  f2unpack(acc1, b0, b1);
  const float rs = (a0 + a1) + (b0 + b1);
  l = first ? rs : l * alpha + rs;
  m = m_use;
  return first ? 1.f : alpha;
}

// ------------------------------------------------------------------ the kernel
constexpr int kSegs = 4;          // segments announced ahead
constexpr int kSegReaders = 11;   // warps that read them: TMA, MMA, zeroing and 8 of softmax

// A stage of the K/V ring holds one tile (D = 128: 32 KB), or V_j with the K tile that is used right after it
// (D = 64: 2 x 16 KB): there the MMA thread and the TMA warp, at some 130 cycles for each wait, would take longer
// than HBM for tiles of their own.
template <int D>
constexpr bool kJoint = D == 64;
template <int D>
constexpr int kStages = D == 128 ? 5 : 6;

// Score tiles in tensor memory.  With three (where the accumulators leave room: D = 64) the score product of a
// split tile runs while both slots are at their softmax.  With the joint stages below: 64 requests of 1-4 tokens
// over 2000-9000, blocks of 128, 135 us (5.2 TB/s) instead of 155.
template <int D>
constexpr int kScores = D == 64 ? 3 : 2;

template <int D, class F>
struct __align__(1024) ChunkSmem {
  uint8_t q[2][BM * D * 2];
  uint8_t kv[kStages<D>][(kJoint<D> ? 2 : 1) * BN * D * 2];   // joint: V, K
  uint64_t q_full[2], q_empty[2], kv_full[kStages<D>], kv_empty[kStages<D>], v_dirty[kStages<D>], v_clean[kStages<D>];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  // With three score tiles slot h uses 2h and 2h + 1 in turn, so that a phase never ends before the one before it
  // has been seen; else h.
  uint64_t s_full[4], p_full[4], pv_done[4];
  uint64_t o_empty[2], ml_full, ml_empty, drain;
  float2 ml[BM];
  SegmentOf<F> seg[kSegs];
  uint32_t tmem_base;
  int abort_flag, bad_block;
};

static_assert(sizeof(ChunkSmem<128, WindowPaged>) + 1024 <= 232448 && sizeof(ChunkSmem<64, WindowPaged>) + 1024 <= 232448,
              "227 KB of shared memory");

// A role's reading of the announced segments, in order, by a whole warp.
struct SegReader {
  uint32_t at = 0;
  bool ok = true;   // false: a wait expired, the part has not ended
  template <class Smem, class Seg>
  __device__ bool next(Smem& sm, Seg& s, volatile int* abort_flag, long long limit) {
    const int i = at & (kSegs - 1);
    const uint32_t bar = smem_u32(&sm.seg_full[i]), ph = (at / kSegs) & 1;
    ok = warp_wait(bar, ph, abort_flag, limit, 570);
    if (!ok) return false;
    s = sm.seg[i];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sm.seg_empty[i]));
    ++at;
    return s.pair >= 0;
  }
};

template <int D, class F>
__global__ void __launch_bounds__(kChunkThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ ChunkArgs a) {
  constexpr int SLABS = D / 64, NS = kStages<D>, NB = kScores<D>;
  constexpr uint32_t kTileBytes = BM * D * 2, kStageBytes = (kJoint<D> ? 2 : 1) * kTileBytes;
  constexpr uint32_t kInStage = kStageBytes - kTileBytes;   // of K
  constexpr uint32_t kColAcc = NB * BN;   // accumulator of slot h: D columns from kColAcc + h * D
  static_assert(kColAcc + 2 * D <= kTmemCols && NS > (kJoint<D> ? NB : 2 * NB - 1));
  constexpr uint32_t kIdescS = idesc_bf16_f32(BM, BN, 0, 0);
  constexpr uint32_t kIdescO = idesc_bf16_f32(BM, D, 0, 1);

  extern __shared__ uint8_t smem_raw[];
  ChunkSmem<D, F>& sm = *reinterpret_cast<ChunkSmem<D, F>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const long long lim = a.wait_limit;
  // barrier (of four) and parity of a slot's c-th use
  auto turn = [](int h, uint32_t c) { return NB == 3 ? 2 * h + (c & 1) : h; };
  auto phase = [](uint32_t c) { return NB == 3 ? (c >> 1) & 1 : c & 1; };

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sm.q_full[b]), 1);
      mbar_init(smem_u32(&sm.q_empty[b]), 1);
      mbar_init(smem_u32(&sm.o_empty[b]), 128);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(smem_u32(&sm.s_full[b]), 1);
      mbar_init(smem_u32(&sm.p_full[b]), 128);
      mbar_init(smem_u32(&sm.pv_done[b]), 1);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(smem_u32(&sm.seg_full[s]), 1);
      mbar_init(smem_u32(&sm.seg_empty[s]), kSegReaders);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&sm.kv_full[s]), 1);
      mbar_init(smem_u32(&sm.kv_empty[s]), 1);
      mbar_init(smem_u32(&sm.v_dirty[s]), 1);
      mbar_init(smem_u32(&sm.v_clean[s]), 1);
    }
    mbar_init(smem_u32(&sm.ml_full), 128);
    mbar_init(smem_u32(&sm.ml_empty), 128);
    mbar_init(smem_u32(&sm.drain), 1);
    sm.abort_flag = 0;
    sm.bad_block = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  Plan plan;
  Req<F> first{};
  uint32_t pre = 0;
  bool mine = false;
  if (warp == 3) mine = make_plan<F>(a, blockIdx.x, plan, first, pre);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  // the joining kernel may come up and make its plan meanwhile; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  SegReader segs;
  SegmentOf<F> sg;

  // Order of the K/V ring in a segment: K_0 .. K_{la-1}, then V_j, K_{j+la} for each j (joint: in one stage), with
  // la = 1 (pair: both slots meet tile j) or NB (split: slot j & 1 meets tile j).
  if (warp == 0) {
    // ============================================================ TMA producer (whole warp: 64 columns of a unit per lane)
    // lanes below `half` for V, the others for K
    const int unit = lane & ((1 << a.lupt) - 1), slab = (lane >> a.lupt) & (SLABS - 1), half = SLABS << a.lupt;
    const bool is_k = lane >= half, used = lane < 2 * half;
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    Ring<NS> ring;
    uint32_t issued = 0;                      // ring entries so far
    uint32_t q_cnt[2] = {0, 0};
    int q_next = 0;
    bool ok = true;
    const uint64_t once = policy_once();      // a split tile's keys are read by one CTA
    const int oob = static_cast<int>(a.c.W * a.c.num_blocks * a.c.Hkv);   // past the last block: zero fill
    while (ok && segs.next(sm, sg, abort_flag, lim)) {
      const int nt = sg.nt;
      if (nt <= 0) continue;
      const bool pair = sg.pair;
      const int la = pair ? 1 : NB, nq = pair ? 2 : 1;
      struct Unit {
        int s0, w, blk;
      };
      // A stage: a tile of V, of K, or both.
      auto load = [&](const Unit* v, bool to_clean, const Unit* k) -> bool {
        if (!warp_wait(smem_u32(&sm.kv_empty[ring.st]), ring.ph ^ 1, abort_flag, lim, 521)) return false;
        const uint32_t bar = smem_u32(&sm.kv_full[ring.st]);
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, v && k ? 2 * kTileBytes : kTileBytes);
          if (v && to_clean) mbar_arrive(smem_u32(&sm.v_dirty[ring.st]));
        }
        __syncwarp();
        if (used && (is_k ? k != nullptr : v != nullptr)) {
          const Unit x = is_k ? *k : *v;
          const CUtensorMap* map = is_k ? &tmK : &tmV;
          const uint32_t dst = smem_u32(sm.kv[ring.st] + (is_k ? kInStage : 0) + slab * BN * 128 + (unit << a.lu) * 128);
          if (F::kPacked) {
            tma_load_3d(dst, map, bar, 64 * slab, sg.g, x.s0);
          } else {
            const int hb = x.blk < 0 ? oob : static_cast<int>((x.w * a.c.num_blocks + x.blk) * a.c.Hkv + sg.g);
            if (pair) tma_load_3d(dst, map, bar, 64 * slab, x.s0, hb);
            else tma_load_3d_once(dst, map, bar, 64 * slab, x.s0, hb, once);
          }
        }
        ++issued;
        ring.advance();
        return true;
      };
      // lane's unit of tile j: device, slot, id of its block; the id is looked at one tile later, so that its
      // load is in flight while the ring is waited for
      auto locate = [&](int j) {
        Unit x;
        int j_unit = ((sg.t0 + j) << a.lupt) + unit;
        bool first = false;   // first tokens
        if constexpr (F::kWindow) {
          first = j_unit < sg.run.first;
          if (F::kPacked) {
            x.s0 = sg.q0 + 32 * j_unit + (first ? 0 : sg.run.skip);
            x.w = x.blk = 0;
            return x;
          }
          if (!first) j_unit += sg.run.skip;
        }
        int rem;
        const int vb = a.by_vbu.div(j_unit, rem);
        const int sub = a.c.by_W.div(rem, x.w);
        x.s0 = sub << a.lu;
        x.blk = -1;
        bool sees = j < nt && used && static_cast<int64_t>(vb) * a.c.V < sg.L;
        // a unit none of whose tokens is in sight is not looked at: its block may be gone
        if constexpr (F::kWindow)
          if (sees && (first || j_unit < sg.border))
            sees = unit_visible(a, vb, sub, x.w, a.n_sink) > 0 || unit_visible(a, vb, sub, x.w, sg.low) < (1 << a.lu);
        if (sees) {
          x.blk = a.c.table[static_cast<int64_t>(sg.r) * a.c.max_vb + vb];
          if (x.blk < 0) x.blk = INT32_MAX;   // in the context, so that a bad id is one
        }
        return x;
      };
      auto checked = [&](Unit& x) {
        if (F::kPacked) return;
        if (x.blk >= a.c.num_blocks) {
          ra_record_error(RA_ERR_DEVICE_BOUNDS, 512);
          *reinterpret_cast<volatile int*>(&sm.bad_block) = 1;
          x.blk = -1;
        }
        __syncwarp();
      };
      // u[i]: unit of tile j + i; the K tiles up to j + la have been issued but for the last
      Unit u[NB + 1];
#pragma unroll
      for (int i = 0; i <= NB; ++i) u[i] = locate(i);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        if (ok && i < la && i < nt) {
          checked(u[i]);
          ok = load(nullptr, false, &u[i]);
        }
      for (int h = 0; h < nq && ok; ++h) {
        const int b = sg.pair ? h : q_next;
        ok = warp_wait(smem_u32(&sm.q_empty[b]), (q_cnt[b] & 1) ^ 1, abort_flag, lim, 520);
        if (!ok) break;
        ++q_cnt[b];
        if (lane == 0) {
          const uint32_t qb = smem_u32(&sm.q_full[b]);
          mbar_arrive_expect_tx(qb, SLABS * a.tpt * a.G * 128);
          const int row = sg.q0 + sg.tok0 + h * a.tpt;
          for (int s = 0; s < SLABS; ++s)
            tma_load_3d(smem_u32(sm.q[b] + s * BM * 128), &tmQ, qb, 64 * s, sg.g * a.G, row);
        }
        __syncwarp();
      }
      if (!sg.pair) q_next ^= 1;
      for (int j = 0; j < nt && ok; ++j) {
        const Unit ahead = locate(j + NB + 1);
        Unit k = pair ? u[1] : u[NB];
        const bool more = j + la < nt;
        if (more) {
          checked(k);
          if (pair) u[1] = k; else u[NB] = k;
        }
        if (kJoint<D>) {
          ok = load(&u[0], j >= sg.dirty, more ? &k : nullptr);
        } else {
          ok = load(&u[0], j >= sg.dirty, nullptr) && (!more || load(nullptr, false, &k));
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < NB; ++i) u[i] = u[i + 1];
        u[NB] = ahead;
      }
    }
    if (lane == 0) {
      // The last load of each buffer lands before the CTA exits, also where another role has given up, or gives up
      // from here on (else each has been waited for by its reader).
      for (int b = 0; b < 2; ++b)
        if (q_cnt[b]) mbar_wait_quiesce(smem_u32(&sm.q_full[b]), (q_cnt[b] - 1) & 1, 1 << 22);
      for (int s = 0; s < NS; ++s) {
        const uint32_t n = issued / NS + (static_cast<uint32_t>(s) < issued % NS ? 1 : 0);
        if (n) mbar_wait_quiesce(smem_u32(&sm.kv_full[s]), (n - 1) & 1, 1 << 22);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    {
      // The whole warp runs this, with one lane elected to issue: operands are then in uniform registers.  Issued by a branch
      // of one thread, a product of 8 instructions took it some 560 cycles whatever its size.
      const uint32_t leader = elect_one();
      Ring<NS> ring;
      uint32_t s0 = 0, s1 = 0, p0 = 0, p1 = 0;   // score tiles issued, P taken, of each slot
      uint32_t q_cnt[2] = {0, 0}, seg = 0, clean_ph = 0;
      int q_next = 0;
      bool ok = true, p_ready = false, v_ready = false, k_ready = false;
      const uint64_t dq0 = desc_sw128(smem_u32(sm.q[0]), 16, 1024);
      const uint64_t dk0 = desc_sw128(smem_u32(sm.kv[0] + kInStage), 16, 1024);
      const uint64_t dv0 = desc_sw128(smem_u32(sm.kv[0]), BN * 128, 1024);
      // A wait that passes at once takes some 130 cycles with the tensor core idle, so the next barriers are looked
      // at while the last products are queued.
      auto test_p = [&](int h) {
        const uint32_t c = h ? p1 : p0;
        return warp_test(smem_u32(&sm.p_full[turn(h, c)]), phase(c));
      };
      auto test_kv = [&] { return warp_test(smem_u32(&sm.kv_full[ring.st]), ring.ph); };
      auto wait_p = [&](int h, int site) -> bool {
        const uint32_t c = h ? p1 : p0;
        if (!p_ready && !warp_wait(smem_u32(&sm.p_full[turn(h, c)]), phase(c), abort_flag, lim, site)) return false;
        p_ready = false;
        if (h) ++p1; else ++p0;
        return true;
      };
      // scores of slot h into tile b: Q tile qb, K tile st; `then` is called while the last products are queued
      auto issue_s = [&](int h, int b, int qb, int st, auto then) {
        const uint64_t dq = dq0 + qb * (kTileBytes >> 4), dk = dk0 + st * (kStageBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off16 = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
          mma_bf16_ss_by(leader, tmem + b * BN, dq + off16, dk + off16, kIdescS, kk > 0 ? 1u : 0u);
          if (kk == D / 16 - 3) then();
        }
        mma_commit_by(leader, smem_u32(&sm.s_full[turn(h, h ? s1++ : s0++)]));
      };
      auto issue_pv = [&](int h, int b, int st, bool first, auto then) {
        const uint64_t dv = dv0 + st * (kStageBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) {
          mma_bf16_ts_by(leader, tmem + kColAcc + h * D, tmem + b * BN + kk * 8, dv + ((kk * 16 * 128) >> 4), kIdescO,
                      (kk > 0 || !first) ? 1u : 0u);
          if (kk == BN / 16 - 3) then();
        }
        mma_commit_by(leader, smem_u32(&sm.pv_done[turn(h, (h ? p1 : p0) - 1)]));   // its P has been counted
      };
      auto nothing = [] {};
      // the V tile at the ring's head is in place, its dead rows zeroed
      auto wait_v = [&](int j, int dirty) -> bool {
        if (!v_ready && !warp_wait(smem_u32(&sm.kv_full[ring.st]), ring.ph, abort_flag, lim, 531)) return false;
        v_ready = false;
        if (j >= dirty) {
          if (!warp_wait(smem_u32(&sm.v_clean[ring.st]), (clean_ph >> ring.st) & 1, abort_flag, lim, 532)) return false;
          clean_ph ^= 1u << ring.st;
        }
        return true;
      };
      while (ok && segs.next(sm, sg, abort_flag, lim)) {
        const int nt = sg.nt;
        if (nt <= 0) continue;
        const int dirty = sg.dirty;
        const bool pair = sg.pair;
        const int qb = pair ? 0 : q_next;
        if (!(ok = warp_wait(smem_u32(&sm.q_full[qb]), q_cnt[qb] & 1, abort_flag, lim, 530))) break;
        ++q_cnt[qb];
        if (pair) {
          if (!(ok = warp_wait(smem_u32(&sm.q_full[1]), q_cnt[1] & 1, abort_flag, lim, 530))) break;
          ++q_cnt[1];
        } else {
          q_next ^= 1;
        }
        auto q_release = [&] {
          mma_commit_by(leader, smem_u32(&sm.q_empty[qb]));
          if (pair) mma_commit_by(leader, smem_u32(&sm.q_empty[1]));
        };
        const uint32_t oph = (seg & 1) ^ 1;
        if (pair) {
          if (!(ok = warp_wait(smem_u32(&sm.kv_full[ring.st]), ring.ph, abort_flag, lim, 533))) break;
          tc_fence_after();
          issue_s(0, 0, 0, ring.st, nothing);
          issue_s(1, 1, 1, ring.st, nothing);
          mma_commit_by(leader, smem_u32(&sm.kv_empty[ring.st]));
          ring.advance();
          if (nt == 1) q_release();
          for (int j = 0; j < nt; ++j) {
            const bool more = j + 1 < nt;
            if (!(ok = wait_v(j, dirty))) break;
            const int sv = ring.st;
            ring.advance();
            if (!kJoint<D> && more && !(ok = warp_wait(smem_u32(&sm.kv_full[ring.st]), ring.ph, abort_flag, lim, 534))) break;
            const int sk = kJoint<D> ? sv : ring.st;
            if (j == 0 && !(ok = warp_wait(smem_u32(&sm.o_empty[0]), oph, abort_flag, lim, 535))) break;
            if (j == 0 && !(ok = warp_wait(smem_u32(&sm.o_empty[1]), oph, abort_flag, lim, 536))) break;
            if (!(ok = wait_p(0, 537))) break;
            tc_fence_after();
            issue_pv(0, 0, sv, j == 0, nothing);
            if (more) issue_s(0, 0, 0, sk, [&] { p_ready = test_p(1); });
            if (!(ok = wait_p(1, 538))) break;
            tc_fence_after();
            issue_pv(1, 1, sv, j == 0, nothing);
            if (!kJoint<D> || !more) mma_commit_by(leader, smem_u32(&sm.kv_empty[sv]));
            if (more) {
              issue_s(1, 1, 1, sk, nothing);
              mma_commit_by(leader, smem_u32(&sm.kv_empty[sk]));
              if (!kJoint<D>) ring.advance();
              if (j + 2 == nt) q_release();
            }
          }
        } else {
          for (int j = 0; j < NB && j < nt; ++j) {
            if (!(ok = warp_wait(smem_u32(&sm.kv_full[ring.st]), ring.ph, abort_flag, lim, 533))) break;
            tc_fence_after();
            issue_s(j & 1, j, qb, ring.st, nothing);
            mma_commit_by(leader, smem_u32(&sm.kv_empty[ring.st]));
            ring.advance();
          }
          if (!ok) break;
          if (nt <= NB) q_release();
          for (int j = 0, b = 0; j < nt; ++j, b = b + 1 == NB ? 0 : b + 1) {
            const int h = j & 1;
            const bool more = j + NB < nt;
            if (!(ok = wait_v(j, dirty))) break;
            const int sv = ring.st;
            ring.advance();
            if (j < 2 && !(ok = warp_wait(smem_u32(&sm.o_empty[h]), oph, abort_flag, lim, 535))) break;
            if (!(ok = wait_p(h, 537))) break;
            tc_fence_after();
            k_ready = kJoint<D>;
            issue_pv(h, b, sv, j < 2, [&] { if (!kJoint<D>) k_ready = more && test_kv(); });
            if (!kJoint<D> || !more) mma_commit_by(leader, smem_u32(&sm.kv_empty[sv]));
            if (more) {
              if (!k_ready && !(ok = warp_wait(smem_u32(&sm.kv_full[ring.st]), ring.ph, abort_flag, lim, 534))) break;
              const int sk = kJoint<D> ? sv : ring.st;
              if (!kJoint<D>) ring.advance();
              issue_s((j + NB) & 1, b, qb, sk, [&] {
                v_ready = test_kv();
                p_ready = test_p(h ^ 1);
              });
              mma_commit_by(leader, smem_u32(&sm.kv_empty[sk]));
              if (j + NB + 1 == nt) q_release();
            }
          }
        }
        ++seg;
      }
      // Every product lands before tensor memory is given back, however short the limit of the other waits and
      // whichever of them expired (in its own loop, or for a segment).
      mma_commit_by(leader, smem_u32(&sm.drain));
      if (!__all_sync(0xffffffffu, mbar_wait_quiesce(smem_u32(&sm.drain), 0, a.drain_limit)) && ok && segs.ok) {
        *abort_flag = 1;
        ra_record_error(RA_ERR_TIMEOUT, 539);
      }
    }
  } else if (warp == 2) {
    // ============================================================ zeroing of V rows past the context
    // A dirty tile is taken up once the producer has announced it: from then on its stage's barrier can
    // only move from loading to loaded, so that the parity waited for is the right one.  Other tiles are passed over here
    // while the other roles work them off, which the limits allow for.
    Ring<NS> ring;
    uint32_t dirty_ph = 0;
    long long past = 0;                // tiles, a segment's start and end counted as one, since the last dirty one
    bool ok = true;
    while (ok && segs.next(sm, sg, abort_flag, limit_over(lim, past))) {
      const int nt = sg.nt;
      ++past;
      if (nt <= 0) continue;
      const int la = sg.pair ? 1 : NB;
      for (int j = 0; j < min(la, nt); ++j) ring.advance();
      for (int j = 0; j < nt; ++j) {
        if (j >= sg.dirty) {
          if (!(ok = warp_wait(smem_u32(&sm.v_dirty[ring.st]), (dirty_ph >> ring.st) & 1, abort_flag, limit_over(lim, past), 540)))
            break;
          past = 0;
          dirty_ph ^= 1u << ring.st;
          if (!(ok = warp_wait(smem_u32(&sm.kv_full[ring.st]), ring.ph, abort_flag, lim, 541))) break;
          const uint64_t lm = F::kWindow ? 0 : tile_limits(a, sg.r, false, sg.t0 + j, sg.L);
#pragma unroll 1
          for (int i0 = 0; i0 < BN; i0 += 32) {
            const int i = i0 + lane;
            bool dead = (lane & 15) >= (static_cast<int>(lm >> (8 * (i >> 4))) & 255);
            if constexpr (F::kWindow) {
              const int j_unit = ((sg.t0 + j) << a.lupt) + (i >> a.lu), shift = j_unit < sg.run.first ? 0 : sg.run.skip;
              if (F::kPacked) {
                dead = 32 * j_unit + (i & 31) + shift >= sg.L;
              } else {
                int rem, w;
                const int vb = a.by_vbu.div(j_unit + shift, rem), sub = a.c.by_W.div(rem, w);
                dead = (i & ((1 << a.lu) - 1)) >= unit_visible(a, vb, sub, w, sg.L);
              }
            }
            if (dead) {
#pragma unroll
              for (int s = 0; s < SLABS; ++s)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  *reinterpret_cast<uint4*>(sm.kv[ring.st] + s * BN * 128 + i * 128 + e * 16) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.v_clean[ring.st]));
          __syncwarp();
        } else {
          ++past;
        }
        ring.advance();
        if (!kJoint<D> && j + la < nt) ring.advance();
      }
    }
  } else if (warp == 3) {
    // ============================================================ segments of this part, announced to the other roles
    const unsigned owner = __ballot_sync(0xffffffffu, mine);
    if (mine || (owner == 0 && lane == 0)) {
      bool more = mine, left = false;
      Join<F>* join = static_cast<Join<F>*>(a.join);
      SegIter<F> it(a, plan, blockIdx.x, first, pre, mine);
      uint32_t i = 0;
      int longest = 0;                   // segment so far, in tiles: as long as one, the others may take to read the next
      do {
        if (more) more = it.next(sg);
        if (!more) sg.pair = -1;
        const int b = i & (kSegs - 1);
        if (!mbar_wait(smem_u32(&sm.seg_empty[b]), ((i / kSegs) & 1) ^ 1, abort_flag, limit_over(lim, longest), 572)) break;
        if (more) longest = max(longest, sg.nt);
        sm.seg[b] = sg;
        mbar_arrive(smem_u32(&sm.seg_full[b]));
        if (more && sg.t0 == 0 && sg.nt < sg.all) {
          join[blockIdx.x] = Join<F>{sg, it.at, plan.over(it.q), it.cost, plan, 1};
          left = true;
        }
        ++i;
      } while (more);
      if (!left) join[blockIdx.x].used = 0;
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ============================================================ softmax + epilogue (slot h)
    const int h = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t colO = kColAcc + h * D;
    const int row_tok = row / a.G, row_head = row - row_tok * a.G;
    uint32_t s_cnt = 0, pv_cnt[2] = {0, 0}, splits = 0;
    // product i of a slot is in its accumulator
    auto wait_pv = [&](int slot, uint32_t i, int site) {
      return warp_wait(smem_u32(&sm.pv_done[turn(slot, i)]), phase(i), abort_flag, lim, site);
    };
    bool ok = true;
    while (ok && segs.next(sm, sg, abort_flag, lim)) {
      const int nt = sg.nt;
      const bool pair = sg.pair;
      const int tok = sg.tok0 + (pair ? h * a.tpt : 0) + row_tok;
      const bool row_ok = row_tok < a.tpt && tok < sg.n;
      const int64_t orow = static_cast<int64_t>(sg.q0 + tok) * a.Hq + sg.g * a.G + row_head;
      if (nt <= 0) {   // the tile sees nothing
        if (row_ok && (pair || h == 0)) {
          for (int e = 0; e < D; e += 8) {
            if (a.out_bf16) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + orow * D + e) = make_uint4(0, 0, 0, 0);
            else {
              float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.o) + orow * D + e);
              dst[0] = dst[1] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
          }
          if (a.lse) a.lse[orow] = -CUDART_INF_F;
        }
        continue;
      }
      // visible positions of this row, and the first tile in which the slot's first row sees a part only
      const int seen = sg.pos0 + min(tok, sg.n - 1) + 1;
      const int vis = F::kWindow || a.causal ? max(0, min(sg.L, seen)) : sg.L;
      const int clean = h ? sg.clean1 : sg.clean0;
      // with a window: its first position, the first tokens that are there, and tiles below which it is masked
      int low = 0, low_tile = 0;
      [[maybe_unused]] const int sinks = F::kWindow ? min(a.n_sink, vis) : 0;
      [[maybe_unused]] Place lim_place, low_place, sink_place;
      if constexpr (F::kWindow) {
        low = seen > a.window ? min(sg.L, seen - a.window) : 0;
        low_tile = h ? sg.low1 : sg.low0;
        if constexpr (!F::kPacked) {
          lim_place.set(a, vis);
          low_place.set(a, low);
          sink_place.set(a, sinks);
        }
      }
      const bool warp_live = __any_sync(0xffffffffu, row_ok);
      float m = -CUDART_INF_F, l = 0.f;
      const int step = pair ? 1 : 2;
      int n_mine = 0;                      // tiles of this slot so far
      int b = h;                           // score tile
      for (int j = pair ? 0 : h; j < nt; j += step) {
        const int use = turn(h, s_cnt);
        if (!(ok = warp_wait_first(smem_u32(&sm.s_full[use]), phase(s_cnt), abort_flag, lim, 550 + h))) break;
        ++s_cnt;
        tc_fence_after();
        const uint32_t colS = (NB == 3 ? b : h) * BN;
        if (warp_live) {
          const bool bad = *reinterpret_cast<volatile int*>(&sm.bad_block) != 0;
          const int tile = sg.t0 + j;
          const bool masked = tile >= clean || bad || (F::kWindow && tile < low_tile);
          auto mask = [&] {
            if constexpr (!F::kWindow) return PrefixMask{masked ? tile_limits(a, sg.r, bad, tile, vis) : 0};
            else if constexpr (F::kPacked) return PackedMask{{}, sg.run, vis, low, sinks, tile << a.lupt};
            else return WindowMask{{}, a, lim_place, low_place, sink_place, sg.run, tile << a.lupt, sg.r, bad};
          }();
          const float alpha = softmax_step(t_lane + colS, n_mine == 0, masked, row_ok, mask, a.scale_log2, m, l);
          if (n_mine > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // O_h must hold the previous P.V before it is rescaled
            if (!(ok = wait_pv(h, pv_cnt[h] + n_mine - 1, 552 + h))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c4 = 0; c4 < D / 32; ++c4) {
              uint32_t orr[32];
              tmem_ld32(t_lane + colO + 32 * c4, orr);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) orr[i] = __float_as_uint(__uint_as_float(orr[i]) * alpha);
              tmem_st32(t_lane + colO + 32 * c4, orr);
            }
          }
          tmem_wait_st();
        }
        ++n_mine;
        tc_fence_before();
        mbar_arrive(smem_u32(&sm.p_full[use]));
        if (NB == 3 && !pair) b = b == 0 ? 2 : b - 1;   // two tiles on
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      const bool whole = nt == sg.all;
      const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (sg.t0 == 0 ? 1 : 0);
      pv_cnt[0] += pair ? nt : (nt + 1) / 2;   // both slots' products so far, whichever this thread waits for
      pv_cnt[1] += pair ? nt : nt / 2;
      if (!pair && h == 1) {
        // hand (m, l) to slot 0, which joins the two accumulators
        if (!(ok = warp_wait(smem_u32(&sm.ml_empty), (splits & 1) ^ 1, abort_flag, lim, 560))) break;
        sm.ml[row] = make_float2(n_mine ? m : -CUDART_INF_F, n_mine ? l : 0.f);
        mbar_arrive(smem_u32(&sm.ml_full));
        ++splits;
        continue;
      }
      if (!(ok = wait_pv(h, pv_cnt[h] - 1, 554 + h))) break;
      float f0 = 1.f, f1 = 0.f;
      bool two = false;
      if (!pair) {
        if (!(ok = warp_wait(smem_u32(&sm.ml_full), splits & 1, abort_flag, lim, 561))) break;
        ++splits;
        const float2 ml1 = sm.ml[row];
        mbar_arrive(smem_u32(&sm.ml_empty));
        two = nt > 1;
        if (two && !(ok = wait_pv(1, pv_cnt[1] - 1, 556))) break;
        const float M = fmaxf(m, ml1.x);
        f0 = M == -CUDART_INF_F ? 0.f : ex2(m - M);
        f1 = M == -CUDART_INF_F ? 0.f : ex2(ml1.x - M);
        l = l * f0 + ml1.y * f1;
        m = M;
      }
      tc_fence_after();
      const float inv_l = !whole ? 1.f : (l != 0.f ? 1.f / l : 0.f);
      f0 *= inv_l;
      f1 *= inv_l;
      if (warp_live) {
        float* po = a.o_part + ((part * 2 + (pair ? h : 0)) * BM + row) * D;
#pragma unroll 1
        for (int c4 = 0; c4 < D / 32; ++c4) {
          uint32_t x[32];
          tmem_ld32(t_lane + colO + 32 * c4, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f0);
          if (two) {
            uint32_t y[32];
            tmem_ld32(t_lane + kColAcc + D + 32 * c4, y);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) + __uint_as_float(y[i]) * f1);
          }
          if (whole && a.out_bf16) {
            store_rows_bf16(static_cast<__nv_bfloat16*>(a.o) + 32 * c4, row_ok ? orow * D : -1, x, 1.f);
          } else if (row_ok) {
            uint4* dst = reinterpret_cast<uint4*>((whole ? static_cast<float*>(a.o) + orow * D : po) + 32 * c4);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&sm.o_empty[h]));
      if (!pair) mbar_arrive(smem_u32(&sm.o_empty[1]));
      if (row_ok) {
        if (!whole) a.ml_part[(part * 2 + (pair ? h : 0)) * BM + row] = make_float2(m, l);
        else if (a.lse) a.lse[orow] = l != 0.f ? (m + log2f(l)) * kLn2 : -CUDART_INF_F;
      }
    }
    tmem_wait_st();   // a wait that expires between P's stores and their own wait leaves them in flight
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ joining
// Row tiles that several parts share: block (c, y) takes the one that part c starts, if it does.  A warp per row.
template <int D, class F>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const __grid_constant__ ChunkArgs a) {
  constexpr int E = D / 32;
  __shared__ int parts[kCtas], n_parts;
  __shared__ __align__(16) float sums[kMergeThreads / 32][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // what the first kernel wrote is complete, and visible, once it has ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Join<F> jn = static_cast<const Join<F>*>(a.join)[blockIdx.x];   // whole, in one latency
  if (jn.used == 0) return;
  const SegmentOf<F> sg = jn.s;
  const int slots = sg.pair ? 2 : 1;
  const int rows = min(sg.n - sg.tok0, slots * a.tpt) * a.G;
  if (static_cast<int>(blockIdx.y) * (rows <= kFewRows ? 1 : (kMergeThreads / 32) * 2) >= rows) return;   // no row in either scheme
  if (warp == 0) {
    // the partials, in order: of this part, and of those that follow
    const Plan plan = jn.plan;
    const uint32_t at = jn.at, over = jn.over, cost = jn.cost;
    int n = 0;
    for (int c0 = blockIdx.x; c0 < kCtas && plan.lo(c0) < at + cost; c0 += 32) {
      const int c = c0 + lane;
      int t0 = 0, t1 = 0;
      if (c < kCtas && plan.lo(c) < at + cost) cut(plan.lo(c), plan.lo(c + 1), at, over, cost, sg.all, t0, t1);
      const unsigned b = __ballot_sync(0xffffffffu, t1 > t0);
      if (t1 > t0) parts[n + __popc(b & ((1u << lane) - 1))] = 2 * c + (t0 == 0 ? 1 : 0);
      n += __popc(b);
    }
    if (lane == 0) n_parts = n;
  }
  __syncthreads();
  const int used = n_parts;
  if (rows <= kMergeRowBlocks || (rows <= kFewRows && used > kMergeThreads / 32)) {
    // A row for each block, or few rows of many parts: a block a row, a warp every eighth part, joined in shared
    // memory.  Against the form below a whole call takes 90 us instead of 94 with tiles of 4 rows in 19 parts, 19.1
    // instead of 20.3 with 4 rows in 4, but 292 instead of 287 with 24 rows in two or three.
    constexpr int kWarps = kMergeThreads / 32;
    for (int i = blockIdx.y; i < rows; i += gridDim.y) {
      const int h = i >= a.tpt * a.G ? 1 : 0, at_row = h * BM + i - h * a.tpt * a.G;
      auto load = [&](int p, float2& ml, float (&v)[E]) {
        const int64_t at = static_cast<int64_t>(parts[p]) * 2 * BM + at_row;
        ml = a.ml_part[at];
        if (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(a.o_part + at * D + E * lane);
        else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(a.o_part + at * D + E * lane);
      };
      float2 ml0 = make_float2(0.f, 0.f);   // of this warp's first part, in flight beside the maxima
      __align__(16) float v0[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v0[e] = 0.f;
      if (warp < used) load(warp, ml0, v0);
      float M = -CUDART_INF_F, l = 0.f;
      for (int p0 = 0; p0 < used; p0 += 32) {
        float2 ml = make_float2(-CUDART_INF_F, 0.f);
        if (p0 + lane < used) ml = a.ml_part[parts[p0 + lane] * 2 * BM + at_row];
        float mn = ml.y != 0.f ? ml.x : -CUDART_INF_F;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mn = fmaxf(M, mn);
        const float old = M == -CUDART_INF_F ? 0.f : ex2(M - mn);
        float ls = ml.y != 0.f ? ex2(ml.x - mn) * ml.y : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        M = mn;
        l = l * old + ls;
      }
      __align__(16) float acc[E];
      const float w0 = ml0.y != 0.f ? ex2(ml0.x - M) : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = w0 * v0[e];
#pragma unroll 4
      for (int p = warp + kWarps; p < used; p += kWarps) {
        float2 ml;
        __align__(16) float v[E];
        load(p, ml, v);
        const float w = ml.y != 0.f ? ex2(ml.x - M) : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += w * v[e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sums[warp][E * lane + e] = acc[e];
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < D) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x += sums[w][threadIdx.x];
        x *= l != 0.f ? 1.f / l : 0.f;
        const int tok = a.by_G.div(i), head = i - tok * a.G;
        const int64_t orow = static_cast<int64_t>(sg.q0 + sg.tok0 + tok) * a.Hq + sg.g * a.G + head;
        if (a.out_bf16) static_cast<__nv_bfloat16*>(a.o)[orow * D + threadIdx.x] = __float2bfloat16_rn(x);
        else static_cast<float*>(a.o)[orow * D + threadIdx.x] = x;
        if (a.lse && threadIdx.x == 0) a.lse[orow] = l != 0.f ? (M + log2f(l)) * kLn2 : -CUDART_INF_F;
      }
      __syncthreads();
    }
    return;
  }
  // two rows at a time, for the loads' latency
  constexpr int kRows = 2;
  for (int i0 = kRows * (blockIdx.y * (kMergeThreads / 32) + warp); i0 < rows; i0 += kRows * gridDim.y * (kMergeThreads / 32)) {
    int at_row[kRows];   // row of the partials
    float M[kRows], l[kRows];
    __align__(16) float acc[kRows][E];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int i = min(i0 + j, rows - 1), h = i >= a.tpt * a.G ? 1 : 0;
      at_row[j] = h * BM + i - h * a.tpt * a.G;
      M[j] = -CUDART_INF_F;
      l[j] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[j][e] = 0.f;
    }
    // lane p holds (m, l) of partial p, then its weight 2^(m - M); partials that saw nothing have weight 0
    for (int p0 = 0; p0 < used; p0 += 32) {
      float w[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        float2 ml = make_float2(-CUDART_INF_F, 0.f);
        if (p0 + lane < used) ml = a.ml_part[parts[p0 + lane] * 2 * BM + at_row[j]];
        float mn = ml.y != 0.f ? ml.x : -CUDART_INF_F;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mn = fmaxf(M[j], mn);
        w[j] = ml.y != 0.f ? ex2(ml.x - mn) : 0.f;
        const float old = M[j] == -CUDART_INF_F ? 0.f : ex2(M[j] - mn);
        float ls = w[j] * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        M[j] = mn;
        l[j] = l[j] * old + ls;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[j][e] *= old;
      }
      const int np = min(32, used - p0);
#pragma unroll 4
      for (int p = 0; p < np; ++p) {
        const float* src = a.o_part + static_cast<int64_t>(parts[p0 + p]) * 2 * BM * D + E * lane;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const float wp = __shfl_sync(0xffffffffu, w[j], p);
          __align__(16) float v[E];
          if (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src + at_row[j] * D);
          else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src + at_row[j] * D);
#pragma unroll
          for (int e = 0; e < E; ++e) acc[j][e] += wp * v[e];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (i0 + j >= rows) break;
      const int tok = a.by_G.div(i0 + j), head = i0 + j - tok * a.G;
      const float inv = l[j] != 0.f ? 1.f / l[j] : 0.f;
      const int64_t orow = static_cast<int64_t>(sg.q0 + sg.tok0 + tok) * a.Hq + sg.g * a.G + head;
      if (a.out_bf16) {
        __align__(8) uint32_t w[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2) w[e / 2] = f2_bf16x2(acc[j][e] * inv, acc[j][e + 1] * inv);
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.o) + orow * D + E * lane);
        if (E == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(w);
        else *dst = w[0];
      } else {
        float* dst = static_cast<float*>(a.o) + orow * D + E * lane;
#pragma unroll
        for (int e = 0; e < E; ++e) dst[e] = acc[j][e] * inv;
      }
      if (a.lse && lane == 0) a.lse[orow] = l[j] != 0.f ? (M[j] + log2f(l[j])) * kLn2 : -CUDART_INF_F;
    }
  }
}

template <int D, class F>
ra_status launch_chunk(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const ChunkArgs& a,
                       cudaStream_t stream) {
  const size_t smem = sizeof(ChunkSmem<D, F>) + 1024;
  RA_CUDA_TRY(cudaFuncSetAttribute(chunk_attn_kernel<D, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(smem)));
  chunk_attn_kernel<D, F><<<kCtas, kChunkThreads, smem, stream>>>(mq, mk, mv, a);
  RA_LAUNCH_CHECK("chunk_attn_kernel");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas, kMergeRowBlocks);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  RA_CUDA_TRY(cudaLaunchKernelEx(&cfg, chunk_merge_kernel<D, F>, a));
  return RA_OK;
}

inline int64_t part_floats(int d) { return static_cast<int64_t>(2 * kCtas) * 2 * BM * d; }

template <class F>
size_t chunk_workspace(int d) { return static_cast<size_t>(part_floats(d) * 4 + part_floats(1) * 8 + kCtas * sizeof(Join<F>)); }

// What all forms share of the arguments.
inline void set_chunk_args(ChunkArgs& a, const int32_t* query_start_loc, const int32_t* ctx_lens, int64_t T, int32_t R,
                           int32_t Hq, int32_t Hkv, int32_t d, float scale, void* o, ra_dtype out_dt, float* lse,
                           void* workspace) {
  a.qsl = query_start_loc; a.ctx = ctx_lens;
  a.T = T; a.R = R; a.Hq = Hq; a.G = Hq / Hkv; a.causal = 1; a.out_bf16 = out_dt == RA_BF16;
  a.tpt = BM / a.G;
  a.by_G = fast_div(a.G);
  a.by_tpi = fast_div(2 * a.tpt);
  a.rates = rates_of(d);
  a.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(d))) * 1.4426950408889634f;
  a.o = o; a.lse = lse;
  a.o_part = static_cast<float*>(workspace);
  a.ml_part = reinterpret_cast<float2*>(a.o_part + part_floats(d));
  a.join = a.ml_part + part_floats(1);
  a.wait_limit = ra::wait_limit();
  a.drain_limit = std::max<long long>(a.wait_limit, 1ll << 22);
  a.window = 1 << 30;
  a.n_sink = 0;
}

// The maps of Q and of the paged cache, and the launch.
template <int D, class F>
ra_status launch_chunk_paged(const void* q, const void* k, const void* v, const ChunkArgs& a, cudaStream_t stream) {
  CUtensorMap mq, mk, mv;
  ra_status st;
  const int64_t blocks = a.c.W * a.c.num_blocks * a.c.Hkv;
  if ((st = box_map(&mq, q, D, a.Hq, a.T, a.G, a.tpt)) != RA_OK) return st;
  if ((st = box_map(&mk, k, D, a.c.bs, blocks, 1 << a.lu, 1)) != RA_OK) return st;
  if ((st = box_map(&mv, v, D, a.c.bs, blocks, 1 << a.lu, 1)) != RA_OK) return st;
  return launch_chunk<D, F>(mq, mk, mv, a, stream);
}

// Host checks of the paged forms; `need`: bytes of workspace.
inline ra_status check_chunk_paged(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                   const int32_t* query_start_loc, const int32_t* ctx_lens, int64_t T, int32_t R, int32_t Hq,
                                   int32_t Hkv, int32_t d, int32_t block_size, int32_t interleave, int32_t pcp, int32_t dcp,
                                   int32_t max_vblocks, int64_t num_blocks, const void* o, ra_dtype out_dt, const void* lse,
                                   const void* workspace, size_t ws_bytes, size_t need) {
  const ra_status st = check_paged(R, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks);
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
  RA_REQUIRE(ws_bytes >= need, "workspace too small (%zu < %zu bytes)", ws_bytes, need);
  const uint64_t rows = static_cast<uint64_t>(T) * Hq;
  const uint64_t cache = static_cast<uint64_t>(pcp) * dcp * num_blocks * Hkv * block_size * d * 2;
  return ra::check_workspace_apart(ra::Span{workspace, need}, ra::Span{q, rows * d * 2}, ra::Span{k_cache, cache},
                                   ra::Span{v_cache, cache}, ra::Span{block_table, static_cast<uint64_t>(R) * max_vblocks * 4},
                                   ra::Span{query_start_loc, (R + 1ull) * 4}, ra::Span{ctx_lens, R * 4ull},
                                   ra::Span{o, rows * d * (out_dt == RA_BF16 ? 2 : 4)}, ra::Span{lse, rows * 4});
}

}  // namespace
