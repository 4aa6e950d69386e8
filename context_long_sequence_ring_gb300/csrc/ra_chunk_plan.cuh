// The division of the chunk attention's work into equal parts: its arithmetic,
// for the device and, in the tests, for the host.
//
// The keys that all row tiles ("items", single or in pairs) of all heads and
// requests meet lie on one axis of cost, which is cut into equal parts, one per
// CTA.  The cost of an item is in keys times what a key costs.  Measured over the
// CTAs of one call at D = 128: a pair tile 1.59 us (tensor core), a split tile 1.24 (HBM),
// and prologue and epilogue of an item as many keys as `over_pair` and `over_split`.
// At D = 64 the numbers are those with the least time over batches of prompts,
// single tokens and both (split tiles at 6 tenths of a pair tile: 24 requests of both kinds
// 102 us, at 5 or 7 tenths 105).
//
// Sums are 64-bit; positions on the axis are 32-bit, in units of 2^shift that are
// chosen from the sum of this call (below 2^30: shift 0).  Only sums are shifted, never what is
// multiplied before: a slope that is shifted by itself can become 0, and a prompt's last row
// tiles then count as little as its first (the longest part of 65536 tokens, 64/8 heads, was
// 1.95 times the mean).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define RA_HD __host__ __device__ __forceinline__
#else
#define RA_HD inline
#endif

namespace {

constexpr int kCtas = 152;         // parts of the work, one CTA per SM of a GB300
constexpr int kPairCost = 10;      // cost of a key in a pair tile

struct Rates {
  int f_split, over_pair, over_split;
};

RA_HD Rates rates_of(int d) { return d == 128 ? Rates{8, 470, 255} : Rates{6, 460, 270}; }

RA_HD float quotient(float a, float b) {
#ifdef __CUDA_ARCH__
  return __fdividef(a, b);
#else
  return a / b;
#endif
}

// The items of one head of a request.
struct Items {
  uint64_t base;                  // cost of item k: base + slope * (k + 1), of which `start` for its start and end
  uint32_t slope, start;
  int items;
  bool pair;
  // cost of items 0 .. k-1
  RA_HD uint64_t upto(int k) const {
    return static_cast<uint64_t>(k) * base + slope * (static_cast<uint64_t>(k) * (k + 1) / 2);
  }
  // n queries from position pos0 on over L tokens, tpt of them to a row tile; n_items: row tiles (pairs of them)
  RA_HD void set(const Rates& rt, int n, int n_items, int tpt, long long pos0, int L, bool causal) {
    items = n_items;
    pair = n > tpt;
    const long long before = pos0 < 0 ? 0 : (pos0 < L ? pos0 : L);
    const int f = pair ? kPairCost : rt.f_split, over = pair ? rt.over_pair : rt.over_split;
    base = static_cast<uint64_t>(over + (causal ? before : L)) * f;
    start = over * f;
    slope = causal ? (pair ? 2 : 1) * tpt * f : 0;
  }
};

// The items of one head of a request whose queries see a window and some first tokens: an item's keys grow with k
// up to those of a whole window.
struct WindowItems {
  uint64_t base;                  // cost of item k: base + slope * min(k + 1, full)
  uint32_t slope, start;
  int items, full;
  bool pair;
  RA_HD uint64_t upto(int k) const {
    const uint64_t m = k < full ? k : full;
    return static_cast<uint64_t>(k) * base + slope * (m * (m + 1) / 2 + static_cast<uint64_t>(k - m) * full);
  }
  RA_HD void set(const Rates& rt, int n, int n_items, int tpt, long long pos0, int L, int window, int n_sink) {
    items = n_items;
    pair = n > tpt;
    const int f = pair ? kPairCost : rt.f_split, over = pair ? rt.over_pair : rt.over_split, tpi = (pair ? 2 : 1) * tpt;
    // half a tile past either end of the window, and the units of first tokens
    const long long most = static_cast<long long>(window) + tpi + 128 + (n_sink + 31ll) / 32 * 32;
    const long long cap = most < L ? most : L, before = pos0 < 0 ? 0 : (pos0 < cap ? pos0 : cap);
    const long long steps = (cap - before) / tpi;
    full = static_cast<int>(steps < n_items ? steps : n_items);
    if (full < 1) full = 1;
    base = static_cast<uint64_t>(over + before) * f;
    start = over * f;
    slope = tpi * f;
  }
};

// Part c of the work is [lo(c), lo(c + 1)), empty from the first c with lo(c) = total on.  Where an equal
// cut leaves few items to a part, and cutting each item into pieces of its own costs less than the second item
// that a part would take up, lengths are counted in such pieces (piece > 0: the cost of one; share is 1 then).
struct Plan {
  uint32_t total, share;
  int shift;
  float piece;
  RA_HD uint32_t lo(int c) const {
    const uint32_t x = share * c;
    return x < total ? x : total;
  }
  // Item k, and items 0 .. k-1 of a head: at least 1 each, so that none is lost.
  template <class I>
  RA_HD uint32_t cost(const I& q, int k) const {
    const uint32_t c = static_cast<uint32_t>((q.upto(k + 1) >> shift) - (q.upto(k) >> shift)) + 1;
    return piece > 0.f ? static_cast<uint32_t>(quotient(static_cast<float>(c), piece)) + 1 : c;
  }
  template <class I>
  RA_HD uint32_t prefix(const I& q, int k) const {
    if (piece <= 0.f) return static_cast<uint32_t>(q.upto(k) >> shift) + k;
    uint32_t sum = 0;
#pragma unroll 1
    for (int i = 0; i < k; ++i) sum += cost(q, i);
    return sum;
  }
  template <class I>
  RA_HD uint32_t over(const I& q) const { return piece > 0.f ? 0 : q.start >> shift; }

  // The steps of a plan: the unit, from the sum of upto() over all heads; the equal cut, from the sum of
  // prefix() in that unit; whether to try pieces; and their number, in which case they are taken or not.
  RA_HD void scale(uint64_t sum) {
    piece = 0.f;
    shift = 0;
    while ((sum >> shift) >> 30) ++shift;
  }
  RA_HD void divide(uint32_t sum, const Rates& rt) {
    total = sum;
    const uint32_t least = (256u * rt.f_split) >> shift, even = (sum + kCtas - 1) / kCtas;
    share = even > least ? even : least;
  }
  RA_HD bool try_pieces(uint32_t items, const Rates& rt) {
    if (items > kCtas / 2) return false;
    // pieces of at most total / (kCtas - items): at most kCtas of them, since an item has one incomplete piece
    const float even = static_cast<float>(share), least = quotient(1.001f * static_cast<float>(total), static_cast<float>(kCtas - items));
    const float p = even > least ? even : least;
    if (!(p < static_cast<float>(share + ((rt.f_split * rt.over_split) >> shift)))) return false;
    piece = p;
    return true;
  }
  RA_HD void use_pieces(uint32_t number) {
    if (number <= kCtas) {
      total = number;
      share = 1;
    } else {
      piece = 0.f;
    }
  }
};

// Tiles [t0, t1) of an item of nt tiles and cost [at, at + cost) that part [lo, hi) takes.  The first `over` of the
// cost stand for the start and end of a segment: a part pays for each item that begins in it (and all parts alike for
// the one they begin inside of).  Spread over the item instead, a batch of short items (12 requests, heads of
// 64) took 46.3 us instead of 43.6.  Fractions are taken in fp32: a boundary gives the same tile to both of its
// sides, whatever its rounding.
RA_HD int cut_at(uint32_t off, uint32_t over, uint32_t cost, int nt) {
  if (off <= over) return 0;
  const int t = static_cast<int>(quotient(static_cast<float>(off - over), static_cast<float>(cost - over)) * static_cast<float>(nt));
  return t < nt ? t : nt;
}
RA_HD void cut(uint32_t lo, uint32_t hi, uint32_t at, uint32_t over, uint32_t cost, int nt, int& t0, int& t1) {
  t0 = lo <= at ? 0 : cut_at(lo - at, over, cost, nt);
  t1 = hi >= at + cost ? nt : cut_at(hi - at, over, cost, nt);
}

}  // namespace
