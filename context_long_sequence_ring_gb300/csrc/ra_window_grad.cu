// The gradient of attention with a sliding window and first tokens that stay
// visible, on packed sequences.
//
// Mathematics.  With P = e^{scale q.k - lse} on the visible pairs and delta = sum dO O of
// each row and head,
//   dV = P^T dO,  dS = P (dO V^T - delta),  dQ = scale dS K,  dK = scale dS^T Q.
//
// Two kernels of seven products in all in place of one of five: dQ is summed over keys and dK, dV over queries, and
// one kernel for both would add its dQ tiles to memory in an order of its own each time; here every sum stays
// in tensor memory and the same call gives the same bits.
//
//   prepare   -lse log2 e and -delta of each row, head by head, and the lists of tiles.
//   dQ        a CTA takes tiles of 128 rows, floor(128/G) tokens with the G heads of a K/V head, past the keys that
//             they see: S = Q K^T and dP = dO V^T in tensor memory, dS (bf16) over S, dQ += dS K.
//   dK, dV    a CTA takes tiles of 128 keys of a K/V head past the (query tile, head) pairs that see them, transposed:
//             S^T = K Q^T, dP^T = V dO^T; P^T and dS^T (bf16) over them are operands from tensor memory of
//             dV += P^T dO and dK += dS^T Q.
//   join      sums the parts of key tiles that several CTAs share.
// 16 warps of softmax, a thread holding 32 columns of a row of a score tile: tensor memory has room for one tile of
// each kind only, so that the chain of a tile (scores, exponentials, next product) sets the pace, and
// 8 warps with 64 columns each took 1.5 times as long for it.  A whole warp issues the products (in a branch of one thread
// dQ took 713 us instead of 529, dK and dV 835 instead of 622: operands moved to uniform registers one by one), one the
// loads, and one zeroes rows past a sequence's end (0 * NaN).
//
// Bound by the tensor core where items are long, and by their starts and ends where a window makes them short.  Measured over
// 16384 tokens, 32/8 heads, dQ / dK and dV in us: D = 128, window 512 227 / 214, 2048 510 / 597, none 1820 / 2400 (1.81 and
// 1.83 PFLOP/s executed); D = 64 177 / 176, 408 / 485, 1421 / 1875.  prepare reads o and dO once, 5.4 TB/s; join 16 us.
//
// Rounding.  P and dS are rounded to bf16, the type of the other operand.  delta is formed from an o that has been rounded,
// whose error all keys of a row share.  Where P sums to 1 over a row, dS sums to 0, so that the dQ kernel's row sums of dS in
// fp32 are that error, and dK gets the delta without it.  Where lse and o are those of more keys than these, P sums to
// less, dS need not sum to 0, and delta stays as it is: a row has all its keys here if its P sum to 1 as closely as
// fp32 tells (sums_to_one) and what its delta would change by is no more than the rounding of o can make, 2^-8 sum |dO O|
// (random q, k, v and dO: up to 0.41 of that).  So other keys' weight that is not told from rounding has no more effect
// than rounding.  In dQ itself the error counts where a row sees few keys (2: 0.0033 of dQ, 3: 0.0026, 8: 0.0020);
// where all of them are in one tile, delta is summed from P and dP before dS is formed, under the same condition.
//
// Work of dK, dV.  Tiles in rounds of one whole tile per CTA, neighbours at the same time, so that the queries they share
// are in L2; the last one or two rounds, and the tiles of first tokens that all later queries see, are laid on one axis
// of cost that is cut into parts which even out what each CTA has had, with at most two shared tiles to a part.
#include <algorithm>

#include "ra_window.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_window_grad)

namespace {

constexpr int kGradCtas = 152;         // one CTA per SM of a GB300
constexpr int kGroups = 4;             // softmax warpgroups, 32 columns each
constexpr int kSoftmax = 128 * kGroups;
constexpr int kGradThreads = 128 + kSoftmax;
constexpr float kUnit = 1.f / 32768.f; // of row sums of P between warps: only whether they sum to 1 is asked
// Row tiles of so many key tiles or fewer have dS in two parts: where a row sees 16 keys, dQ is then off by 0.0018 instead of
// 0.0025 (its own rounding is 0.0017); a window of 128 over 16384 tokens takes 398 us instead of 378.
constexpr int kFewTiles = 2;
constexpr int kPlanThreads = 1024;
constexpr int kOver = 4;               // start and end of a key tile, in query tiles

struct Tile {
  int q0, n, k, pad;                   // first row and length of the sequence, number of the tile in it
};

struct Plan {
  int row_tiles, key_tiles;            // of a head
  int plain;                           // key tiles that only a window sees: the first of the list
  int whole;                           // items in whole rounds
  int64_t lo[kGradCtas + 1];           // parts of the rest, in cost
  int start[kGradCtas];                // key tile in which part c starts
};

// A key tile that several parts share, as its first part leaves it.
struct Shared {
  int used, q0, n, k, g, its;
  int64_t at;                          // on the axis of cost
};

struct GradArgs {
  const int32_t* qsl;
  int64_t T;
  int R, Hq, Hkv, G, window, n_sink, tpt, out_bf16;
  float scale, scale_log2;
  const __nv_bfloat16 *o, *d_o;
  const float* lse;
  void *dq, *dk, *dv;
  int64_t dq_rs, dk_rs, dv_rs;
  float *neg_lse, *neg_delta;          // [Hq][T]
  float* slack;                        // [Hq][T] what the rounding of o can change delta by
  Tile *rows, *keys;
  int64_t* base;                       // [key tiles] place of a tile's first head on the axis of cost
  Plan* plan;
  Shared* shared;                      // [kGradCtas]
  float* parts;                        // [2 * kGradCtas][2][D / 4][128][4]
  FastDiv by_G, by_Hkv;
  long long wait_limit, drain_limit;
};

// ------------------------------------------------------------------ geometry
// Query tiles [k, k + count) of 128 rows see key tile k of a sequence of n tokens.
__device__ __forceinline__ int query_tiles(const GradArgs& a, int n, int k) {
  const int all = (n + BM - 1) / BM - k;
  if (k * BM < a.n_sink) return all;
  const int64_t far = (static_cast<int64_t>(a.window) + BM - 2) / BM + 1;   // (128k + 127 + window - 1) / 128 - k + 1
  return all < far ? all : static_cast<int>(far);
}
// Tiles of first tokens that are longer than a window makes them: a prefix of a sequence's key tiles.
__device__ __forceinline__ int long_tiles(const GradArgs& a, int n) {
  const int64_t sinks = (static_cast<int64_t>(a.n_sink) + BM - 1) / BM;
  const int64_t more = (n + BM - 1) / BM - ((static_cast<int64_t>(a.window) + BM - 2) / BM + 1);
  const int64_t x = sinks < more ? sinks : more;
  return x < 0 ? 0 : static_cast<int>(x);
}
__device__ __forceinline__ int64_t cost_of(const GradArgs& a, int n, int k) {
  return static_cast<int64_t>(query_tiles(a, n, k)) * a.G + kOver;
}

// ------------------------------------------------------------------ prepare
// Inclusive prefix sum (or maximum, of values that are not negative) over the block.
template <bool MAX = false, class X>
__device__ __forceinline__ X block_scan(X x, X* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const X y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = MAX ? max(x, y) : x + y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  // the warps before this one, each lane one of them
  X before = lane < warp ? warps[lane] : X(0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const X y = __shfl_xor_sync(0xffffffffu, before, o);
    before = MAX ? max(before, y) : before + y;
  }
  return MAX ? max(x, before) : x + before;
}

// Sequence `base + thread`: its rows [q0, q0 + n); n = 0 where its range is bad or starts before an earlier one ends, so
// that all tiles together are no more than the lists hold.  `ended`: where those before `base` end, brought up to date.
__device__ __forceinline__ void load_seq(const GradArgs& a, int base, int& q0, int& n, int& ended, int* sums, int* shared_end) {
  q0 = n = 0;
  const int i = base + threadIdx.x;
  if (i < a.R) query_range(load_lens(a.qsl, a.qsl, i, a.R), a.T, q0, n, 900);
  const int end = max(ended, block_scan<true>(q0 + n, sums));
  int before = __shfl_up_sync(0xffffffffu, end, 1);
  __syncthreads();
  if ((threadIdx.x & 31) == 31) shared_end[threadIdx.x >> 5] = end;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) before = threadIdx.x == 0 ? ended : shared_end[(threadIdx.x >> 5) - 1];
  if (n > 0 && q0 < before) {
    ra_record_error(RA_ERR_DEVICE_BOUNDS, 901);
    n = 0;
  }
  ended = shared_end[kPlanThreads / 32 - 1];
}

// The lists of tiles and the division of the key tiles, by one block.
__device__ void make_lists(const GradArgs& a) {
  __shared__ int seq[kPlanThreads][2];                              // q0, n
  __shared__ int ends[3][kPlanThreads];                             // row tiles, plain and long key tiles up to request i
  __shared__ int sums[32];
  __shared__ int64_t sums64[32];
  __shared__ int64_t total, had_total, lo[kGradCtas + 1];
  const int tid = threadIdx.x;
  // plain key tiles of all sequences, so that the long ones can follow them in the list
  int plain = 0, ended = 0, q0, n;
  for (int base = 0; base < a.R; base += kPlanThreads) {
    load_seq(a, base, q0, n, ended, sums, ends[0]);
    plain += (n + BM - 1) / BM - long_tiles(a, n);
  }
  plain = block_scan(plain, sums);
  __syncthreads();
  if (tid == kPlanThreads - 1) sums[0] = plain;
  __syncthreads();
  plain = sums[0];
  int at[3] = {0, 0, plain};
  ended = 0;
  for (int base = 0; base < a.R; base += kPlanThreads) {
    if (a.R > kPlanThreads) load_seq(a, base, q0, n, ended, sums, &seq[0][0]);   // else they are in hand
    const int more = long_tiles(a, n);
    const int mine[3] = {(n + a.tpt - 1) / a.tpt, (n + BM - 1) / BM - more, more};
    __syncthreads();
    seq[tid][0] = q0;
    seq[tid][1] = n;
#pragma unroll
    for (int l = 0; l < 3; ++l) ends[l][tid] = block_scan(mine[l], sums);
    __syncthreads();
#pragma unroll
    for (int l = 0; l < 3; ++l) {
      const int count = ends[l][kPlanThreads - 1];
      for (int i = tid; i < count; i += kPlanThreads) {
        int x = 0, y = kPlanThreads - 1;                            // first request that ends past i
        while (x < y) {
          const int mid = (x + y) >> 1;
          if (ends[l][mid] > i) y = mid; else x = mid + 1;
        }
        int k = i - (x ? ends[l][x - 1] : 0);
        if (l == 1) k += long_tiles(a, seq[x][1]);
        (l == 0 ? a.rows : a.keys)[at[l] + i] = Tile{seq[x][0], seq[x][1], k, 0};
      }
      at[l] += count;
    }
  }
  __syncthreads();
  const int key_tiles = at[2];
  // whole rounds of plain items, and at least one round (as far as there is one) for the rest
  const int64_t items = static_cast<int64_t>(plain) * a.Hkv;
  const int rounds = items >= 2 * kGradCtas ? static_cast<int>(items / kGradCtas) - 1 : 0;
  const int whole = rounds * kGradCtas;
  int64_t had = 0;                                                  // cost of CTA tid's whole items
  if (tid < kGradCtas)
    for (int m = 0; m < rounds; ++m) {
      const Tile t = a.keys[(m * kGradCtas + tid) / a.Hkv];
      had += cost_of(a, t.n, t.k);
    }
  // places of the rest
  const int tile0 = whole / a.Hkv, g0 = whole - tile0 * a.Hkv;
  int64_t before = 0;
  for (int base = tile0; base < key_tiles; base += kPlanThreads) {
    const int i = base + tid;
    int64_t c = 0;
    if (i < key_tiles) {
      const Tile t = a.keys[i];
      c = cost_of(a, t.n, t.k);
      if (i == tile0) before = -g0 * c;
    }
    if (base == tile0) {
      __syncthreads();
      if (tid == 0) total = before;
      __syncthreads();
      before = total;
    }
    const int64_t s = block_scan(c * a.Hkv, sums64);
    if (i < key_tiles) a.base[i] = before + s - c * a.Hkv;
    __syncthreads();
    if (tid == kPlanThreads - 1) total = before + s;
    __syncthreads();
    before = total;
  }
  if (tid == 0 && tile0 >= key_tiles) total = 0;
  // each part's share: what is left of the mean over all work, scaled to the whole of the rest
  const int64_t all_had = block_scan(tid < kGradCtas ? had : int64_t(0), sums64);
  __syncthreads();
  if (tid == kPlanThreads - 1) had_total = all_had;
  __syncthreads();
  const int64_t rest = total;
  const float mean = static_cast<float>(had_total + rest) / kGradCtas;
  const int64_t want = tid < kGradCtas ? static_cast<int64_t>(fmaxf(0.f, mean - static_cast<float>(had))) + 1 : 0;
  const int64_t upto = block_scan(want, sums64);
  __syncthreads();
  if (tid == kGradCtas - 1) had_total = upto;
  __syncthreads();
  const int64_t wanted = had_total;
  if (tid < kGradCtas) {
    const int64_t x = static_cast<int64_t>(static_cast<double>(upto) / static_cast<double>(wanted) * static_cast<double>(rest));
    lo[tid + 1] = tid == kGradCtas - 1 ? rest : (x < rest ? x : rest);
  }
  if (tid == 0) lo[0] = 0;
  __syncthreads();
  if (tid <= kGradCtas) a.plan->lo[tid] = lo[tid];
  for (int i = tile0 + tid; i < key_tiles; i += kPlanThreads) {
    const Tile t = a.keys[i];
    const int64_t from = a.base[i], to = from + cost_of(a, t.n, t.k) * a.Hkv;
    int x = 0, y = kGradCtas;                                       // first part that starts at `from` or later
    while (x < y) {
      const int mid = (x + y) >> 1;
      if (lo[mid] >= from) y = mid; else x = mid + 1;
    }
    for (; x < kGradCtas && lo[x] < to; ++x) a.plan->start[x] = i;
  }
  if (tid == 0) {
    a.plan->row_tiles = at[0];
    a.plan->key_tiles = key_tiles;
    a.plan->plain = plain;
    a.plan->whole = whole;
  }
}

// Block 0: the lists.  The others: a warp takes 8 tokens of a head, D/8 lanes a row (8 and not 32, so that the last of a
// warp's tasks is short).
template <int D>
__global__ void __launch_bounds__(kPlanThreads) grad_prepare_kernel(const __grid_constant__ GradArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) {
    make_lists(a);
    return;
  }
  constexpr int LANES = D / 8;                                      // of a row, 16 bytes each
  constexpr int ROWS = 32 / LANES;
  const int lane = threadIdx.x & 31;
  constexpr int TASK = 8;
  const int64_t groups = (a.T + TASK - 1) / TASK;
  const int64_t w0 = static_cast<int64_t>(blockIdx.x - 1) * (kPlanThreads / 32) + (threadIdx.x >> 5);
  for (int64_t w = w0; w < groups * a.Hq; w += static_cast<int64_t>(gridDim.x - 1) * (kPlanThreads / 32)) {
    const int64_t t0 = w / a.Hq * TASK;
    const int h = static_cast<int>(w % a.Hq);
    const int64_t mine_t = t0 + (lane % TASK);
    const float lse = mine_t < a.T ? a.lse[mine_t * a.Hq + h] : 0.f;
    uint4 x[TASK / ROWS], y[TASK / ROWS];
#pragma unroll
    for (int i = 0; i < TASK / ROWS; ++i) {
      const int64_t t = t0 + i * ROWS + lane / LANES, at = (t * a.Hq + h) * D + (lane % LANES) * 8;
      x[i] = t < a.T ? *reinterpret_cast<const uint4*>(a.o + at) : make_uint4(0, 0, 0, 0);
      y[i] = t < a.T ? *reinterpret_cast<const uint4*>(a.d_o + at) : make_uint4(0, 0, 0, 0);
    }
    float mine = 0.f, size = 0.f;
#pragma unroll
    for (int i = 0; i < TASK / ROWS; ++i) {
      const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
      float s = 0.f, m = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = __uint_as_float(xs[e] << 16) * __uint_as_float(ys[e] << 16);
        const float v = __uint_as_float(xs[e] & 0xffff0000u) * __uint_as_float(ys[e] & 0xffff0000u);
        s += u + v;
        m += fabsf(u) + fabsf(v);
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        m += __shfl_xor_sync(0xffffffffu, m, o);
      }
      // lane i * ROWS + r keeps the row of the r-th part of the warp
      const int from = (lane - i * ROWS) * LANES & 31;
      const float got = __shfl_sync(0xffffffffu, s, from), got_m = __shfl_sync(0xffffffffu, m, from);
      if (lane / ROWS == i) {
        mine = got;
        size = got_m;
      }
    }
    if (lane < TASK && mine_t < a.T) {
      // a row that sees nothing has no weight
      a.neg_lse[h * a.T + mine_t] = lse == -CUDART_INF_F ? -CUDART_INF_F : -lse * 1.4426950408889634f;
      a.neg_delta[h * a.T + mine_t] = -mine;
      a.slack[h * a.T + mine_t] = size * (1.f / 256);
    }
  }
}

// ------------------------------------------------------------------ pieces of both kernels
// One arrival for a warp, whose lanes have all done what it stands for.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// p = 2^(s * scale + nl) of a pair of columns.
__device__ __forceinline__ void exp_pair(uint32_t s0, uint32_t s1, uint64_t sc2, uint64_t nl2, float& p0, float& p1) {
  float t0, t1;
  f2unpack(ffma2(f2pack(__uint_as_float(s0), __uint_as_float(s1)), sc2, nl2), t0, t1);
  p0 = ex2(t0);
  p1 = ex2(t1);
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Whether a row's P are all its weights, as closely as fp32 tells: sums of a few thousand terms in fp32, the units in
// which parts of the sum pass between warps (3 * 2^-16), and -lse log2 e, its own rounding and that of scores as large.
__device__ __forceinline__ bool sums_to_one(float p_sum, float neg_lse) {
  return fabsf(p_sum - 1.f) < 1.f / 8192 + fabsf(neg_lse) * (1.f / (1 << 21));
}

// 32 accumulator columns of a row per lane to memory, times f; at < 0: not stored.
__device__ __forceinline__ void store_cols(void* out, bool bf, int64_t at, const uint32_t (&x)[32], float f) {
  if (bf) {
    store_rows_bf16(static_cast<__nv_bfloat16*>(out), at, x, f);
  } else if (at >= 0) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      dst[i] = make_float4(__uint_as_float(x[4 * i]) * f, __uint_as_float(x[4 * i + 1]) * f, __uint_as_float(x[4 * i + 2]) * f,
                           __uint_as_float(x[4 * i + 3]) * f);
  }
}

// ------------------------------------------------------------------ dQ
// Keys of a row tile: units of 32, unit j at position 32 j, `skip` further from unit `first` on (as in the forward kernel).
struct RowItem {
  int q0, n, g, tok0, first, skip, nt, dirty;
  int low0, clean;                     // tiles [low0, clean) are seen whole by all rows
  __device__ __forceinline__ void set(const GradArgs& a, const Tile& t, int head) {
    q0 = t.q0; n = t.n; g = head;
    tok0 = t.k * a.tpt;
    const int last = min(n, tok0 + a.tpt) - 1;                      // last position
    const int low = max(0, tok0 + 1 - a.window), low_last = max(0, last + 1 - a.window);
    const int sinks = (min(a.n_sink, last + 1) + 31) >> 5;
    first = skip = 0;
    if (low >= 32 * sinks) {
      first = sinks;
      skip = low - 32 * sinks;
    }
    nt = (last + 1 - skip + BN - 1) / BN;
    dirty = (n - skip) / BN;                                        // first tile with rows past the sequence
    clean = (tok0 + 1 - skip) / BN;
    low0 = (max(low_last - skip, 0) + BN - 1) / BN;
  }
};

template <int D>
struct __align__(1024) RowSmem {
  static constexpr int KS = D == 128 ? 3 : 6, VS = D == 128 ? 2 : 4;
  uint8_t q[BM * D * 2], d_o[BM * D * 2], k[KS][BN * D * 2], v[VS][BN * D * 2];
  uint64_t q_full, q_empty, k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], k_dirty[KS], k_clean[KS];
  uint64_t s_full[2], dp_full, ds_full[2], acc_full, acc_empty, sums_full, sums_free, all_read, drain;
  float sums[kGroups - 1][BM];         // of dS
  uint16_t p_sums[kGroups - 1][BM];    // of P, in units of kUnit
  uint32_t tmem_base;
  int abort_flag;
};

// Tensor memory: dQ, then two score tiles (dS of each 32 columns over the first half of them, what its rounding leaves
// over the second), then dP.
template <int D>
__global__ void __launch_bounds__(kGradThreads, 1)
    grad_q_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                  const __grid_constant__ GradArgs a) {
  using Smem = RowSmem<D>;
  constexpr int SLABS = D / 64, KS = Smem::KS, VS = Smem::VS;
  constexpr uint32_t kTileBytes = BM * D * 2;
  constexpr uint32_t kColS = D, kColP = D + 2 * BN;
  static_assert(kColP + BN <= kTmemCols);
  constexpr uint32_t kIdescS = idesc_bf16_f32(BM, BN, 0, 0), kIdescQ = idesc_bf16_f32(BM, D, 0, 1);

  extern __shared__ __align__(1024) uint8_t smem_grad[];   // no room to align it by hand
  Smem& sm = *reinterpret_cast<Smem*>(smem_grad);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const long long lim = a.wait_limit;
  if (smem_u32(smem_grad) & 1023) {
    if (threadIdx.x == 0) ra_record_error(RA_ERR_CUDA, 904);
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sm.q_full), 1);
    mbar_init(smem_u32(&sm.q_empty), 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(smem_u32(&sm.k_full[s]), 1);
      mbar_init(smem_u32(&sm.k_empty[s]), 1);
      mbar_init(smem_u32(&sm.k_dirty[s]), 1);
      mbar_init(smem_u32(&sm.k_clean[s]), 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(smem_u32(&sm.v_full[s]), 1);
      mbar_init(smem_u32(&sm.v_empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sm.s_full[b]), 1);
      mbar_init(smem_u32(&sm.ds_full[b]), kSoftmax / 32);
    }
    mbar_init(smem_u32(&sm.dp_full), 1);
    mbar_init(smem_u32(&sm.sums_full), kSoftmax / 32 - 4);
    mbar_init(smem_u32(&sm.sums_free), 4);
    mbar_init(smem_u32(&sm.all_read), kSoftmax / 32);
    mbar_init(smem_u32(&sm.acc_full), 1);
    mbar_init(smem_u32(&sm.acc_empty), kSoftmax / 32);
    mbar_init(smem_u32(&sm.drain), 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Items in rounds, every other one backwards: where they get longer along a sequence the CTAs' sums stay even.
  const int items = a.plan->row_tiles * a.Hkv;
  auto item_of = [&](int m) {
    const int64_t i = static_cast<int64_t>(m) * kGradCtas + (m & 1 ? kGradCtas - 1 - blockIdx.x : blockIdx.x);
    return i < items ? static_cast<int>(i) : -1;
  };
  const int rounds = (items + kGradCtas - 1) / kGradCtas;
  auto get = [&](int m, RowItem& it) {
    const int i = item_of(m);
    if (i < 0) return false;
    int g;
    const int t = a.by_Hkv.div(i, g);
    it.set(a, a.rows[t], g);
    return true;
  };
  RowItem it;

  if (warp == 0) {
    // ============================================================ loads: lane = (K or V, slab, unit)
    const int unit = lane & 3, slab = (lane >> 2) & (SLABS - 1), half = 4 * SLABS;
    const bool is_v = lane >= half, used = lane < 2 * half;
    Ring<KS> kr;
    Ring<VS> vr;
    uint32_t k_n = 0, v_n = 0, q_n = 0;
    bool ok = true;
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmO);
    }
    for (int m = 0; m < rounds && ok; ++m) {
      if (!get(m, it)) continue;
      if (!(ok = warp_wait(smem_u32(&sm.q_empty), (q_n & 1) ^ 1, abort_flag, lim, 910))) break;
      ++q_n;
      if (lane == 0) {
        const uint32_t qb = smem_u32(&sm.q_full);
        mbar_arrive_expect_tx(qb, 2 * SLABS * a.tpt * a.G * 128);
        for (int s = 0; s < SLABS; ++s) {
          tma_load_3d(smem_u32(sm.q + s * BM * 128), &tmQ, qb, 64 * s, it.g * a.G, it.q0 + it.tok0);
          tma_load_3d(smem_u32(sm.d_o + s * BM * 128), &tmO, qb, 64 * s, it.g * a.G, it.q0 + it.tok0);
        }
      }
      __syncwarp();
      for (int j = 0; j < it.nt; ++j) {
        if (!(ok = warp_wait(smem_u32(&sm.k_empty[kr.st]), kr.ph ^ 1, abort_flag, lim, 911))) break;
        if (!(ok = warp_wait(smem_u32(&sm.v_empty[vr.st]), vr.ph ^ 1, abort_flag, lim, 912))) break;
        const uint32_t kb = smem_u32(&sm.k_full[kr.st]), vb = smem_u32(&sm.v_full[vr.st]);
        if (lane == 0) {
          mbar_arrive_expect_tx(kb, kTileBytes);
          mbar_arrive_expect_tx(vb, kTileBytes);
          if (j >= it.dirty) mbar_arrive(smem_u32(&sm.k_dirty[kr.st]));
        }
        __syncwarp();
        if (used) {
          const int u = 4 * j + unit, row = it.q0 + 32 * u + (u < it.first ? 0 : it.skip);
          tma_load_3d(smem_u32((is_v ? sm.v[vr.st] : sm.k[kr.st]) + slab * BN * 128 + unit * 32 * 128), is_v ? &tmV : &tmK,
                      is_v ? vb : kb, 64 * slab, it.g, row);
        }
        ++k_n;
        ++v_n;
        kr.advance();
        vr.advance();
      }
    }
    if (lane == 0) {
      // the last load of each buffer lands before the CTA exits
      if (q_n) mbar_wait_quiesce(smem_u32(&sm.q_full), (q_n - 1) & 1, 1 << 22);
      for (int s = 0; s < KS; ++s) {
        const uint32_t n = k_n / KS + (static_cast<uint32_t>(s) < k_n % KS ? 1 : 0);
        if (n) mbar_wait_quiesce(smem_u32(&sm.k_full[s]), (n - 1) & 1, 1 << 22);
      }
      for (int s = 0; s < VS; ++s) {
        const uint32_t n = v_n / VS + (static_cast<uint32_t>(s) < v_n % VS ? 1 : 0);
        if (n) mbar_wait_quiesce(smem_u32(&sm.v_full[s]), (n - 1) & 1, 1 << 22);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================================================ products
    {
      // The whole warp runs this, with one lane elected to issue: operands are then in uniform registers.  Issued by a branch
      // of one thread, a product of 8 instructions took it some 560 cycles whatever its size.
      const uint32_t leader = elect_one();
      Ring<KS> kr, kd;                  // K tile of the next S, of the next dQ
      Ring<VS> vr;
      uint32_t q_n = 0, done = 0, s_n = 0, clean_ph = 0;
      bool ok = true;
      const uint64_t dq = desc_sw128(smem_u32(sm.q), 16, 1024), ddo = desc_sw128(smem_u32(sm.d_o), 16, 1024);
      const uint64_t dk = desc_sw128(smem_u32(sm.k[0]), 16, 1024), dv = desc_sw128(smem_u32(sm.v[0]), 16, 1024);
      const uint64_t dkt = desc_sw128(smem_u32(sm.k[0]), BN * 128, 1024);
      // A wait that passes at once takes some 130 cycles with the tensor core idle, so the next barriers are looked at
      // while the last products are queued.
      bool k_ready = false, v_ready = false, ds_ready = false;
      auto nothing = [] {};
      auto test_k = [&] { return warp_test(smem_u32(&sm.k_full[kr.st]), kr.ph); };
      auto test_v = [&] { return warp_test(smem_u32(&sm.v_full[vr.st]), vr.ph); };
      auto issue_s = [&](int j, auto then) -> bool {
        if (!k_ready && !warp_wait(smem_u32(&sm.k_full[kr.st]), kr.ph, abort_flag, lim, 920)) return false;
        k_ready = false;
        if (j >= it.dirty) {
          if (!warp_wait(smem_u32(&sm.k_clean[kr.st]), (clean_ph >> kr.st) & 1, abort_flag, lim, 921)) return false;
          clean_ph ^= 1u << kr.st;
        }
        tc_fence_after();
        const uint32_t b = s_n & 1;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off16 = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
          mma_bf16_ss_by(leader, tmem + kColS + b * BN, dq + off16, dk + kr.st * (kTileBytes >> 4) + off16, kIdescS, kk > 0 ? 1u : 0u);
          if (kk == D / 16 - 3) then();
        }
        mma_commit_by(leader, smem_u32(&sm.s_full[b]));
        ++s_n;
        kr.advance();
        return true;
      };
      auto issue_dp = [&]() -> bool {
        if (!v_ready && !warp_wait(smem_u32(&sm.v_full[vr.st]), vr.ph, abort_flag, lim, 922)) return false;
        v_ready = false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off16 = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
          mma_bf16_ss_by(leader, tmem + kColP, ddo + off16, dv + vr.st * (kTileBytes >> 4) + off16, kIdescS, kk > 0 ? 1u : 0u);
        }
        mma_commit_by(leader, smem_u32(&sm.dp_full));
        mma_commit_by(leader, smem_u32(&sm.v_empty[vr.st]));
        vr.advance();
        return true;
      };
      for (int m = 0; m < rounds && ok; ++m) {
        if (!get(m, it)) continue;
        if (!(ok = warp_wait(smem_u32(&sm.q_full), q_n & 1, abort_flag, lim, 924))) break;
        ++q_n;
        tc_fence_after();
        if (!(ok = issue_s(0, nothing))) break;
        if (!(ok = issue_dp())) break;
        if (it.nt > 1 && !(ok = issue_s(1, nothing))) break;
        if (it.nt == 1) mma_commit_by(leader, smem_u32(&sm.q_empty));
        for (int j = 0; j < it.nt; ++j) {
          const uint32_t at = s_n - (j + 1 < it.nt ? 2 : 1);          // this tile among all
          if (j == 0 && !(ok = warp_wait(smem_u32(&sm.acc_empty), (done & 1) ^ 1, abort_flag, lim, 925))) break;
          if (!ds_ready && !(ok = warp_wait(smem_u32(&sm.ds_full[at & 1]), (at >> 1) & 1, abort_flag, lim, 926))) break;
          ds_ready = false;
          tc_fence_after();
          // dS tells that dP has been read as well
          if (j + 1 < it.nt) {
            if (!(ok = issue_dp())) break;
            if (j + 2 == it.nt) mma_commit_by(leader, smem_u32(&sm.q_empty));   // the last S and dP
          }
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            mma_bf16_ts_by(leader, tmem, tmem + kColS + (at & 1) * BN + (kk >> 1) * 32 + (kk & 1) * 8,
                        dkt + kd.st * (kTileBytes >> 4) + ((kk * 16 * 128) >> 4), kIdescQ, (kk > 0 || j > 0) ? 1u : 0u);
            if (kk == BN / 16 - 3) k_ready = j + 2 < it.nt && test_k();
          }
          if (it.nt <= kFewTiles)
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              mma_bf16_ts_by(leader, tmem, tmem + kColS + (at & 1) * BN + 16 + (kk >> 1) * 32 + (kk & 1) * 8,
                          dkt + kd.st * (kTileBytes >> 4) + ((kk * 16 * 128) >> 4), kIdescQ, 1u);
          mma_commit_by(leader, smem_u32(&sm.k_empty[kd.st]));
          kd.advance();
          if (j + 2 < it.nt && !(ok = issue_s(j + 2, [&] {
                ds_ready = warp_test(smem_u32(&sm.ds_full[(at + 1) & 1]), ((at + 1) >> 1) & 1);
                v_ready = test_v();
              })))
            break;
        }
        if (!ok) break;
        mma_commit_by(leader, smem_u32(&sm.acc_full));
        ++done;
      }
      mma_commit_by(leader, smem_u32(&sm.drain));
      if (!__all_sync(0xffffffffu, mbar_wait_quiesce(smem_u32(&sm.drain), 0, a.drain_limit)) && ok) {
        *abort_flag = 1;
        ra_record_error(RA_ERR_TIMEOUT, 927);
      }
    }
  } else if (warp == 2) {
    // ============================================================ zeroing of K rows past the sequence
    // A dirty tile is taken up once the load has been announced: from then on its stage's barrier can
    // only move from loading to loaded, so that the parity waited for is the right one.  The tiles before it are passed over
    // here while the others work them off (of one long sequence nearly all), which the limit allows for.
    Ring<KS> kr;
    uint32_t dirty_ph = 0;
    long long past = 0;                // tiles, an item's start and end counted as one, since the last dirty one
    bool ok = true;
    for (int m = 0; m < rounds && ok; ++m) {
      if (!get(m, it)) continue;
      ++past;
      for (int j = 0; j < it.nt; ++j, kr.advance()) {
        if (j < it.dirty) {
          ++past;
          continue;
        }
        if (!(ok = warp_wait(smem_u32(&sm.k_dirty[kr.st]), (dirty_ph >> kr.st) & 1, abort_flag, limit_over(lim, past), 930)))
          break;
        past = 0;
        dirty_ph ^= 1u << kr.st;
        if (!(ok = warp_wait(smem_u32(&sm.k_full[kr.st]), kr.ph, abort_flag, lim, 931))) break;
        const int left = it.n - it.skip - BN * j;                     // rows of the sequence in this tile
        for (int i = left + lane; i < BN; i += 32)
#pragma unroll
          for (int s = 0; s < SLABS; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(sm.k[kr.st] + s * BN * 128 + i * 128 + e * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.k_clean[kr.st]));
        __syncwarp();
      }
    }
  } else if (warp >= 4) {
    // ============================================================ dS and epilogue: rows by lane, 32 columns of a tile
    const int h = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int row_tok = a.by_G.div(row), row_head = row - row_tok * a.G;
    const uint64_t sc2 = f2pack(a.scale_log2, a.scale_log2);
    uint32_t s_n = 0, done = 0, wholes = 0;
    bool ok = true;
    for (int m = 0; m < rounds && ok; ++m) {
      if (!get(m, it)) continue;
      const int pos = it.tok0 + row_tok, head = it.g * a.G + row_head;
      const bool row_ok = row_tok < a.tpt && pos < it.n;
      const int64_t at = static_cast<int64_t>(head) * a.T + it.q0 + pos;
      const float nl = row_ok ? a.neg_lse[at] : -CUDART_INF_F;
      float nd = row_ok ? a.neg_delta[at] : 0.f;
      const uint64_t nl2 = f2pack(nl, nl);
      const int p = row_ok ? pos : -1, low = max(0, p + 1 - a.window), sinks = min(a.n_sink, p + 1);
      auto seen = [&](int u) {                                        // keys of unit u that the row sees
        const int from = 32 * u + (u < it.first ? 0 : it.skip);
        return (low_bits(p + 1 - from) & ~low_bits(low - from)) | low_bits(sinks - from);
      };
      uint64_t sum2 = f2pack(0.f, 0.f), p_sum2 = sum2;
      if (it.nt == 1) {
        // delta = sum of P dP, by each group over all columns, before any of them stores dS over the scores
        const float slack = row_ok ? a.slack[at] : 0.f;
        if (!(ok = warp_wait_first(smem_u32(&sm.s_full[s_n & 1]), (s_n >> 1) & 1, abort_flag, lim, 945))) break;
        if (!(ok = warp_wait(smem_u32(&sm.dp_full), s_n & 1, abort_flag, lim, 946))) break;
        tc_fence_after();
        float pd = 0.f, ps = 0.f;
#pragma unroll 1
        for (int g = 0; g < kGroups; ++g) {
          const uint32_t f = seen(g);
          uint32_t x[32], y[32];
          tmem_ld32(t_lane + kColS + (s_n & 1) * BN + 32 * g, x);
          tmem_ld32(t_lane + kColP + 32 * g, y);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float p0, p1;
            exp_pair(x[i], x[i + 1], sc2, nl2, p0, p1);
            if (f >> i & 1) {
              ps += p0;
              pd = fmaf(p0, __uint_as_float(y[i]), pd);
            }
            if (f >> i & 2) {
              ps += p1;
              pd = fmaf(p1, __uint_as_float(y[i + 1]), pd);
            }
          }
        }
        if (row_ok && sums_to_one(ps, nl) && fabsf(nd + pd) <= slack) nd = -pd;
        tc_fence_before();
        warp_arrive(smem_u32(&sm.all_read));
        if (!(ok = warp_wait(smem_u32(&sm.all_read), wholes & 1, abort_flag, lim, 947))) break;
        ++wholes;
        tc_fence_after();
      }
      const uint64_t nd2 = f2pack(nd, nd);
      for (int j = 0; j < it.nt; ++j) {
        const uint32_t b = s_n & 1;
        if (!(ok = warp_wait_first(smem_u32(&sm.s_full[b]), (s_n >> 1) & 1, abort_flag, lim, 940))) break;
        tc_fence_after();
        const uint32_t s_addr = t_lane + kColS + b * BN + 32 * h;
        uint32_t x[32], y[32], pk[16];
        tmem_ld32(s_addr, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          float p0, p1;
          exp_pair(x[i], x[i + 1], sc2, nl2, p0, p1);
          x[i] = __float_as_uint(p0);
          x[i + 1] = __float_as_uint(p1);
        }
        if (!(ok = warp_wait(smem_u32(&sm.dp_full), s_n & 1, abort_flag, lim, 941))) break;
        ++s_n;
        tc_fence_after();
        tmem_ld32(t_lane + kColP + 32 * h, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          float d0, d1;
          f2unpack(fmul2(fadd2(f2pack(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), nd2),
                         f2pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1]))),
                   d0, d1);
          y[i] = __float_as_uint(d0);
          y[i + 1] = __float_as_uint(d1);
        }
        if (j < it.low0 || j >= it.clean) {                            // not all of the tile is seen by all rows
          const uint32_t f = seen(4 * j + h);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(f >> i & 1)) x[i] = y[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          pk[i / 2] = f2_bf16x2(__uint_as_float(y[i]), __uint_as_float(y[i + 1]));
        }
        tmem_st16(s_addr, pk);
        if (it.nt <= kFewTiles) {
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            pk[i / 2] = f2_bf16x2(__uint_as_float(y[i]) - __uint_as_float(pk[i / 2] << 16),
                                  __uint_as_float(y[i + 1]) - __uint_as_float(pk[i / 2] & 0xffff0000u));
          tmem_st16(s_addr + 16, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(smem_u32(&sm.ds_full[b]));
        // the sums, while the next tile is on its way
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          sum2 = fadd2(sum2, f2pack(__uint_as_float(y[i]), __uint_as_float(y[i + 1])));
          p_sum2 = fadd2(p_sum2, f2pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
        }
      }
      if (!ok) break;
      // the row's sum of dS is the error of its delta
      float s0, s1, p0, p1;
      f2unpack(sum2, s0, s1);
      f2unpack(p_sum2, p0, p1);
      if (h > 0) {
        if (!(ok = warp_wait(smem_u32(&sm.sums_free), (done & 1) ^ 1, abort_flag, lim, 943))) break;
        sm.sums[h - 1][row] = s0 + s1;
        sm.p_sums[h - 1][row] = static_cast<uint16_t>(fminf((p0 + p1) / kUnit + 0.5f, 65535.f));
        warp_arrive(smem_u32(&sm.sums_full));
      } else {
        const float slack = row_ok ? a.slack[at] : 0.f;
        if (!(ok = warp_wait(smem_u32(&sm.sums_full), done & 1, abort_flag, lim, 944))) break;
        float sum = s0 + s1, p_sum = p0 + p1;
#pragma unroll
        for (int g = 1; g < kGroups; ++g) {
          sum += sm.sums[g - 1][row];
          p_sum += sm.p_sums[g - 1][row] * kUnit;
        }
        warp_arrive(smem_u32(&sm.sums_free));
        if (row_ok && sums_to_one(p_sum, nl) && fabsf(sum) <= slack) a.neg_delta[at] = nd - sum;
      }
      if (!(ok = warp_wait(smem_u32(&sm.acc_full), done & 1, abort_flag, lim, 942))) break;
      ++done;
      tc_fence_after();
      if (h < D / 32) {
        uint32_t z[32];
        tmem_ld32(t_lane + 32 * h, z);
        tmem_wait_ld();
        store_cols(a.dq, a.out_bf16, row_ok ? (it.q0 + static_cast<int64_t>(pos)) * a.dq_rs + head * D + 32 * h : -1, z, a.scale);
      }
      tc_fence_before();
      warp_arrive(smem_u32(&sm.acc_empty));
    }
    tmem_wait_st();   // a wait that expires between the stores and their own wait leaves them in flight
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ dK, dV
// A key tile, or the part [it0, it0 + its) of its (query tile, head) pairs, heads side by side.
struct KeyItem {
  int q0, n, k, g, it0, its, all;
  int64_t at;                          // on the axis of cost, of a part
};

// Items on their way from the warp that finds them to the others (TMA, products, rows' numbers, softmax), three ahead, so
// that nobody waits for their divisions and loads (window 512 over 16384 tokens, heads 32 on 8, d 128: 214 us; with every warp
// finding its own 236).  The kernel of dQ finds its items with less, and keeps what it finds in registers: read from such a
// ring they take that kernel's softmax further beyond its 96 registers (254 us instead of 238; as it is it spills 64 bytes).
constexpr int kAhead = 3;
constexpr int kReaders = 3 + kSoftmax / 32;
struct ItemRing {
  uint64_t full[kAhead], empty[kAhead];
  KeyItem item[kAhead];                   // n = 0: the end
  __device__ void init() {
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kReaders);
    }
  }
};
// By one thread.  It waits for whole items where the others wait for a tile, so its limit is that of a tile times the
// tiles of the longest item.
struct Announcer {
  ItemRing& ring;
  volatile int* abort_flag;
  long long lim;
  uint32_t at = 0;
  int longest = 0;
  __device__ bool put(const KeyItem& x) {
    const int i = at % kAhead;
    if (!mbar_wait(smem_u32(&ring.empty[i]), ((at / kAhead) & 1) ^ 1, abort_flag, limit_over(lim, longest), 906)) return false;
    longest = max(longest, x.its);
    ring.item[i] = x;
    mbar_arrive(smem_u32(&ring.full[i]));
    ++at;
    return true;
  }
};
// By whole warps.
struct ItemReader {
  ItemRing& ring;
  volatile int* abort_flag;
  long long lim;
  uint32_t at = 0;
  bool ok = true;                      // false: a wait has expired
  __device__ bool get(KeyItem& x) {
    const int i = at % kAhead;
    ok = warp_wait(smem_u32(&ring.full[i]), (at / kAhead) & 1, abort_flag, lim, 907);
    if (!ok) return false;
    x = ring.item[i];
    warp_arrive(smem_u32(&ring.empty[i]));
    ++at;
    return x.n > 0;
  }
};

// The items of a CTA: whole rounds, then its part of the rest.
struct KeyIter {
  const GradArgs& a;
  const Plan& plan;
  int whole, next, tile, g;
  int64_t lo, hi, at, cost;
  bool started, live;
  __device__ KeyIter(const GradArgs& args) : a(args), plan(*args.plan) {
    whole = plan.whole;
    next = blockIdx.x;
    lo = plan.lo[blockIdx.x];
    hi = plan.lo[blockIdx.x + 1];
    started = false;
    live = lo < hi;
  }
  __device__ bool get(KeyItem& s) {
    if (next < whole) {
      int head;
      const Tile t = a.keys[a.by_Hkv.div(next, head)];
      s.q0 = t.q0; s.n = t.n; s.k = t.k; s.g = head;
      s.it0 = 0;
      s.its = s.all = query_tiles(a, t.n, t.k) * a.G;
      s.at = -1;
      next += kGradCtas;
      return true;
    }
    while (live) {
      if (!started) {
        started = true;
        tile = plan.start[blockIdx.x];
        const Tile t = a.keys[tile];
        cost = cost_of(a, t.n, t.k);
        g = static_cast<int>((lo - a.base[tile]) / cost);
        at = a.base[tile] + g * cost;
      } else {
        at += cost;
        if (++g == a.Hkv) {
          g = 0;
          if (++tile >= plan.key_tiles) return live = false;
        }
      }
      if (at >= hi) return live = false;
      const Tile t = a.keys[tile];
      cost = cost_of(a, t.n, t.k);
      s.all = static_cast<int>(cost) - kOver;
      // the first kOver of the cost are the start and end
      const int64_t from = lo - at - kOver, to = hi - at - kOver;
      s.it0 = from > 0 ? static_cast<int>(from < s.all ? from : s.all) : 0;
      const int end = hi >= at + cost ? s.all : to > 0 ? static_cast<int>(to < s.all ? to : s.all) : 0;
      if (end <= s.it0) continue;
      s.its = end - s.it0;
      s.q0 = t.q0; s.n = t.n; s.k = t.k; s.g = g;
      s.at = at;
      return true;
    }
    return false;
  }
};

template <int D>
struct __align__(1024) KeySmem {
  static constexpr int QS = D == 128 ? 3 : 4, OS = D == 128 ? 2 : 4, XS = 2;
  uint8_t k[BN * D * 2], v[BN * D * 2], q[QS][BM * D * 2], d_o[OS][BM * D * 2];
  uint64_t k_full, k_empty, v_full, v_empty, q_full[QS], q_empty[QS], o_full[OS], o_empty[OS], x_full[XS], x_empty[XS];
  uint64_t s_full, p_full, dp_full, ds_full, acc_full, acc_empty, drain;
  ItemRing items;
  __align__(16) float neg_lse[XS][BM], neg_delta[XS][BM];   // read four at a time
  uint32_t tmem_base;
  int abort_flag;
};

static_assert(sizeof(RowSmem<128>) <= 232448 && sizeof(RowSmem<64>) <= 232448 && sizeof(KeySmem<128>) <= 232448 &&
                  sizeof(KeySmem<64>) <= 232448,
              "227 KB of shared memory");

// Tensor memory: dK, dV, then S^T with P^T of each 32 columns over the first half of them, then dP^T with dS^T likewise.
template <int D>
__global__ void __launch_bounds__(kGradThreads, 1)
    grad_kv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                   const __grid_constant__ GradArgs a) {
  using Smem = KeySmem<D>;
  constexpr int SLABS = D / 64, QS = Smem::QS, OS = Smem::OS, XS = Smem::XS;
  constexpr uint32_t kTileBytes = BM * D * 2;
  constexpr uint32_t kColV = D, kColS = 2 * D, kColP = 2 * D + BN;
  static_assert(kColP + BN <= kTmemCols);
  constexpr uint32_t kIdescS = idesc_bf16_f32(BN, BM, 0, 0), kIdescA = idesc_bf16_f32(BN, D, 0, 1);

  extern __shared__ __align__(1024) uint8_t smem_grad[];   // no room to align it by hand
  Smem& sm = *reinterpret_cast<Smem*>(smem_grad);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const long long lim = a.wait_limit;
  if (smem_u32(smem_grad) & 1023) {
    if (threadIdx.x == 0) ra_record_error(RA_ERR_CUDA, 905);
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sm.k_full), 1);
    mbar_init(smem_u32(&sm.k_empty), 1);
    mbar_init(smem_u32(&sm.v_full), 1);
    mbar_init(smem_u32(&sm.v_empty), 1);
    for (int s = 0; s < QS; ++s) {
      mbar_init(smem_u32(&sm.q_full[s]), 1);
      mbar_init(smem_u32(&sm.q_empty[s]), 1);
    }
    for (int s = 0; s < OS; ++s) {
      mbar_init(smem_u32(&sm.o_full[s]), 1);
      mbar_init(smem_u32(&sm.o_empty[s]), 1);
    }
    for (int s = 0; s < XS; ++s) {
      mbar_init(smem_u32(&sm.x_full[s]), 1);
      mbar_init(smem_u32(&sm.x_empty[s]), kSoftmax / 32);
    }
    mbar_init(smem_u32(&sm.s_full), 1);
    mbar_init(smem_u32(&sm.p_full), kSoftmax / 32);
    mbar_init(smem_u32(&sm.dp_full), 1);
    mbar_init(smem_u32(&sm.ds_full), kSoftmax / 32);
    mbar_init(smem_u32(&sm.acc_full), 1);
    mbar_init(smem_u32(&sm.acc_empty), kSoftmax / 32);
    mbar_init(smem_u32(&sm.drain), 1);
    sm.items.init();
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  ItemReader items{sm.items, abort_flag, lim};
  KeyItem it;

  if (warp == 0) {
    // ============================================================ loads
    Ring<QS> qr;
    Ring<OS> orr;
    uint32_t q_n = 0, o_n = 0, kv_n = 0, v_n = 0;
    bool ok = true;
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(&tmO);
    }
    auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int hd, int row) {
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(bar), kTileBytes);
        for (int s = 0; s < SLABS; ++s) tma_load_3d(smem_u32(dst + s * BM * 128), map, smem_u32(bar), 64 * s, hd, row);
      }
      __syncwarp();
    };
    while (ok && items.get(it)) {
      int qt = it.k + a.by_G.div(it.it0);
      int head = it.it0 - (qt - it.k) * a.G;
      for (int j = 0; j < it.its; ++j) {
        const int row = it.q0 + BM * qt, hd = it.g * a.G + head;
        if (!(ok = warp_wait(smem_u32(&sm.q_empty[qr.st]), qr.ph ^ 1, abort_flag, lim, 951))) break;
        load(sm.q[qr.st], &tmQ, &sm.q_full[qr.st], hd, row);
        ++q_n;
        qr.advance();
        if (j == 0) {   // the keys after the first queries, which need not wait for the last keys
          if (!(ok = warp_wait(smem_u32(&sm.k_empty), (kv_n & 1) ^ 1, abort_flag, lim, 950))) break;
          ++kv_n;
          load(sm.k, &tmK, &sm.k_full, it.g, it.q0 + BN * it.k);
        }
        if (!(ok = warp_wait(smem_u32(&sm.o_empty[orr.st]), orr.ph ^ 1, abort_flag, lim, 953))) break;
        load(sm.d_o[orr.st], &tmO, &sm.o_full[orr.st], hd, row);
        ++o_n;
        orr.advance();
        if (j == 0) {
          if (!(ok = warp_wait(smem_u32(&sm.v_empty), (v_n & 1) ^ 1, abort_flag, lim, 952))) break;
          ++v_n;
          load(sm.v, &tmV, &sm.v_full, it.g, it.q0 + BN * it.k);
        }
        if (++head == a.G) {
          head = 0;
          ++qt;
        }
      }
    }
    if (lane == 0) {
      // the last load of each buffer lands before the CTA exits
      if (kv_n) mbar_wait_quiesce(smem_u32(&sm.k_full), (kv_n - 1) & 1, 1 << 22);
      if (v_n) mbar_wait_quiesce(smem_u32(&sm.v_full), (v_n - 1) & 1, 1 << 22);
      for (int s = 0; s < QS; ++s) {
        const uint32_t n = q_n / QS + (static_cast<uint32_t>(s) < q_n % QS ? 1 : 0);
        if (n) mbar_wait_quiesce(smem_u32(&sm.q_full[s]), (n - 1) & 1, 1 << 22);
      }
      for (int s = 0; s < OS; ++s) {
        const uint32_t n = o_n / OS + (static_cast<uint32_t>(s) < o_n % OS ? 1 : 0);
        if (n) mbar_wait_quiesce(smem_u32(&sm.o_full[s]), (n - 1) & 1, 1 << 22);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================================================ products
    {
      const uint32_t leader = elect_one();
      Ring<QS> qs, qd;                  // Q tile of the next S, of the next dK
      Ring<OS> op, od;                  // dO tile of the next dP, of the next dV
      Ring<XS> xs;
      uint32_t kv_n = 0, it_n = 0, done = 0;
      bool ok = true;
      const uint64_t dk = desc_sw128(smem_u32(sm.k), 16, 1024), dv = desc_sw128(smem_u32(sm.v), 16, 1024);
      const uint64_t dq = desc_sw128(smem_u32(sm.q[0]), 16, 1024), ddo = desc_sw128(smem_u32(sm.d_o[0]), 16, 1024);
      const uint64_t dqt = desc_sw128(smem_u32(sm.q[0]), BM * 128, 1024), dot = desc_sw128(smem_u32(sm.d_o[0]), BM * 128, 1024);
      // As in the dQ kernel the next barrier is looked at while the last products are queued.
      bool q_ready = false, o_ready = false, p_ready = false, ds_ready = false;
      auto scores = [&](uint32_t col, uint64_t da, uint64_t db, uint64_t* bar, auto then) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off16 = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
          mma_bf16_ss_by(leader, tmem + col, da + off16, db + off16, kIdescS, kk > 0 ? 1u : 0u);
          if (kk == D / 16 - 3) then();
        }
        mma_commit_by(leader, smem_u32(bar));
      };
      auto add = [&](uint32_t acc, uint32_t col, uint64_t db, bool first, auto then) {
#pragma unroll
        for (int kk = 0; kk < BM / 16; ++kk) {
          mma_bf16_ts_by(leader, tmem + acc, tmem + col + (kk >> 1) * 32 + (kk & 1) * 8, db + ((kk * 16 * 128) >> 4), kIdescA,
                      (kk > 0 || !first) ? 1u : 0u);
          if (kk == BM / 16 - 3) then();
        }
      };
      while (ok && items.get(it)) {
        // pairs of the sequence's last query tile, where it is not full, wait for its rows past the end to be zeroed
        const int last = it.n % BM == 0 ? INT32_MAX : ((it.n / BM) - it.k) * a.G - it.it0;
        auto issue_s = [&](int j) -> bool {
          if (!q_ready && !warp_wait(smem_u32(&sm.q_full[qs.st]), qs.ph, abort_flag, lim, 960)) return false;
          q_ready = false;
          if (j >= last && !warp_wait(smem_u32(&sm.x_full[xs.st]), xs.ph, abort_flag, lim, 961)) return false;
          xs.advance();
          tc_fence_after();
          scores(kColS, dk, dq + qs.st * (kTileBytes >> 4), &sm.s_full,
                 [&] { ds_ready = j > 0 && warp_test(smem_u32(&sm.ds_full), it_n & 1); });
          qs.advance();
          return true;
        };
        auto issue_dp = [&]() -> bool {
          if (!o_ready && !warp_wait(smem_u32(&sm.o_full[op.st]), op.ph, abort_flag, lim, 962)) return false;
          o_ready = false;
          tc_fence_after();
          scores(kColP, dv, ddo + op.st * (kTileBytes >> 4), &sm.dp_full,
                 [&] { p_ready = warp_test(smem_u32(&sm.p_full), it_n & 1); });
          op.advance();
          return true;
        };
        if (!(ok = warp_wait(smem_u32(&sm.k_full), kv_n & 1, abort_flag, lim, 963))) break;
        if (!(ok = issue_s(0))) break;
        if (it.its == 1) mma_commit_by(leader, smem_u32(&sm.k_empty));
        if (!(ok = warp_wait(smem_u32(&sm.v_full), kv_n & 1, abort_flag, lim, 964))) break;
        ++kv_n;
        if (!(ok = issue_dp())) break;
        if (it.its == 1) mma_commit_by(leader, smem_u32(&sm.v_empty));
        for (int j = 0; j < it.its; ++j) {
          const bool more = j + 1 < it.its;
          if (j == 0 && !(ok = warp_wait(smem_u32(&sm.acc_empty), (done & 1) ^ 1, abort_flag, lim, 965))) break;
          if (!p_ready && !(ok = warp_wait(smem_u32(&sm.p_full), it_n & 1, abort_flag, lim, 966))) break;
          p_ready = ds_ready = false;
          tc_fence_after();
          add(kColV, kColS, dot + od.st * (kTileBytes >> 4), j == 0,
              [&] { q_ready = more && warp_test(smem_u32(&sm.q_full[qs.st]), qs.ph); });
          mma_commit_by(leader, smem_u32(&sm.o_empty[od.st]));
          od.advance();
          if (more) {
            if (!(ok = issue_s(j + 1))) break;
            if (j + 2 == it.its) mma_commit_by(leader, smem_u32(&sm.k_empty));
          }
          if (!ds_ready && !(ok = warp_wait(smem_u32(&sm.ds_full), it_n & 1, abort_flag, lim, 967))) break;
          ds_ready = false;
          ++it_n;
          tc_fence_after();
          add(0, kColP, dqt + qd.st * (kTileBytes >> 4), j == 0,
              [&] { o_ready = more && warp_test(smem_u32(&sm.o_full[op.st]), op.ph); });
          mma_commit_by(leader, smem_u32(&sm.q_empty[qd.st]));
          qd.advance();
          if (more) {
            if (!(ok = issue_dp())) break;
            if (j + 2 == it.its) mma_commit_by(leader, smem_u32(&sm.v_empty));
          }
        }
        if (!ok) break;
        mma_commit_by(leader, smem_u32(&sm.acc_full));
        ++done;
      }
      mma_commit_by(leader, smem_u32(&sm.drain));
      if (!__all_sync(0xffffffffu, mbar_wait_quiesce(smem_u32(&sm.drain), 0, a.drain_limit)) && ok && items.ok) {
        *abort_flag = 1;
        ra_record_error(RA_ERR_TIMEOUT, 968);
      }
    }
  } else if (warp == 2) {
    // ============================================================ -lse and -delta of the query rows; rows past the end to zero
    Ring<XS> xr;
    Ring<QS> qr;
    Ring<OS> orr;
    bool ok = true;
    while (ok && items.get(it)) {
      int qt = it.k + a.by_G.div(it.it0);
      int head = it.it0 - (qt - it.k) * a.G;
      for (int j = 0; j < it.its; ++j) {
        const int left = it.n - BM * qt;                              // rows of the sequence in this tile
        const int64_t at = static_cast<int64_t>(it.g * a.G + head) * a.T + it.q0 + BM * qt;
        float nl[4], nd[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 32 * i + lane;
          nl[i] = r < left ? a.neg_lse[at + r] : -CUDART_INF_F;
          nd[i] = r < left ? a.neg_delta[at + r] : 0.f;
        }
        if (!(ok = warp_wait(smem_u32(&sm.x_empty[xr.st]), xr.ph ^ 1, abort_flag, lim, 970))) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sm.neg_lse[xr.st][32 * i + lane] = nl[i];
          sm.neg_delta[xr.st][32 * i + lane] = nd[i];
        }
        if (left < BM) {
          if (!(ok = warp_wait(smem_u32(&sm.q_full[qr.st]), qr.ph, abort_flag, lim, 971))) break;
          if (!(ok = warp_wait(smem_u32(&sm.o_full[orr.st]), orr.ph, abort_flag, lim, 972))) break;
          for (int i = left + lane; i < BM; i += 32)
#pragma unroll
            for (int s = 0; s < SLABS; ++s)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                *reinterpret_cast<uint4*>(sm.q[qr.st] + s * BM * 128 + i * 128 + e * 16) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(sm.d_o[orr.st] + s * BM * 128 + i * 128 + e * 16) = make_uint4(0, 0, 0, 0);
              }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.x_full[xr.st]));
        __syncwarp();
        xr.advance();
        qr.advance();
        orr.advance();
        if (++head == a.G) {
          head = 0;
          ++qt;
        }
      }
    }
  } else if (warp == 3) {
    // ============================================================ the items, and the tile that this CTA's part starts and
    // others go on with
    if (lane == 0) {
      Announcer out{sm.items, abort_flag, lim};
      KeyIter found(a);
      Shared s = {};
      bool going = true;
      while (going && found.get(it)) {
        if (it.at >= 0 && it.it0 == 0 && it.its < it.all) s = Shared{1, it.q0, it.n, it.k, it.g, it.all, it.at};
        going = out.put(it);
      }
      it.n = it.its = 0;
      if (going) out.put(it);
      a.shared[blockIdx.x] = s;
    }
    __syncwarp();
  } else {
    // ============================================================ P^T, dS^T and epilogue: keys by lane, 32 queries of a tile
    const int h = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_addr = t_lane + kColS + 32 * h, p_addr = t_lane + kColP + 32 * h;
    const uint64_t sc2 = f2pack(a.scale_log2, a.scale_log2);
    Ring<XS> xr;
    uint32_t it_n = 0, done = 0;
    bool ok = true;
    while (ok && items.get(it)) {
      int qt = it.k + a.by_G.div(it.it0);
      int head = it.it0 - (qt - it.k) * a.G;
      const int key = BN * it.k + row;                                // its position, seen by [key, far)
      const int64_t far64 = key < a.n_sink ? it.n : min(static_cast<int64_t>(it.n), static_cast<int64_t>(key) + a.window);
      const int far = static_cast<int>(far64);
      const bool tile_sinks = BN * (it.k + 1) <= a.n_sink;             // all keys of the tile are first tokens
      for (int j = 0; j < it.its; ++j) {
        // the diagonal, the window's far end for the tile's first key, the sequence's end
        const bool masked = qt == it.k || BM * qt + BM > it.n || (!tile_sinks && BM * (qt - it.k) + BM > a.window);
        if (!(ok = warp_wait(smem_u32(&sm.x_full[xr.st]), xr.ph, abort_flag, lim, 980))) break;
        if (!(ok = warp_wait_first(smem_u32(&sm.s_full), it_n & 1, abort_flag, lim, 981))) break;
        tc_fence_after();
        const ulonglong2* nl = reinterpret_cast<const ulonglong2*>(sm.neg_lse[xr.st] + 32 * h);
        const ulonglong2* nd = reinterpret_cast<const ulonglong2*>(sm.neg_delta[xr.st] + 32 * h);
        float p[32];
        uint32_t x[32], pk[16];
        tmem_ld32(s_addr, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const ulonglong2 l = nl[i / 4];
          exp_pair(x[i], x[i + 1], sc2, l.x, p[i], p[i + 1]);
          exp_pair(x[i + 2], x[i + 3], sc2, l.y, p[i + 2], p[i + 3]);
        }
        uint32_t seen = 0xffffffffu;
        if (masked) {
          const int from = BM * qt + 32 * h;                          // position of the first of these queries
          seen = low_bits(far - from) & ~low_bits(key - from);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(seen >> i & 1)) p[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[i] = f2_bf16x2(p[2 * i], p[2 * i + 1]);
        tmem_st16(s_addr, pk);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(smem_u32(&sm.p_full));
        if (!(ok = warp_wait(smem_u32(&sm.dp_full), it_n & 1, abort_flag, lim, 982))) break;
        ++it_n;
        tc_fence_after();
        tmem_ld32(p_addr, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const ulonglong2 dl = nd[i / 4];
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            float d0, d1;
            f2unpack(fmul2(fadd2(f2pack(__uint_as_float(x[i + e]), __uint_as_float(x[i + e + 1])), e ? dl.y : dl.x),
                           f2pack(p[i + e], p[i + e + 1])),
                     d0, d1);
            x[i + e] = __float_as_uint(d0);
            x[i + e + 1] = __float_as_uint(d1);
          }
        }
        if (masked)   // 0 * inf
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(seen >> i & 1)) x[i] = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[i] = f2_bf16x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
        tmem_st16(p_addr, pk);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(smem_u32(&sm.ds_full));
        warp_arrive(smem_u32(&sm.x_empty[xr.st]));
        xr.advance();
        if (++head == a.G) {
          head = 0;
          ++qt;
        }
      }
      if (!ok) break;
      if (!(ok = warp_wait(smem_u32(&sm.acc_full), done & 1, abort_flag, lim, 983))) break;
      ++done;
      tc_fence_after();
      const bool part = it.its < it.all;
      // warpgroups 0 and 1 take dK, 2 and 3 dV, half the columns each
      const int v = h >> 1, col0 = (h & 1) * (D / 2);
      float* to = a.parts + ((2 * static_cast<int64_t>(blockIdx.x) + (it.it0 == 0 ? 1 : 0)) * 2 + v) * (BN * D);
      const int64_t out = (it.q0 + static_cast<int64_t>(key)) * (v ? a.dv_rs : a.dk_rs) + it.g * D;
#pragma unroll 1
      for (int c = col0; c < col0 + D / 2; c += 32) {
        uint32_t z[32];
        tmem_ld32(t_lane + (v ? kColV : 0) + c, z);
        tmem_wait_ld();
        if (part) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(to + ((c / 4 + i) * BN + row) * 4) = make_uint4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
        } else {
          store_cols(v ? a.dv : a.dk, a.out_bf16, key < it.n ? out + c : -1, z, v ? 1.f : a.scale);
        }
      }
      tc_fence_before();
      warp_arrive(smem_u32(&sm.acc_empty));
    }
    tmem_wait_st();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ joining
// Block (c, y) sums the parts of the key tile that part c starts, if it does, four columns of all rows at a time, in order.
template <int D>
__global__ void __launch_bounds__(BN) grad_join_kernel(const __grid_constant__ GradArgs a) {
  __shared__ int slots[kGradCtas], counts[BN / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Shared s = a.shared[blockIdx.x];
  if (!s.used) return;
  const int row = threadIdx.x, lane = row & 31, key = BN * s.k + row;
  const int64_t cost = s.its + kOver;
  int n = 0;
  for (int c0 = blockIdx.x; c0 < kGradCtas; c0 += BN) {
    const int c = c0 + row;
    int it0 = 0, end = 0;
    if (c < kGradCtas) {
      // as KeyIter cuts it
      const int64_t lo = a.plan->lo[c], hi = a.plan->lo[c + 1], from = lo - s.at - kOver, to = hi - s.at - kOver;
      if (lo < s.at + cost) {
        it0 = from > 0 ? static_cast<int>(from < s.its ? from : s.its) : 0;
        end = hi >= s.at + cost ? s.its : to > 0 ? static_cast<int>(to < s.its ? to : s.its) : 0;
      }
    }
    const unsigned b = __ballot_sync(0xffffffffu, end > it0);
    if (lane == 0) counts[row >> 5] = __popc(b);
    __syncthreads();
    int at = n + __popc(b & ((1u << lane) - 1));
    for (int w = 0; w < BN / 32; ++w) {
      if (w < row >> 5) at += counts[w];
      n += counts[w];
    }
    if (end > it0) slots[at] = 2 * c + (it0 == 0 ? 1 : 0);
    __syncthreads();
  }
  for (int u = blockIdx.y; u < 2 * (D / 4); u += gridDim.y) {
    const int h = u / (D / 4), col = u - h * (D / 4);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(a.parts + (slots[i] * int64_t(2) + h) * (BN * D) + (col * BN + row) * 4);
      sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
    }
    if (key >= s.n) continue;
    const float f = h ? 1.f : a.scale;
    const int64_t at = (s.q0 + static_cast<int64_t>(key)) * (h ? a.dv_rs : a.dk_rs) + s.g * D + 4 * col;
    void* out = h ? a.dv : a.dk;
    if (a.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
          make_uint2(f2_bf16x2(sum.x * f, sum.y * f), f2_bf16x2(sum.z * f, sum.w * f));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(sum.x * f, sum.y * f, sum.z * f, sum.w * f);
  }
}

// ------------------------------------------------------------------ host side
// Places in the workspace, 256-byte aligned.
struct Layout {
  size_t lse, delta, slack, rows, keys, base, plan, shared, parts, bytes;
  Layout(int64_t T, int32_t R, int32_t Hq, int32_t Hkv, int32_t d) {
    size_t at = 0;
    auto put = [&](size_t n) {
      const size_t x = at;
      at += (n + 255) / 256 * 256;
      return x;
    };
    // sequences do not lie over one another, and each may end inside a tile
    const size_t key_tiles = T / BN + R, row_tiles = T / (BM / (Hq / Hkv)) + R;
    lse = put(static_cast<size_t>(T) * Hq * 4);
    delta = put(static_cast<size_t>(T) * Hq * 4);
    slack = put(static_cast<size_t>(T) * Hq * 4);
    rows = put(row_tiles * sizeof(Tile));
    keys = put(key_tiles * sizeof(Tile));
    base = put(key_tiles * 8);
    plan = put(sizeof(Plan));
    shared = put(kGradCtas * sizeof(Shared));
    parts = put(static_cast<size_t>(2 * kGradCtas) * 2 * BN * d * 4);
    bytes = at + 256;
  }
};

template <int D>
ra_status launch_grad(const void* q, int64_t q_rs, const void* k, int64_t k_rs, const void* v, int64_t v_rs, const GradArgs& a,
                      cudaStream_t stream) {
  CUtensorMap mq, mk, mv, mo, mqt, mkt, mvt, mot;
  ra_status st;
  const int64_t o_rs = static_cast<int64_t>(a.Hq) * D;
  if ((st = row_map(&mq, q, D, a.Hq, a.T, q_rs, a.G, a.tpt)) != RA_OK) return st;
  if ((st = row_map(&mo, a.d_o, D, a.Hq, a.T, o_rs, a.G, a.tpt)) != RA_OK) return st;
  if ((st = row_map(&mk, k, D, a.Hkv, a.T, k_rs, 1, 32)) != RA_OK) return st;
  if ((st = row_map(&mv, v, D, a.Hkv, a.T, v_rs, 1, 32)) != RA_OK) return st;
  if ((st = row_map(&mqt, q, D, a.Hq, a.T, q_rs, 1, BM)) != RA_OK) return st;
  if ((st = row_map(&mot, a.d_o, D, a.Hq, a.T, o_rs, 1, BM)) != RA_OK) return st;
  if ((st = row_map(&mkt, k, D, a.Hkv, a.T, k_rs, 1, BN)) != RA_OK) return st;
  if ((st = row_map(&mvt, v, D, a.Hkv, a.T, v_rs, 1, BN)) != RA_OK) return st;
  const int64_t warps = (a.T + 7) / 8 * a.Hq;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(ra::ceil_div(warps, kPlanThreads / 32), 2 * 152)) + 1;
  grad_prepare_kernel<D><<<blocks, kPlanThreads, 0, stream>>>(a);
  RA_LAUNCH_CHECK("grad_prepare_kernel");
  const size_t rows = sizeof(RowSmem<D>), keys = sizeof(KeySmem<D>);
  RA_CUDA_TRY(cudaFuncSetAttribute(grad_q_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(rows)));
  RA_CUDA_TRY(cudaFuncSetAttribute(grad_kv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(keys)));
  // Each kernel comes up while the one before it ends, and waits for its end before it reads what it wrote.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kGradCtas);
  cfg.blockDim = dim3(kGradThreads);
  cfg.dynamicSmemBytes = rows;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  RA_CUDA_TRY(cudaLaunchKernelEx(&cfg, grad_q_kernel<D>, mq, mk, mv, mo, a));
  cfg.dynamicSmemBytes = keys;
  RA_CUDA_TRY(cudaLaunchKernelEx(&cfg, grad_kv_kernel<D>, mqt, mkt, mvt, mot, a));
  cfg.gridDim = dim3(kGradCtas, 16);
  cfg.blockDim = dim3(BN);
  cfg.dynamicSmemBytes = 0;
  RA_CUDA_TRY(cudaLaunchKernelEx(&cfg, grad_join_kernel<D>, a));
  return RA_OK;
}

}  // namespace

namespace ra {
size_t window_backward_workspace(int64_t T, int32_t R, int32_t Hq, int32_t Hkv, int32_t d) {
  return Layout(T, R, Hq, Hkv, d).bytes;
}
}  // namespace ra

extern "C" ra_status ra_window_attn_bwd(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                        const void* v, int64_t v_row_stride, const void* o, const float* lse,
                                        const void* d_o, const int32_t* query_start_loc, int64_t T, int32_t R, int32_t Hq,
                                        int32_t Hkv, int32_t d, int32_t window, int32_t n_sink, float scale, void* dq,
                                        int64_t dq_row_stride, void* dk, int64_t dk_row_stride, void* dv,
                                        int64_t dv_row_stride, ra_dtype out_dt, void* workspace, size_t ws_bytes,
                                        ra_stream stream) {
  ra::clear_error();
  size_t need = 0;
  ra_status st = check_packed(q, q_row_stride, k, k_row_stride, v, v_row_stride, query_start_loc, T, R, Hq, Hkv, d, window,
                              n_sink, out_dt, workspace, ws_bytes, need);
  if (st != RA_OK) return st;
  const int64_t lim = int64_t(1) << 31, es = out_dt == RA_BF16 ? 2 : 4, qw = static_cast<int64_t>(Hq) * d,
                kw = static_cast<int64_t>(Hkv) * d;
  RA_REQUIRE(dq_row_stride >= qw && dk_row_stride >= kw && dv_row_stride >= kw && dq_row_stride < lim &&
                 dk_row_stride < lim && dv_row_stride < lim,
             "row strides must be at least heads * d, below 2^31");
  RA_REQUIRE(dq_row_stride * es % 16 == 0 && dk_row_stride * es % 16 == 0 && dv_row_stride * es % 16 == 0,
             "row strides must be multiples of 16 bytes");
  if (T == 0) return RA_OK;
  RA_REQUIRE(o && lse && d_o && dq && dk && dv, "NULL pointer");
  RA_REQUIRE(ra::aligned16(o) && ra::aligned16(d_o) && ra::aligned16(dq) && ra::aligned16(dk) && ra::aligned16(dv),
             "o, d_o, dq, dk and dv must be 16-byte aligned");
  struct Rows {
    const void* p;
    int64_t s, w;
  };
  const Rows outs[3] = {{dq, dq_row_stride * es, qw * es}, {dk, dk_row_stride * es, kw * es}, {dv, dv_row_stride * es, kw * es}};
  const Rows ins[6] = {{q, q_row_stride * 2, qw * 2}, {k, k_row_stride * 2, kw * 2}, {v, v_row_stride * 2, kw * 2},
                       {o, qw * 2, qw * 2},           {d_o, qw * 2, qw * 2},         {lse, Hq * 4, Hq * 4}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      RA_REQUIRE(!ra::rows_meet(outs[i].p, outs[i].s, outs[i].w, outs[j].p, outs[j].s, outs[j].w, T), "dq, dk and dv must not overlap");
    for (const Rows& in : ins)
      RA_REQUIRE(!ra::rows_meet(outs[i].p, outs[i].s, outs[i].w, in.p, in.s, in.w, T),
                 "dq, dk and dv must not overlap the inputs");
  }
  const Layout at(T, R, Hq, Hkv, d);
  auto span = [&](const Rows& x) { return ra::row_span(x.p, T, x.s, x.w); };
  if ((st = ra::check_workspace_apart(ra::Span{workspace, need}, span(outs[0]), span(outs[1]), span(outs[2]), span(ins[3]),
                                      span(ins[4]), span(ins[5]))) != RA_OK)
    return st;
  uint8_t* ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
  GradArgs a = {};
  a.qsl = query_start_loc; a.T = T; a.R = R; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv;
  a.window = std::min(window, kFar);
  a.n_sink = std::min(n_sink, kFar);
  a.tpt = BM / a.G;
  a.out_bf16 = out_dt == RA_BF16;
  a.scale = scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(d));
  a.scale_log2 = a.scale * 1.4426950408889634f;
  a.o = static_cast<const __nv_bfloat16*>(o);
  a.d_o = static_cast<const __nv_bfloat16*>(d_o);
  a.lse = lse;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dq_rs = dq_row_stride; a.dk_rs = dk_row_stride; a.dv_rs = dv_row_stride;
  a.neg_lse = reinterpret_cast<float*>(ws + at.lse);
  a.neg_delta = reinterpret_cast<float*>(ws + at.delta);
  a.slack = reinterpret_cast<float*>(ws + at.slack);
  a.rows = reinterpret_cast<Tile*>(ws + at.rows);
  a.keys = reinterpret_cast<Tile*>(ws + at.keys);
  a.base = reinterpret_cast<int64_t*>(ws + at.base);
  a.plan = reinterpret_cast<Plan*>(ws + at.plan);
  a.shared = reinterpret_cast<Shared*>(ws + at.shared);
  a.parts = reinterpret_cast<float*>(ws + at.parts);
  a.by_G = fast_div(a.G);
  a.by_Hkv = fast_div(Hkv);
  a.wait_limit = ra::wait_limit();
  a.drain_limit = std::max<long long>(a.wait_limit, 1ll << 22);
  return d == 128 ? launch_grad<128>(q, q_row_stride, k, k_row_stride, v, v_row_stride, a, stream)
                  : launch_grad<64>(q, q_row_stride, k, k_row_stride, v, v_row_stride, a, stream);
}
