// New tokens' K and V on their way into the sharded paged cache, K (and Q beside
// it) turned by the rotary positions as they pass.
//
// Mathematics.  Token i of request r is the context's token x = ctx_r - n_r + i:
// K[x] = mscale * Rot(pos) k, V[x] = v, q_out = mscale * Rot(pos) q, with the
// rotation of ra_rope_turn.cuh and the place of x of ra_paged.cuh.
//
// One launch in place of four (the rotation of Q, that of K, the slot mapping, the
// scatter), so that K passes through the chip once.  A group of threads takes a token at a time: it finds the token's
// request and place, forms the angles of its pairs once (for all heads, in shared memory), and takes the words of its
// heads, whose loads are a step ahead of the stores and start before the place is known.
//
// Bound by memory: Q, K and V of a token are read once and written once.  16384 tokens with 32 + 8 + 8 heads of 128 (bf16)
// move 403 MB in 72 us, 5.6 TB/s; 48 tokens take 6.4 us, the latency of request, block table, angles and stores.  A
// group is a warp, so that nothing waits for a block (with barriers between every few tokens 77 to 82 us); where
// the tokens are few it is a block, whose 256 threads are through with a token sooner (64 tokens 6.4 us, by warps 10.5).
#include <algorithm>
#include <type_traits>

#include "ra_paged.cuh"
#include "ra_rope_turn.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_rope_append)

namespace {

constexpr int kAppendThreads = 256;
// Of an SM, and the heads of a thread whose loads are in flight together: 3 and 2 are 80 registers, of which bf16 in halves
// of 16-byte words spills 24 bytes (a block to a token) or 40 (a warp): 16384 tokens 72 us.  4 and 2 spill more, 92; 5 and 1
// 78; 2 and 4 86.
constexpr int kAppendBlocks = 3;
constexpr int kAppendHeads = 2;
// So many tokens or fewer have a block each, two rounds of them: 608 tokens take 8.5 us (by warps 10.5), 912 10.5 (10.6),
// 1216 12.8 (10.9), 16384 121 (70).
constexpr int kBlockTokens = 912;

struct AppendParams : Turns {
  Paged c;
  const void *k, *v, *q;
  void *k_cache, *v_cache, *q_out;
  const int32_t *qsl, *ctx;
  const int32_t* positions;      // of axis a: positions + a * T; NULL: the token's place in its context
  int64_t T, k_rs, k_hs, v_rs, v_hs, q_rs, q_hs, qo_rs, qo_hs;
  int R, d, rot;
  // a unit is a word of pairs (interleaved), a word of real parts with its partner of imaginary parts (half) or a word that
  // is copied; a thread's work is a unit of one or two heads: of a token Q's, from k_first on K's, from v_first on V's
  int turn_units, per_token, k_first, v_first, heads, Hq;
  FastDiv by_q, by_k, by_v;      // by the units of a head of each
};

// The first request whose end lies after token t (R: none), by a warp: ends of 32 parts at a time.
__device__ __forceinline__ int request_of(const int32_t* qsl, int R, int64_t t) {
  const int lane = threadIdx.x & 31;
  int r = 0;
  for (int n = R; n > 0;) {
    const int step = (n + 31) / 32, last = min((lane + 1) * step, n);
    const int before = min(__popc(__ballot_sync(0xffffffffu, qsl[r + last] <= t)) * step, n);
    n = min(step, n - before) - 1;   // the part's own end lies after t
    r += before;
  }
  return r;
}

// N values to a word, aligned to A bytes; P pairs to a unit that turns; GROUP threads, a warp or a block, to a token at a time.
template <typename T, int N, int A, bool INTER, bool AXES, int GROUP>
__global__ void __launch_bounds__(kAppendThreads, kAppendBlocks) append_kernel(const __grid_constant__ AppendParams p) {
  static_assert(GROUP == 32 || GROUP == kAppendThreads);
  using V = Vec<T, N, A>;
  constexpr int P = INTER ? N / 2 : N, kGroups = kAppendThreads / GROUP;
  __shared__ float2 all_turns[kGroups][kMaxPairs];
  const int half = p.rot / 2, tid = threadIdx.x % GROUP;
  float2* turns = all_turns[threadIdx.x / GROUP];   // (cos, sin) of pair i of unit u at i * turn_units + u
  const int64_t groups = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / GROUP;
  auto sync = [] {
    if constexpr (GROUP == 32) __syncwarp();
    else __syncthreads();
  };

  // A thread's work: unit e of heads h0 .. h0 + nh - 1 (nh = 0: none).
  struct Work {
    int what, e, h0, nh;
    bool turn_it;
    V a[kAppendHeads], b[kAppendHeads];
  };
  auto load = [&](Work& w, int64_t t, int i) {
    w.nh = 0;
    if (i >= p.per_token || t >= p.T) return;
    w.what = i < p.k_first ? 0 : i < p.v_first ? 1 : 2;
    w.h0 = (w.what == 0 ? p.by_q.div(i, w.e) : w.what == 1 ? p.by_k.div(i - p.k_first, w.e) : p.by_v.div(i - p.v_first, w.e)) *
           p.heads;
    w.nh = min((w.what == 0 ? p.Hq : p.c.Hkv) - w.h0, p.heads);
    w.turn_it = w.what < 2 && w.e < p.turn_units;
    const int64_t hs = w.what == 0 ? p.q_hs : w.what == 1 ? p.k_hs : p.v_hs;
    const T* x = (w.what == 0 ? static_cast<const T*>(p.q) + t * p.q_rs
                              : w.what == 1 ? static_cast<const T*>(p.k) + t * p.k_rs : static_cast<const T*>(p.v) + t * p.v_rs) +
                 w.h0 * hs + (w.what == 2 || w.turn_it ? w.e * N : p.rot + (w.e - p.turn_units) * N);
#pragma unroll
    for (int j = 0; j < kAppendHeads; ++j)
      if (j < w.nh) {
        w.a[j] = *reinterpret_cast<const V*>(x + j * hs);
        if (!INTER && w.turn_it) w.b[j] = *reinterpret_cast<const V*>(x + j * hs + half);
      }
  };
  // `row`: of the cache, for head 0 (-1: not stored); `live`: of a request
  auto store = [&](const Work& w, int64_t t, int64_t row, bool live) {
    if (w.nh == 0) return;
    T* y;
    int64_t hs;
    if (w.what == 0) {
      if (!live) return;
      y = static_cast<T*>(p.q_out) + t * p.qo_rs;
      hs = p.qo_hs;
    } else {
      if (row < 0) return;
      y = static_cast<T*>(w.what == 1 ? p.k_cache : p.v_cache) + row * p.d;
      hs = static_cast<int64_t>(p.c.bs) * p.d;
    }
    y += w.h0 * hs + (w.what == 2 || w.turn_it ? w.e * N : p.rot + (w.e - p.turn_units) * N);
    if (!w.turn_it) {
#pragma unroll
      for (int j = 0; j < kAppendHeads; ++j)
        if (j < w.nh) *reinterpret_cast<V*>(y + j * hs) = w.a[j];
      return;
    }
    float c[P], s[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 cs = turns[i * p.turn_units + w.e];
      c[i] = cs.x;
      s[i] = cs.y;
    }
#pragma unroll
    for (int j = 0; j < kAppendHeads; ++j) {
      if (j >= w.nh) break;
      float f[N], o[N];
      V v;
      unpack(w.a[j], f);
      if (INTER) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          o[2 * i % N] = turn_re(f[2 * i % N], f[(2 * i + 1) % N], c[i], s[i]);
          o[(2 * i + 1) % N] = turn_im(f[2 * i % N], f[(2 * i + 1) % N], c[i], s[i]);
        }
        pack(v, o);
        *reinterpret_cast<V*>(y + j * hs) = v;
      } else {
        float g[N], o2[N];
        unpack(w.b[j], g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          o[i] = turn_re(f[i], g[i], c[i % P], s[i % P]);
          o2[i] = turn_im(f[i], g[i], c[i % P], s[i % P]);
        }
        pack(v, o);
        *reinterpret_cast<V*>(y + j * hs) = v;
        pack(v, o2);
        *reinterpret_cast<V*>(y + j * hs + half) = v;
      }
    }
  };
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.R; i += kAppendThreads) {
      const int32_t begin = p.qsl[i], end = p.qsl[i + 1];
      if (begin < 0 || end < begin || end > p.T) ra_record_error(RA_ERR_DEVICE_BOUNDS, 700);
    }
  Work work;
  load(work, t, tid);
  for (; t < p.T; t += groups) {
    const int r = request_of(p.qsl, p.R, t);
    int64_t x = -1, row = -1;
    const bool live = r < p.R && t >= p.qsl[r];
    if (live) {
      x = static_cast<int64_t>(p.ctx[r]) - (p.qsl[r + 1] - t);
      if (x < 0 || x >= (int64_t(1) << 30) || x >= static_cast<int64_t>(p.c.max_vb) * p.c.V)
        ra_record_error(RA_ERR_DEVICE_BOUNDS, 701);
      else
        row = paged_row(p.c, r, static_cast<int>(x), 0, 702);
      if (p.turn_units > 0) {
        const bool in = x >= 0 && x < kPositionLimit;
        if (!p.positions && !in) ra_record_error(RA_ERR_DEVICE_BOUNDS, 703);
        const float place = in ? static_cast<float>(x) : 0.f;
        for (int i = tid; i < half; i += GROUP) {
          const float m = p.positions ? position_at(p.positions, (AXES ? p.axis[i] : 0) * p.T + t, 703) : place;
          float2 cs;
          turn(p, i, m, cs.x, cs.y);
          turns[i % P * p.turn_units + i / P] = cs;
        }
      }
    }
    sync();
    for (int i = tid; i < p.per_token; i += 2 * GROUP) {
      Work other;
      load(other, t, i + GROUP);
      store(work, t, row, live);
      if (i + 2 * GROUP < p.per_token) load(work, t, i + 2 * GROUP);
      else load(work, t + groups, tid);
      store(other, t, row, live);
    }
    sync();
  }
}

// Launches the kernel on words of N values aligned to A bytes.
template <typename T, int N, int A>
ra_status launch_append(AppendParams& p, int32_t Hq, bool inter, bool axes, cudaStream_t stream) {
  const int64_t Hkv = p.c.Hkv;
  p.turn_units = inter ? p.rot / N : p.rot / 2 / N;
  const bool q_moves = p.q && p.q != p.q_out;             // in place the rest of a head stays where it is
  const int64_t k_units = p.turn_units + (p.d - p.rot) / N, v_units = p.d / N;
  const int64_t q_units = p.q ? p.turn_units + (q_moves ? (p.d - p.rot) / N : 0) : 0;
  const bool by_warps = p.T > kBlockTokens;
  for (p.heads = kAppendHeads; p.heads > 1; p.heads /= 2) {
    const int64_t work = q_units * ra::ceil_div(Hq, p.heads) + (k_units + v_units) * ra::ceil_div(Hkv, p.heads);
    if (work >= (by_warps ? 32 : kAppendThreads)) break;
  }
  p.Hq = p.q ? Hq : 0;
  p.k_first = static_cast<int>(q_units * ra::ceil_div(p.Hq, p.heads));
  p.v_first = p.k_first + static_cast<int>(k_units * ra::ceil_div(Hkv, p.heads));
  p.per_token = p.v_first + static_cast<int>(v_units * ra::ceil_div(Hkv, p.heads));
  p.by_q = fast_div(std::max<int64_t>(1, q_units));
  p.by_k = fast_div(k_units);
  p.by_v = fast_div(v_units);
  const unsigned blocks = static_cast<unsigned>(
      std::min<int64_t>(152 * kAppendBlocks, by_warps ? ra::ceil_div(p.T, kAppendThreads / 32) : p.T));
  auto go = [&](auto in, auto ax) {
    constexpr bool I = decltype(in)::value, X = decltype(ax)::value;
    if (by_warps) append_kernel<T, N, A, I, X, 32><<<blocks, kAppendThreads, 0, stream>>>(p);
    else append_kernel<T, N, A, I, X, kAppendThreads><<<blocks, kAppendThreads, 0, stream>>>(p);
  };
  if constexpr (N % 2 == 0) {
    if (inter && axes) go(std::true_type{}, std::true_type{});
    if (inter && !axes) go(std::true_type{}, std::false_type{});
  }
  if (!inter && axes) go(std::false_type{}, std::true_type{});
  if (!inter && !axes) go(std::false_type{}, std::false_type{});
  RA_LAUNCH_CHECK("append_kernel");
  return RA_OK;
}

template <typename T>
ra_status launch_append_type(AppendParams& p, int32_t Hq, bool inter, bool axes, cudaStream_t stream) {
  constexpr int es = sizeof(T);
  // whole words: every address that is read or written as one is a multiple of its size
  auto words = [&](int bytes) {
    const int n = bytes / es;
    uint64_t m = reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v) | reinterpret_cast<uintptr_t>(p.q) |
                 reinterpret_cast<uintptr_t>(p.q_out) | reinterpret_cast<uintptr_t>(p.k_cache) |
                 reinterpret_cast<uintptr_t>(p.v_cache);
    if (p.T > 1) m |= static_cast<uint64_t>(p.k_rs * es) | static_cast<uint64_t>(p.v_rs * es);
    if (p.T > 1 && p.q) m |= static_cast<uint64_t>(p.q_rs * es) | static_cast<uint64_t>(p.qo_rs * es);
    if (p.c.Hkv > 1) m |= static_cast<uint64_t>(p.k_hs * es) | static_cast<uint64_t>(p.v_hs * es);
    if (p.q && Hq > 1) m |= static_cast<uint64_t>(p.q_hs * es) | static_cast<uint64_t>(p.qo_hs * es);
    return m % bytes == 0 && p.d % n == 0 && p.rot % n == 0 && (inter || (p.rot / 2) % n == 0);
  };
  if (words(16)) return launch_append<T, 16 / es, 16>(p, Hq, inter, axes, stream);
  if (words(8)) return launch_append<T, 8 / es, 8>(p, Hq, inter, axes, stream);
  // element by element: a pair to a unit (d is even here, the rows of the cache being 16-byte words)
  return inter ? launch_append<T, 2, es>(p, Hq, inter, axes, stream) : launch_append<T, 1, es>(p, Hq, inter, axes, stream);
}

}  // namespace

extern "C" ra_status ra_cp_rope_append(const void* k, int64_t k_row_stride, int64_t k_head_stride, const void* v,
                                       int64_t v_row_stride, int64_t v_head_stride, const void* q, int64_t q_row_stride,
                                       int64_t q_head_stride, void* q_out, int64_t q_out_row_stride,
                                       int64_t q_out_head_stride, void* k_cache, void* v_cache, const int32_t* block_table,
                                       const int32_t* query_start_loc, const int32_t* ctx_lens, int64_t T, int32_t R,
                                       int32_t Hq, int32_t Hkv, int32_t d, ra_dtype dt, int32_t block_size,
                                       int32_t interleave, int32_t pcp, int32_t dcp, int32_t max_vblocks, int64_t num_blocks,
                                       const int32_t* positions, int32_t n_axes, int32_t rot, ra_rope_style style,
                                       const double* inv_freq, const int32_t* axis, double mscale, ra_stream stream) {
  ra::clear_error();
  ra_status st = check_paged(R, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks);
  if (st != RA_OK) return st;
  RA_REQUIRE(dt == RA_BF16 || dt == RA_F32, "dtype must be RA_BF16 or RA_F32");
  RA_REQUIRE(d >= 1 && d <= 1024, "1 <= d <= 1024 required");
  RA_REQUIRE(!q || Hq >= 1, "Hq must be >= 1");
  RA_REQUIRE(static_cast<int64_t>(Hkv) * d < (int64_t(1) << 26) && (!q || static_cast<int64_t>(Hq) * d < (int64_t(1) << 26)),
             "heads * d must be below 2^26");   // the work of a token: 31 bits
  const int es = dt == RA_BF16 ? 2 : 4;
  if (d * es % 16 != 0) return ra::fail(RA_ERR_UNSUPPORTED, "d*elem_size must be a multiple of 16");
  RA_REQUIRE(T >= 0 && T < (int64_t(1) << 31), "T must be in [0, 2^31)");
  const int64_t lim = int64_t(1) << 40;
  auto strides = [&](int64_t a, int64_t b) { return a >= 0 && b >= 0 && a < lim && b < lim; };
  RA_REQUIRE(strides(k_row_stride, k_head_stride) && strides(v_row_stride, v_head_stride) &&
                 (!q || (strides(q_row_stride, q_head_stride) && strides(q_out_row_stride, q_out_head_stride))),
             "strides must be in [0, 2^40)");
  AppendParams p;
  if (inv_freq) {
    RA_REQUIRE(positions || n_axes == 1, "several axes need positions");
    if ((st = make_turns(p, d, rot, style, inv_freq, axis, n_axes, mscale, false)) != RA_OK) return st;
  } else {
    RA_REQUIRE(rot == 0, "rot must be 0 without inv_freq");
  }
  if (T == 0) return RA_OK;
  RA_REQUIRE(k && v && k_cache && v_cache && block_table && query_start_loc && ctx_lens && (!q || q_out), "NULL pointer");
  auto at = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  RA_REQUIRE((at(k) | at(v) | at(q) | at(q_out)) % es == 0, "k, v, q and q_out must be aligned to their elements");
  RA_REQUIRE(ra::aligned16(k_cache) && ra::aligned16(v_cache), "the caches must be 16-byte aligned");
  // [begin, end) of what each tensor spans
  struct Span {
    uintptr_t b, e;
  };
  auto span = [&](const void* x, int64_t rs, int64_t H, int64_t hs) {
    return Span{at(x), at(x) + es * ((T - 1) * rs + (H - 1) * hs + d)};
  };
  auto meet = [](const Span& a, const Span& b) { return a.b < b.e && b.b < a.e; };
  const int64_t cache_bytes = static_cast<int64_t>(pcp) * dcp * num_blocks * Hkv * block_size * d * es;
  const Span kc{at(k_cache), at(k_cache) + cache_bytes}, vc{at(v_cache), at(v_cache) + cache_bytes};
  const Span ks = span(k, k_row_stride, Hkv, k_head_stride), vs = span(v, v_row_stride, Hkv, v_head_stride);
  RA_REQUIRE(!meet(kc, vc) && !meet(ks, kc) && !meet(ks, vc) && !meet(vs, kc) && !meet(vs, vc),
             "k, v and the caches must not overlap");
  p.q = q;
  p.q_out = q ? q_out : nullptr;
  if (q) {
    RA_REQUIRE(apart(T, q_out_row_stride, Hq, q_out_head_stride, d), "the elements of q_out must not alias one another");
    const Span qs = span(q, q_row_stride, Hq, q_head_stride), qo = span(q_out, q_out_row_stride, Hq, q_out_head_stride);
    const bool same = q == q_out && (T == 1 || q_row_stride == q_out_row_stride) && (Hq == 1 || q_head_stride == q_out_head_stride);
    RA_REQUIRE(same || !meet(qs, qo), "q_out must be q itself with its strides or not overlap it");
    RA_REQUIRE(!meet(qs, kc) && !meet(qs, vc) && !meet(qo, kc) && !meet(qo, vc), "q and q_out must not overlap the caches");
    // Q's elements, turned in place, lie between K's and V's where they come out of one projection: by rows, each Q, K or V
    // as a whole, or by heads
    auto meets = [&](const void* x, int64_t rs, int64_t hs) {
      if (!ra::rows_meet(q_out, es * q_out_row_stride, es * ((Hq - 1) * q_out_head_stride + d), x, es * rs,
                         es * ((Hkv - 1) * hs + d), T))
        return false;
      if (hs != q_out_head_stride || hs <= 0 || (T > 1 && (rs != q_out_row_stride || rs % hs != 0))) return true;
      const int64_t step = es * hs, off = ((static_cast<int64_t>(at(x) - at(q_out)) % step) + step) % step;
      return off < es * d || off + es * d > step;
    };
    RA_REQUIRE(!meets(k, k_row_stride, k_head_stride) && !meets(v, v_row_stride, v_head_stride), "q_out must not overlap k and v");
  }
  p.c = make_paged(block_table, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks);
  p.k = k; p.v = v; p.k_cache = k_cache; p.v_cache = v_cache;
  p.k_rs = k_row_stride; p.k_hs = k_head_stride; p.v_rs = v_row_stride; p.v_hs = v_head_stride;
  p.q_rs = q_row_stride; p.q_hs = q_head_stride; p.qo_rs = q_out_row_stride; p.qo_hs = q_out_head_stride;
  p.qsl = query_start_loc; p.ctx = ctx_lens; p.positions = positions;
  p.T = T; p.R = R; p.d = d; p.rot = inv_freq ? rot : 0;
  const bool inter = inv_freq && style == RA_ROPE_INTERLEAVED;
  return dt == RA_BF16 ? launch_append_type<__nv_bfloat16>(p, Hq, inter, inv_freq && axis, stream)
                       : launch_append_type<float>(p, Hq, inter, inv_freq && axis, stream);
}
