// New tokens' K and V on their way into the sharded paged cache, K (and Q beside
// it) turned by the rotary positions as they pass.
//
// Mathematics.  Token i of request r is the context's token x = ctx_r - n_r + i:
// K[x] = mscale * Rot(pos) k, V[x] = v, q_out = mscale * Rot(pos) q, with the
// rotation of ra_rope_turn.cuh and the place of x of ra_paged.cuh.
//
// One launch in place of four (the rotation of Q, that of K, the slot mapping, the
// scatter), so that K passes through the chip once.  A thread owns a "unit" of a
// token, a word of pairs (interleaved), a word of real parts with its partner of
// imaginary parts (half) or a word that is copied, for up to 8 of Q's, K's or V's
// heads: it issues all their loads, finds the token's request, place and angles
// meanwhile, and then turns and stores each head.
#include <algorithm>
#include <type_traits>

#include "ra_paged.cuh"
#include "ra_rope_turn.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_rope_append)

namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendHeads = 8;   // heads of a thread, at most

struct AppendParams : Turns {
  Paged c;
  const void *k, *v, *q;
  void *k_cache, *v_cache, *q_out;
  const int32_t *qsl, *ctx;
  const int32_t* positions;      // of axis a: positions + a * T; NULL: the token's place in its context
  int64_t T, k_rs, k_hs, v_rs, v_hs, q_rs, q_hs, qo_rs, qo_hs;
  int64_t t0;                    // tokens t0 .. t0 + n_t - 1 of this launch
  int R, Hq, d, rot, n_t;
  int turn_units, per_token, k_first, v_first, heads;   // threads of a token: Q's, from k_first on K's, from v_first on V's
  FastDiv by_token, by_q, by_k, by_v;                   // by the threads of a token, the units of a head of each
};

template <typename T, int N, int A>
struct alignas(A) Vec {
  T x[N];
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float& y, float x) { y = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// N values to a word, aligned to A bytes; P pairs to a unit that turns.
template <typename T, int N, int A, bool INTER, bool AXES>
__global__ void __launch_bounds__(kAppendThreads, 2) append_kernel(const __grid_constant__ AppendParams p) {
  using V = Vec<T, N, A>;
  constexpr int P = INTER ? N / 2 : N;
  const uint32_t w = blockIdx.x * kAppendThreads + threadIdx.x;
  const bool used = w < static_cast<uint32_t>(p.n_t) * p.per_token;
  int sub = 0;
  const int64_t t = p.t0 + (used ? p.by_token.div(static_cast<int>(w), sub) : 0);
  // Q, K or V, the unit of a head and the first head
  const int what = sub < p.k_first ? 0 : sub < p.v_first ? 1 : 2;
  int u;
  const int h0 = (what == 0 ? p.by_q.div(sub, u) : what == 1 ? p.by_k.div(sub - p.k_first, u) : p.by_v.div(sub - p.v_first, u)) * p.heads;
  const int nh = min((what == 0 ? p.Hq : p.c.Hkv) - h0, p.heads);
  const bool turns = what < 2 && u < p.turn_units;
  const int half = p.rot / 2;
  const int e0 = what == 2 ? u * N : turns ? u * N : p.rot + (u - p.turn_units) * N;
  const int64_t rs = what == 0 ? p.q_rs : what == 1 ? p.k_rs : p.v_rs, hs = what == 0 ? p.q_hs : what == 1 ? p.k_hs : p.v_hs;
  const T* x = static_cast<const T*>(what == 0 ? p.q : what == 1 ? p.k : p.v) + t * rs + h0 * hs + e0;
  V a[kAppendHeads], b[kAppendHeads];
  if (used) {
#pragma unroll
    for (int j = 0; j < kAppendHeads; ++j)
      if (j < nh) {
        a[j] = *reinterpret_cast<const V*>(x + j * hs);
        if (!INTER && turns) b[j] = *reinterpret_cast<const V*>(x + j * hs + half);
      }
  }
  // the request of the block's first token, by all threads together; from there each thread walks to its own
  const int64_t first = p.t0 + p.by_token.div(static_cast<int>(blockIdx.x * kAppendThreads));
  int r = 0;
  for (int base = 0; base < p.R; base += kAppendThreads) {
    const int i = base + threadIdx.x;
    int32_t end = INT32_MAX;
    if (i < p.R) {
      end = p.qsl[i + 1];
      if (blockIdx.x == 0 && p.t0 == 0) {
        const int32_t begin = p.qsl[i];
        if (begin < 0 || end < begin || end > p.T) ra_record_error(RA_ERR_DEVICE_BOUNDS, 700);
      }
    }
    r += __syncthreads_count(i < p.R && end <= first);
  }
  if (!used) return;
  while (r < p.R && p.qsl[r + 1] <= t) ++r;
  if (r >= p.R || t < p.qsl[r]) return;   // a token of no request
  const int64_t place = static_cast<int64_t>(p.ctx[r]) - (p.qsl[r + 1] - t);
  T* y;
  int64_t yhs;
  if (what == 0) {
    y = static_cast<T*>(p.q_out) + t * p.qo_rs + h0 * p.qo_hs + e0;
    yhs = p.qo_hs;
  } else {
    if (place < 0 || place >= (int64_t(1) << 30) || place >= static_cast<int64_t>(p.c.max_vb) * p.c.V) {
      ra_record_error(RA_ERR_DEVICE_BOUNDS, 701);
      return;
    }
    const int64_t row = paged_row(p.c, r, static_cast<int>(place), h0, 702);
    if (row < 0) return;
    y = static_cast<T*>(what == 1 ? p.k_cache : p.v_cache) + row * p.d + e0;
    yhs = static_cast<int64_t>(p.c.bs) * p.d;
  }
  float c[P], s[P];
  if (turns) {
    float m = 0.f;
    int last = -1;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int ax = AXES ? p.axis[u * P + i] : 0;
      if (ax != last) {
        if (p.positions) {
          m = position_at(p.positions, ax * p.T + t, 703);
        } else if (place < 0 || place >= kPositionLimit) {
          ra_record_error(RA_ERR_DEVICE_BOUNDS, 703);
        } else {
          m = static_cast<float>(place);
        }
      }
      last = ax;
      turn(p, u * P + i, m, c[i], s[i]);
    }
  }
#pragma unroll
  for (int j = 0; j < kAppendHeads; ++j) {
    if (j >= nh) break;
    T* out = y + j * yhs;
    if (!turns) {
      *reinterpret_cast<V*>(out) = a[j];
      continue;
    }
    V o, o2;
    if (INTER) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float re = to_float(a[j].x[2 * i]), im = to_float(a[j].x[2 * i + 1]);
        from_float(o.x[2 * i], turn_re(re, im, c[i], s[i]));
        from_float(o.x[2 * i + 1], turn_im(re, im, c[i], s[i]));
      }
      *reinterpret_cast<V*>(out) = o;
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float re = to_float(a[j].x[i]), im = to_float(b[j].x[i]);
        from_float(o.x[i], turn_re(re, im, c[i], s[i]));
        from_float(o2.x[i], turn_im(re, im, c[i], s[i]));
      }
      *reinterpret_cast<V*>(out) = o;
      *reinterpret_cast<V*>(out + half) = o2;
    }
  }
}

// Launches the kernel on words of N values aligned to A bytes; more than 2^31 threads in several launches.
template <typename T, int N, int A>
ra_status launch_append(AppendParams& p, bool inter, bool axes, cudaStream_t stream) {
  const int Hkv = p.c.Hkv;
  p.turn_units = inter ? p.rot / N : p.rot / 2 / N;
  const bool q_moves = p.q && p.q != p.q_out;             // in place the rest of a head stays where it is
  const int k_units = p.turn_units + (p.d - p.rot) / N, q_units = p.q ? p.turn_units + (q_moves ? (p.d - p.rot) / N : 0) : 0;
  const int v_units = p.d / N;
  // Heads of a thread: 8 where that leaves about 1024 threads to each SM, else fewer for latency.
  const int64_t want = 152 * 1024;
  int64_t per = 0;
  for (p.heads = kAppendHeads;; p.heads /= 2) {
    per = q_units * ra::ceil_div(p.Hq, p.heads) + (static_cast<int64_t>(k_units) + v_units) * ra::ceil_div(Hkv, p.heads);
    if (p.heads == 1 || p.T * per >= want) break;
  }
  p.per_token = static_cast<int>(per);
  p.k_first = static_cast<int>(q_units * ra::ceil_div(p.Hq, p.heads));
  p.v_first = p.k_first + static_cast<int>(k_units * ra::ceil_div(Hkv, p.heads));
  p.by_token = fast_div(per);
  p.by_q = fast_div(std::max(1, q_units));
  p.by_k = fast_div(k_units);
  p.by_v = fast_div(v_units);
  const int64_t most = ((int64_t(1) << 31) - kAppendThreads) / per;
  for (p.t0 = 0; p.t0 < p.T; p.t0 += most) {
    p.n_t = static_cast<int>(std::min(most, p.T - p.t0));
    const unsigned blocks = static_cast<unsigned>(ra::ceil_div(p.n_t * per, kAppendThreads));
    auto go = [&](auto in, auto ax) {
      append_kernel<T, N, A, decltype(in)::value, decltype(ax)::value><<<blocks, kAppendThreads, 0, stream>>>(p);
    };
    if constexpr (N % 2 == 0) {
      if (inter && axes) go(std::true_type{}, std::true_type{});
      if (inter && !axes) go(std::true_type{}, std::false_type{});
    }
    if (!inter && axes) go(std::false_type{}, std::true_type{});
    if (!inter && !axes) go(std::false_type{}, std::false_type{});
    RA_LAUNCH_CHECK("append_kernel");
  }
  return RA_OK;
}

template <typename T>
ra_status launch_append_type(AppendParams& p, bool inter, bool axes, cudaStream_t stream) {
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
    if (p.q && p.Hq > 1) m |= static_cast<uint64_t>(p.q_hs * es) | static_cast<uint64_t>(p.qo_hs * es);
    return m % bytes == 0 && p.d % n == 0 && p.rot % n == 0 && (inter || (p.rot / 2) % n == 0);
  };
  if (words(16)) return launch_append<T, 16 / es, 16>(p, inter, axes, stream);
  if (words(8)) return launch_append<T, 8 / es, 8>(p, inter, axes, stream);
  // element by element: a pair to a unit (d is even here, the rows of the cache being 16-byte words)
  return inter ? launch_append<T, 2, es>(p, inter, axes, stream) : launch_append<T, 1, es>(p, inter, axes, stream);
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
  RA_REQUIRE(static_cast<int64_t>(Hkv) * d < (int64_t(1) << 29) && (!q || static_cast<int64_t>(Hq) * d < (int64_t(1) << 29)),
             "heads * d must be below 2^29");   // threads of a token: 32 bits
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
    // in place Q's elements lie between K's and V's where they come out of one projection: no element is in two of them
    if (!same) RA_REQUIRE(!meet(qo, ks) && !meet(qo, vs), "q_out must not overlap k and v");
  }
  p.c = make_paged(block_table, Hkv, block_size, interleave, pcp, dcp, max_vblocks, num_blocks);
  p.k = k; p.v = v; p.k_cache = k_cache; p.v_cache = v_cache;
  p.k_rs = k_row_stride; p.k_hs = k_head_stride; p.v_rs = v_row_stride; p.v_hs = v_head_stride;
  p.q_rs = q_row_stride; p.q_hs = q_head_stride; p.qo_rs = q_out_row_stride; p.qo_hs = q_out_head_stride;
  p.qsl = query_start_loc; p.ctx = ctx_lens; p.positions = positions;
  p.T = T; p.R = R; p.Hq = q ? Hq : 1; p.d = d; p.rot = inv_freq ? rot : 0;
  const bool inter = inv_freq && style == RA_ROPE_INTERLEAVED;
  return dt == RA_BF16 ? launch_append_type<__nv_bfloat16>(p, inter, inv_freq && axis, stream)
                       : launch_append_type<float>(p, inter, inv_freq && axis, stream);
}
