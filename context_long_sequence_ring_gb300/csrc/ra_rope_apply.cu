// Rotary positions on strided rows: both pairings, part of the head, any
// frequency table, and the gradient direction.
//
// Mathematics.  Pair i of a row at position m is turned by the angle
// m * f_i: (a, b) -> mscale * (a cos - b sin, b cos + a sin).  The backward
// direction is the transposed rotation, i.e. the angle -m * f_i.
// Angles are taken in turns, m * phi_i with phi_i = f_i / 2 pi held as an
// unevaluated sum of two floats.  m * hi is split exactly into p + e with one
// FMA, the whole turns rint(p) drop out exactly, and the rest goes to
// sincospif: the angle error is about 1e-7 turns at any position below 2^24.
#include <algorithm>
#include <cmath>

#include "ra_paged.cuh"

RA_DEFINE_ERROR_FETCH(fetch_error_rope_apply)

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;           // rot <= 256
constexpr int kPositionLimit = 1 << 24;  // positions are exact in a float below this

struct Params {
  const void* src;
  void* dst;
  const int32_t* idx;
  const int32_t* positions;
  int64_t src_rows, src_rs, src_hs, dst_rs, dst_hs, rows;
  int32_t H, d, rot;
  // rows of whole words: rows row0 .. row0 + row_end of this launch, threads of a row, its units that turn,
  // heads of a thread
  int64_t row0;
  int32_t row_end, per_row, turn_units, heads;
  FastDiv by_units, by_groups;
  float mscale, sign;
  float2 phase[kMaxPairs];  // phi_i as hi + lo
};

// mscale * cos and mscale * sin (signed by the direction) of pair i at position m.
__device__ __forceinline__ void turn(const Params& p, int i, float m, float& c, float& s) {
  const float2 ph = p.phase[i];
  const float t = m * ph.x;
  const float err = fmaf(m, ph.x, -t);           // m * hi = t + err exactly
  const float f = (t - rintf(t)) + fmaf(m, ph.y, err);
  sincospif(2.0f * f, &s, &c);
  c *= p.mscale;
  s *= p.mscale * p.sign;
}

// Source row of output row r; -1 for a zero row.
__device__ __forceinline__ int64_t source_row(const Params& p, int64_t r) {
  if (!p.idx) return r;
  const int32_t s = p.idx[r];
  if (s >= p.src_rows) {
    ra_record_error(RA_ERR_DEVICE_BOUNDS, 400);
    return -1;
  }
  return s;
}

__device__ __forceinline__ float position(const Params& p, int64_t r) {
  const int32_t m = p.positions[r];
  if (m < 0 || m >= kPositionLimit) {
    ra_record_error(RA_ERR_DEVICE_BOUNDS, 401);
    return 0.f;
  }
  return static_cast<float>(m);
}

__device__ __forceinline__ float load1(const __nv_bfloat16* x) { return __bfloat162float(*x); }
__device__ __forceinline__ float load1(const float* x) { return *x; }
__device__ __forceinline__ void store1(__nv_bfloat16* x, float v) { *x = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* x, float v) { *x = v; }

// A word of 16 or 8 bytes as fp32 values, and back (rounded to nearest even).
template <typename T, typename W> struct Word;
template <typename W> struct Word<float, W> {
  static constexpr int N = sizeof(W) / 4;
  __device__ static void unpack(const W& u, float (&f)[N]) {
    const float* x = reinterpret_cast<const float*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = x[i];
  }
  __device__ static W pack(const float (&f)[N]) {
    W u;
    float* x = reinterpret_cast<float*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = f[i];
    return u;
  }
};
template <typename W> struct Word<__nv_bfloat16, W> {
  static constexpr int N = sizeof(W) / 2;
  __device__ static void unpack(const W& u, float (&f)[N]) {
    const uint32_t* x = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      f[2 * i] = __uint_as_float(x[i] << 16);
      f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
    }
  }
  __device__ static W pack(const float (&f)[N]) {
    W u;
    uint32_t* x = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      x[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return u;
  }
};

// The turned pair: real and imaginary part.  One form for all kernels, so that they agree to the bit.
__device__ __forceinline__ float turn_re(float a, float b, float c, float s) { return fmaf(a, c, -__fmul_rn(b, s)); }
__device__ __forceinline__ float turn_im(float a, float b, float c, float s) { return fmaf(b, c, __fmul_rn(a, s)); }

constexpr int kHeads = 8;   // heads of a thread, at most

// Rows of whole words.  A "unit" of a head is one word of pairs (interleaved),
// a word of real parts and its partner word of imaginary parts (half), or a word
// past rot, which is copied.  A thread owns a unit for up to 8 heads of a row:
// it issues all their loads, forms the unit's angles meanwhile and applies them to each head.
// Bound by HBM, a row being read and written once: 32768 rows of 40 heads of 128
// in bf16 (half) take 99 us, 6.8 TB/s, the rate of a plain copy.  4 heads a thread:
// 103 us; all 40 in a loop that has 8 in flight: 140 us, since a thread's loads then
// wait for its stores.
template <typename T, typename W, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) rope_words_kernel(const __grid_constant__ Params p) {
  using V = Word<T, W>;
  constexpr int N = V::N, P = INTER ? N / 2 : N;      // values of a word, pairs of a unit
  const uint32_t w = blockIdx.x * kThreads + threadIdx.x;   // (row, head group, unit)
  if (w >= static_cast<uint32_t>(p.row_end) * p.per_row) return;
  int u, group;
  const int r32 = p.by_units.div(static_cast<int>(w), u);
  const int64_t r = p.row0 + p.by_groups.div(r32, group);
  const int64_t s = source_row(p, r);
  const bool turns = u < p.turn_units;
  const int e0 = turns ? u * N : p.rot + (u - p.turn_units) * N;
  const int h0 = group * p.heads;
  T* y = static_cast<T*>(p.dst) + r * p.dst_rs + h0 * p.dst_hs + e0;
  const T* x = static_cast<const T*>(p.src) + (s < 0 ? 0 : s) * p.src_rs + h0 * p.src_hs + e0;
  const int half = p.rot / 2;
  const int nh = min(p.H - h0, p.heads);
  W a[kHeads], b[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j)
    if (j < nh && s >= 0) {
      a[j] = *reinterpret_cast<const W*>(x + j * p.src_hs);
      if (!INTER && turns) b[j] = *reinterpret_cast<const W*>(x + j * p.src_hs + half);
    }
  float c[P], sn[P];
  if (s >= 0 && turns) {
    const float m = position(p, r);
#pragma unroll
    for (int i = 0; i < P; ++i) turn(p, u * P + i, m, c[i], sn[i]);
  }
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    if (j >= nh) break;
    T* out = y + j * p.dst_hs;
    if (s < 0) a[j] = b[j] = W{};
    if (s < 0 || !turns) {
      *reinterpret_cast<W*>(out) = a[j];
      if (!INTER && turns) *reinterpret_cast<W*>(out + half) = b[j];
      continue;
    }
    float f[N], o[N];
    V::unpack(a[j], f);
    if (INTER) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        o[2 * i] = turn_re(f[2 * i], f[2 * i + 1], c[i], sn[i]);
        o[2 * i + 1] = turn_im(f[2 * i], f[2 * i + 1], c[i], sn[i]);
      }
      *reinterpret_cast<W*>(out) = V::pack(o);
    } else {
      float f2[N], o2[N];
      V::unpack(b[j], f2);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        o[i] = turn_re(f[i], f2[i], c[i], sn[i]);
        o2[i] = turn_im(f[i], f2[i], c[i], sn[i]);
      }
      *reinterpret_cast<W*>(out) = V::pack(o);
      *reinterpret_cast<W*>(out + half) = V::pack(o2);
    }
  }
}

// Element-wise form for any stride and alignment: one thread per (row, unit),
// units 0 .. rot/2-1 the pairs, the others the elements past rot.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const __grid_constant__ Params p) {
  const int half = p.rot / 2;
  const int units = half + (p.d - p.rot);
  const int64_t total = p.rows * units;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; w < total; w += stride) {
    const int64_t r = w / units;
    const int u = static_cast<int>(w - r * units);
    const int64_t s = source_row(p, r);
    const bool pair = u < half;
    const int e0 = pair ? (INTER ? 2 * u : u) : p.rot + (u - half);
    const int e1 = INTER ? e0 + 1 : e0 + half;
    float c = 1.f, sn = 0.f;
    if (pair && s >= 0) turn(p, u, position(p, r), c, sn);
    const T* x = static_cast<const T*>(p.src) + s * p.src_rs;
    T* y = static_cast<T*>(p.dst) + r * p.dst_rs;
    for (int h = 0; h < p.H; ++h, x += p.src_hs, y += p.dst_hs) {
      if (!pair) {
        y[e0] = s >= 0 ? x[e0] : T(0.f);
        continue;
      }
      const float a = s >= 0 ? load1(x + e0) : 0.f, b = s >= 0 ? load1(x + e1) : 0.f;
      store1(y + e0, turn_re(a, b, c, sn));
      store1(y + e1, turn_im(a, b, c, sn));
    }
  }
}

// Launches the kernel on rows of words W; more than 2^31 threads in several launches.
template <typename T, typename W>
ra_status launch_words(Params& p, bool inter, cudaStream_t stream) {
  constexpr int N = Word<T, W>::N;
  p.turn_units = inter ? p.rot / N : p.rot / 2 / N;
  const bool copies = p.src != p.dst;                   // in place the rest of a head stays where it is
  const int units = p.turn_units + (copies ? (p.d - p.rot) / N : 0);
  // Heads of a thread: 8 where that leaves about 1024 threads to each SM, else as few as it takes for latency
  // (64 rows of 40 heads: 2.4 us with one or two heads a thread, 3.2 with 8).
  const int64_t want = 152 * 1024;
  int64_t groups = std::min<int64_t>(p.H, std::max(ra::ceil_div(p.H, kHeads), ra::ceil_div(want, p.rows * units)));
  p.heads = static_cast<int32_t>(ra::ceil_div(p.H, groups));
  groups = ra::ceil_div(p.H, p.heads);
  p.by_units = fast_div(units);
  p.by_groups = fast_div(groups);
  p.per_row = static_cast<int32_t>(units * groups);
  const int64_t rows = p.rows, most = ((int64_t(1) << 31) - kThreads) / p.per_row;
  for (p.row0 = 0; p.row0 < rows; p.row0 += most) {
    p.row_end = static_cast<int32_t>(std::min(most, rows - p.row0));
    const unsigned blocks = static_cast<unsigned>(ra::ceil_div(static_cast<int64_t>(p.row_end) * p.per_row, kThreads));
    if (inter) rope_words_kernel<T, W, true><<<blocks, kThreads, 0, stream>>>(p);
    else rope_words_kernel<T, W, false><<<blocks, kThreads, 0, stream>>>(p);
    RA_LAUNCH_CHECK("rope_words_kernel");
  }
  return RA_OK;
}

// Whether the elements of [rows, H, d] at these strides are all apart.
bool apart(int64_t rows, int64_t rs, int64_t H, int64_t hs, int64_t d) {
  if (rows > 1 && H > 1)
    return (hs >= d && rs >= (H - 1) * hs + d) || (rs >= d && hs >= (rows - 1) * rs + d);
  return (rows <= 1 || rs >= d) && (H <= 1 || hs >= d);
}

}  // namespace

extern "C" ra_status ra_rope_apply(const void* src, int64_t src_rows, int64_t src_row_stride,
                                   int64_t src_head_stride, void* dst, int64_t dst_row_stride,
                                   int64_t dst_head_stride, int64_t rows, int32_t H, int32_t d, int32_t rot,
                                   ra_dtype dt, ra_rope_style style, const int32_t* idx, const int32_t* positions,
                                   const double* inv_freq, double mscale, int32_t backward, ra_stream stream) {
  ra::clear_error();
  RA_REQUIRE(dt == RA_BF16 || dt == RA_F32, "dtype must be RA_BF16 or RA_F32");
  RA_REQUIRE(style == RA_ROPE_HALF || style == RA_ROPE_INTERLEAVED, "unknown rope style");
  RA_REQUIRE(H >= 1 && d >= 1 && d <= 1024, "H >= 1 and 1 <= d <= 1024 required");
  RA_REQUIRE(static_cast<int64_t>(H) * d < (int64_t(1) << 31), "H*d must be below 2^31");   // threads of a row: 32 bits
  RA_REQUIRE(rot >= 2 && rot % 2 == 0 && rot <= d && rot <= 2 * kMaxPairs, "rot must be even, in [2, min(d, %d)]",
             2 * kMaxPairs);
  RA_REQUIRE(rows >= 0 && src_rows >= 0, "negative size");
  RA_REQUIRE(idx || rows == src_rows, "without idx, rows must equal src_rows");
  const int64_t lim = int64_t(1) << 40;
  RA_REQUIRE(src_row_stride >= 0 && src_head_stride >= 0 && dst_row_stride >= 0 && dst_head_stride >= 0 &&
                 src_row_stride < lim && src_head_stride < lim && dst_row_stride < lim && dst_head_stride < lim &&
                 rows < (int64_t(1) << 31) && src_rows < (int64_t(1) << 31),
             "strides must be in [0, 2^40), rows in [0, 2^31)");
  RA_REQUIRE(inv_freq != nullptr && std::isfinite(mscale), "inv_freq must be given and mscale finite");
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < rot / 2; ++i)
    RA_REQUIRE(std::fabs(inv_freq[i]) <= two_pi, "inv_freq[%d] must be in [-2 pi, 2 pi]", i);
  if (rows == 0) return RA_OK;
  RA_REQUIRE(src && dst && positions, "NULL pointer");
  RA_REQUIRE(apart(rows, dst_row_stride, H, dst_head_stride, d), "the elements of dst must not alias one another");
  const int es = dt == RA_BF16 ? 2 : 4;
  const uintptr_t s0 = reinterpret_cast<uintptr_t>(src), d0 = reinterpret_cast<uintptr_t>(dst);
  RA_REQUIRE((s0 | d0) % es == 0, "src and dst must be aligned to their elements");
  const bool same = src == dst && (rows == 1 || src_row_stride == dst_row_stride) &&
                    (H == 1 || src_head_stride == dst_head_stride);
  if (idx || !same) {
    const uintptr_t s1 =
        s0 + es * (std::max<int64_t>(src_rows - 1, 0) * src_row_stride + (H - 1) * src_head_stride + d);
    const uintptr_t d1 = d0 + es * ((rows - 1) * dst_row_stride + (H - 1) * dst_head_stride + d);
    RA_REQUIRE(d1 <= s0 || s1 <= d0, "dst must be src itself with its strides (without idx) or not overlap it");
  }

  Params p;
  p.src = src; p.dst = dst; p.idx = idx; p.positions = positions;
  p.src_rows = src_rows; p.src_rs = src_row_stride; p.src_hs = src_head_stride;
  p.dst_rs = dst_row_stride; p.dst_hs = dst_head_stride; p.rows = rows;
  p.H = H; p.d = d; p.rot = rot;
  p.mscale = static_cast<float>(mscale);
  p.sign = backward ? -1.f : 1.f;
  for (int i = 0; i < kMaxPairs; ++i) {
    const double phi = i < rot / 2 ? inv_freq[i] / two_pi : 0.0;
    const float hi = static_cast<float>(phi);
    p.phase[i] = make_float2(hi, static_cast<float>(phi - static_cast<double>(hi)));
  }
  // whole words: every address that is read or written as one is a multiple of its size
  auto words = [&](int bytes) {
    const int n = bytes / es;
    uint64_t m = s0 | d0;
    if (rows > 1 || idx) m |= static_cast<uint64_t>(src_row_stride * es) | static_cast<uint64_t>(dst_row_stride * es);
    if (H > 1) m |= static_cast<uint64_t>(src_head_stride * es) | static_cast<uint64_t>(dst_head_stride * es);
    return m % bytes == 0 && d % n == 0 && rot % n == 0 && (style == RA_ROPE_INTERLEAVED || (rot / 2) % n == 0);
  };
  if (words(16))
    return dt == RA_BF16 ? launch_words<__nv_bfloat16, uint4>(p, style == RA_ROPE_INTERLEAVED, stream)
                         : launch_words<float, uint4>(p, style == RA_ROPE_INTERLEAVED, stream);
  if (words(8))
    return dt == RA_BF16 ? launch_words<__nv_bfloat16, uint2>(p, style == RA_ROPE_INTERLEAVED, stream)
                         : launch_words<float, uint2>(p, style == RA_ROPE_INTERLEAVED, stream);
  const int64_t units = rot / 2 + (d - rot);
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(ra::ceil_div(rows * units, kThreads), 152 * 64));
  const bool inter = style == RA_ROPE_INTERLEAVED;
  if (dt == RA_BF16) {
    if (inter) rope_any_kernel<__nv_bfloat16, true><<<blocks, kThreads, 0, stream>>>(p);
    else rope_any_kernel<__nv_bfloat16, false><<<blocks, kThreads, 0, stream>>>(p);
  } else {
    if (inter) rope_any_kernel<float, true><<<blocks, kThreads, 0, stream>>>(p);
    else rope_any_kernel<float, false><<<blocks, kThreads, 0, stream>>>(p);
  }
  RA_LAUNCH_CHECK("rope_any_kernel");
  return RA_OK;
}

extern "C" ra_status ra_rope_frequencies(ra_rope_scaling scaling, double base, int32_t rot, double factor,
                                         double trained_len, double* inv_freq, double* mscale) {
  ra::clear_error();
  RA_REQUIRE(scaling >= RA_ROPE_NONE && scaling <= RA_ROPE_YARN, "unknown scaling");
  RA_REQUIRE(base > 1.0 && std::isfinite(base), "base must be finite and > 1");
  RA_REQUIRE(rot >= 2 && rot % 2 == 0 && rot <= 2 * kMaxPairs, "rot must be even, in [2, %d]", 2 * kMaxPairs);
  RA_REQUIRE(factor >= 1.0 && std::isfinite(factor), "factor must be finite and >= 1");
  RA_REQUIRE(scaling != RA_ROPE_YARN || (trained_len >= 1.0 && std::isfinite(trained_len)),
             "trained_len must be finite and >= 1");
  RA_REQUIRE(scaling != RA_ROPE_NTK || rot > 2, "RA_ROPE_NTK needs rot > 2");
  RA_REQUIRE(inv_freq != nullptr, "inv_freq is NULL");
  const double two_pi = 6.283185307179586476925286766559;
  const double b = scaling == RA_ROPE_NTK ? base * std::pow(factor, static_cast<double>(rot) / (rot - 2)) : base;
  RA_REQUIRE(std::isfinite(b), "base * factor^(rot/(rot-2)) overflows");
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rot);
    if (scaling == RA_ROPE_LINEAR) f /= factor;
    if (scaling == RA_ROPE_YARN) {
      const double turns = trained_len * f / two_pi;
      const double g = std::min(1.0, std::max(0.0, (turns - 1.0) / 31.0));
      f = (1.0 - g) * f / factor + g * f;
    }
    inv_freq[i] = f;
  }
  if (mscale) *mscale = scaling == RA_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return RA_OK;
}
