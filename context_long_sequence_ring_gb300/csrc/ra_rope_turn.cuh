// Rotary positions as the kernels apply them: the angles of a table of
// frequencies and the turned pair.  One form for all kernels, so that they agree to the bit.
//
// Angles are taken in turns, m * phi_i with phi_i = f_i / 2 pi held as an
// unevaluated sum of two floats.  m * hi is split exactly into p + e with one
// FMA, the whole turns rint(p) drop out exactly, and the rest goes to
// sincospif: the angle error is about 1e-7 turns at any position below 2^24.
#pragma once

#include <cmath>

#include "ra_common.cuh"

namespace {

constexpr int kMaxPairs = 128;           // rot <= 256
constexpr int kPositionLimit = 1 << 24;  // positions are exact in a float below this
constexpr int kMaxAxes = 16;

struct Turns {
  float mscale, sign;
  float2 phase[kMaxPairs];    // phi_i as hi + lo
  uint8_t axis[kMaxPairs];    // whose position turns pair i
};

// mscale * cos and mscale * sin (signed by the direction) of pair i at position m.
__device__ __forceinline__ void turn(const Turns& p, int i, float m, float& c, float& s) {
  const float2 ph = p.phase[i];
  const float t = m * ph.x;
  const float err = fmaf(m, ph.x, -t);           // m * hi = t + err exactly
  const float f = (t - rintf(t)) + fmaf(m, ph.y, err);
  sincospif(2.0f * f, &s, &c);
  c *= p.mscale;
  s *= p.mscale * p.sign;
}

// The turned pair: real and imaginary part.
__device__ __forceinline__ float turn_re(float a, float b, float c, float s) { return fmaf(a, c, -__fmul_rn(b, s)); }
__device__ __forceinline__ float turn_im(float a, float b, float c, float s) { return fmaf(b, c, __fmul_rn(a, s)); }

// N values aligned to A bytes, and as fp32 ones (rounded to nearest even on the way back).
template <typename T, int N, int A>
struct alignas(A) Vec {
  T x[N];
};
template <int N, int A>
__device__ __forceinline__ void unpack(const Vec<float, N, A>& v, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = v.x[i];
}
template <int N, int A>
__device__ __forceinline__ void pack(Vec<float, N, A>& v, const float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v.x[i] = f[i];
}
template <int N, int A>
__device__ __forceinline__ void unpack(const Vec<__nv_bfloat16, N, A>& v, float (&f)[N]) {
  if constexpr (A >= 4) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __bfloat162float(v.x[i]);
  }
}
template <int N, int A>
__device__ __forceinline__ void pack(Vec<__nv_bfloat16, N, A>& v, const float (&f)[N]) {
  if constexpr (A >= 4) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v.x[i] = __float2bfloat16_rn(f[i]);
  }
}

// A position as a float; 0 where it is out of range.
__device__ __forceinline__ float position_at(const int32_t* positions, int64_t at, int site) {
  const int32_t m = positions[at];
  if (m < 0 || m >= kPositionLimit) {
    ra_record_error(RA_ERR_DEVICE_BOUNDS, site);
    return 0.f;
  }
  return static_cast<float>(m);
}

// Host checks of the rotation itself, and its table.  axis NULL: one axis.
inline ra_status make_turns(Turns& p, int32_t d, int32_t rot, ra_rope_style style, const double* inv_freq, const int32_t* axis,
                            int32_t n_axes, double mscale, bool backward) {
  RA_REQUIRE(style == RA_ROPE_HALF || style == RA_ROPE_INTERLEAVED, "unknown rope style");
  RA_REQUIRE(rot >= 2 && rot % 2 == 0 && rot <= d && rot <= 2 * kMaxPairs, "rot must be even, in [2, min(d, %d)]",
             2 * kMaxPairs);
  RA_REQUIRE(inv_freq != nullptr && std::isfinite(mscale), "inv_freq must be given and mscale finite");
  RA_REQUIRE(n_axes >= 1 && n_axes <= kMaxAxes && (axis || n_axes == 1), "1 to %d axes, and the axis of each pair", kMaxAxes);
  const double two_pi = 6.283185307179586476925286766559;
  p.mscale = static_cast<float>(mscale);
  p.sign = backward ? -1.f : 1.f;
  for (int i = 0; i < kMaxPairs; ++i) {
    const bool used = i < rot / 2;
    RA_REQUIRE(!used || std::fabs(inv_freq[i]) <= two_pi, "inv_freq[%d] must be in [-2 pi, 2 pi]", i);
    RA_REQUIRE(!used || !axis || (axis[i] >= 0 && axis[i] < n_axes), "axis[%d] must be in [0, n_axes)", i);
    const double phi = used ? inv_freq[i] / two_pi : 0.0;
    const float hi = static_cast<float>(phi);
    p.phase[i] = make_float2(hi, static_cast<float>(phi - static_cast<double>(hi)));
    p.axis[i] = static_cast<uint8_t>(used && axis ? axis[i] : 0);
  }
  return RA_OK;
}

// Whether the elements of [rows, H, d] at these strides are all apart.
inline bool apart(int64_t rows, int64_t rs, int64_t H, int64_t hs, int64_t d) {
  if (rows > 1 && H > 1)
    return (hs >= d && rs >= (H - 1) * hs + d) || (rs >= d && hs >= (rows - 1) * rs + d);
  return (rows <= 1 || rs >= d) && (H <= 1 || hs >= d);
}

}  // namespace
