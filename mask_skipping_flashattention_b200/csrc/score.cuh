// Shaped attention scores: a tanh cap and a penalty linear in the distance,
//   z = cap * tanh(scale * s / cap) - slope_h * |i - j|     (s = q . k),
// carried in log2 units (times log2 e), and the factor 1 - tanh^2 that the
// cap's chain rule puts on the score gradient.
//
// tanh: |x| <= kTanhPoly takes the odd polynomial x * P(x^2) (a minimax fit of
// tanh(x) / x, relative error 3e-8, 1.6e-7 as evaluated in fp32); larger |x| take
// 1 - 2 / (1 + e^(2|x|)), whose absolute error of about 2e-7 is a relative one
// of 4e-7 there.  Both keep the score's error proportional to the score, which
// the hardware's tanh (relative 2^-11) would not: with a cap of 50 that one moves a
// score by up to 0.02 and its weight by 2 %.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace bfa {

constexpr float kLog2e = 1.4426950408889634f;

// Device view of a call's score shape (all zero: plain scores).
struct ScoreParams {
  float c0;             // scale / cap
  float c1;             // cap * log2(e)  (0: no cap)
  const float* slopes;  // [H] or nullptr
};

constexpr float kTanhPoly = 0.75f;
constexpr int kTanhTerms = 6;
// coefficients of P in u = x^2, lowest first
__device__ constexpr float kTanhC[kTanhTerms] = {0.999999971f,   -0.333329589f, 0.13325406f,
                                                 -0.0533444299f, 0.0195829077f, -0.00471625689f};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh of |x| <= kTanhPoly
__device__ __forceinline__ float tanh_small(float x) {
  const float u = x * x;
  float p = kTanhC[kTanhTerms - 1];
#pragma unroll
  for (int i = kTanhTerms - 2; i >= 0; --i) p = fmaf(p, u, kTanhC[i]);
  return x * p;
}

// tanh of any x (infinities give +-1, NaN stays NaN)
__device__ __forceinline__ float tanh_any(float x) {
  const float a = fabsf(x);
  const float big = 1.f - 2.f * rcp_approx(1.f + ptx::ex2_approx(2.f * kLog2e * a));
  return a <= kTanhPoly ? tanh_small(x) : copysignf(big, x);
}

// two tanh values at once, |x| <= kTanhPoly (packed fp32 pairs)
__device__ __forceinline__ uint64_t tanh_small2(uint64_t x) {
  const uint64_t u = ptx::f2_mul(x, x);
  uint64_t p = ptx::f2_pack(kTanhC[kTanhTerms - 1], kTanhC[kTanhTerms - 1]);
#pragma unroll
  for (int i = kTanhTerms - 2; i >= 0; --i) p = ptx::f2_fma(p, u, ptx::f2_pack(kTanhC[i], kTanhC[i]));
  return ptx::f2_mul(x, p);
}

// The penalty along one row (or column) of a tile: -slope * |d0 + step * j| for
// entry j = 0..127 (step is +1 or -1; slope times log2 e).  Where d0 + step * j
// keeps its sign over the tile it is a + b * j.
struct ScoreBias {
  float slope, d0, step;
  float a, b;
  bool linear;  // warp-uniform
};

// Called by whole warps.
__device__ __forceinline__ ScoreBias score_bias(float slope, int d0, int step) {
  ScoreBias r;
  r.slope = slope;
  r.d0 = static_cast<float>(d0);
  r.step = static_cast<float>(step);
  const int d1 = d0 + step * 127;
  const bool up = __all_sync(0xffffffffu, d0 >= 0 && d1 >= 0), down = __all_sync(0xffffffffu, d0 <= 0 && d1 <= 0);
  r.linear = up || down;
  const float f = up ? -slope : slope;
  r.a = f * r.d0;
  r.b = f * r.step;
  return r;
}

__device__ __forceinline__ float bias_at(const ScoreBias& r, int j) {
  return -r.slope * fabsf(fmaf(r.step, static_cast<float>(j), r.d0));
}

// A row of 128 products s becomes shaped scores in log2 units, in place (the
// forward: one row a thread).  Called by whole warps.
__device__ __forceinline__ void shape_row(float* s, const ScoreParams& sp, float scale_log2, float slope, int d0) {
  if (sp.c1 != 0.f) {
    float mx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 128; j += 2)
      mx[(j >> 1) & 3] = ptx::fmax3(mx[(j >> 1) & 3], fabsf(s[j]), fabsf(s[j + 1]));
    const float big = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    if (__all_sync(0xffffffffu, big * sp.c0 <= kTanhPoly)) {
      const uint64_t c0 = ptx::f2_pack(sp.c0, sp.c0), c1 = ptx::f2_pack(sp.c1, sp.c1);
#pragma unroll
      for (int j = 0; j < 128; j += 2)
        ptx::f2_unpack(ptx::f2_mul(tanh_small2(ptx::f2_mul(ptx::f2_pack(s[j], s[j + 1]), c0)), c1), s[j], s[j + 1]);
    } else {
#pragma unroll
      for (int j = 0; j < 128; ++j) s[j] = sp.c1 * tanh_any(s[j] * sp.c0);
    }
  }
  if (sp.slopes) {
    const float mul = sp.c1 != 0.f ? 1.f : scale_log2;
    const ScoreBias r = score_bias(slope, d0, -1);
    if (r.linear) {
      const uint64_t mul2 = ptx::f2_pack(mul, mul);
#pragma unroll
      for (int j = 0; j < 128; j += 2)
        ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(s[j], s[j + 1]), mul2,
                                   ptx::f2_pack(fmaf(r.b, static_cast<float>(j), r.a),
                                                fmaf(r.b, static_cast<float>(j + 1), r.a))),
                       s[j], s[j + 1]);
    } else {
#pragma unroll
      for (int j = 0; j < 128; ++j) s[j] = fmaf(s[j], mul, bias_at(r, j));
    }
  }
}

// How the backward treats a group of scores: no cap; a cap with every |x| within
// the polynomial's range; a cap with any x.
enum ScoreTanh { kTanhNone = 0, kTanhSmall = 1, kTanhAny = 2 };

// A pair of products (entries j, j + 1) as shaped scores z (log2 units), and the
// cap's factor f = 1 - tanh^2 (untouched for kTanhNone).  kSlow also takes the
// attend-bits of the group's 32 entries (bit jb for entry j: masked scores -inf,
// their products not looked at) and penalties that change direction in the tile.
template <int kTanh, bool kSlow>
__device__ __forceinline__ void shape_pair(float s0, float s1, int j, int jb, uint32_t bits, const ScoreBias& r,
                                           const ScoreParams& sp, float scale_log2, uint64_t& z, uint64_t& f) {
  if (kSlow) {
    if (!((bits >> jb) & 1u)) s0 = 0.f;
    if (!((bits >> (jb + 1)) & 1u)) s1 = 0.f;
  }
  const uint64_t bias = kSlow ? ptx::f2_pack(bias_at(r, j), bias_at(r, j + 1))
                              : ptx::f2_pack(fmaf(r.b, static_cast<float>(j), r.a),
                                             fmaf(r.b, static_cast<float>(j + 1), r.a));
  if (kTanh == kTanhNone) {
    z = ptx::f2_fma(ptx::f2_pack(s0, s1), ptx::f2_pack(scale_log2, scale_log2), bias);
  } else {
    const uint64_t x = ptx::f2_mul(ptx::f2_pack(s0, s1), ptx::f2_pack(sp.c0, sp.c0));
    uint64_t t;
    if (kTanh == kTanhSmall) {
      t = tanh_small2(x);
    } else {
      float x0, x1;
      ptx::f2_unpack(x, x0, x1);
      t = ptx::f2_pack(tanh_any(x0), tanh_any(x1));
    }
    z = ptx::f2_fma(t, ptx::f2_pack(sp.c1, sp.c1), bias);
    f = ptx::f2_fma(ptx::f2_mul(t, ptx::f2_pack(-1.f, -1.f)), t, ptx::f2_pack(1.f, 1.f));
  }
  if (kSlow) {
    float z0, z1;
    ptx::f2_unpack(z, z0, z1);
    if (!((bits >> jb) & 1u)) z0 = -INFINITY;
    if (!((bits >> (jb + 1)) & 1u)) z1 = -INFINITY;
    z = ptx::f2_pack(z0, z1);
  }
}

// Which form a group of 32 products takes (warp-uniform); masked ones count too:
// they only cost the choice.
__device__ __forceinline__ int score_form(const uint32_t (&s)[32], const ScoreParams& sp) {
  if (sp.c1 == 0.f) return kTanhNone;
  float mx = 0.f;
#pragma unroll
  for (int j = 0; j < 32; j += 2) mx = ptx::fmax3(mx, fabsf(__uint_as_float(s[j])), fabsf(__uint_as_float(s[j + 1])));
  return __all_sync(0xffffffffu, mx * sp.c0 <= kTanhPoly) ? kTanhSmall : kTanhAny;
}

// Run body(form tag, slow tag) for the form at hand.
template <int V>
struct ScoreTag {
  static constexpr int value = V;
};
template <typename F>
__device__ __forceinline__ void score_dispatch(int form, bool slow, F&& body) {
  if (form == kTanhNone) {
    if (slow) body(ScoreTag<kTanhNone>(), ScoreTag<1>());
    else body(ScoreTag<kTanhNone>(), ScoreTag<0>());
  } else if (form == kTanhSmall) {
    if (slow) body(ScoreTag<kTanhSmall>(), ScoreTag<1>());
    else body(ScoreTag<kTanhSmall>(), ScoreTag<0>());
  } else {
    body(ScoreTag<kTanhAny>(), ScoreTag<1>());
  }
}

}  // namespace bfa
