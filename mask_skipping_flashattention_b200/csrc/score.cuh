// Shaped attention scores: a tanh cap and a penalty linear in the distance,
//   z = cap * tanh(scale * s / cap) - slope_h * |i - j|     (s = q . k),
// carried in log2 units (times log2 e), and the factor 1 - tanh^2 that the
// cap's chain rule puts on the score gradient.
//
// tanh(x), x = c0 s with c0 = scale / cap, from minimax fits of tanh(x) / x in u = x^2:
//   |x| <= 0.625  5 terms, relative error 1.1e-7 (2.1e-7 as evaluated in fp32);
//   |x| <= 1      7 terms, 5e-8 (1.6e-7);
//   any x         5 terms over 5, to |x| = 9 (then constant), 2e-8 (3.3e-7).
// They keep the score's error proportional to the score, which the hardware's tanh
// (relative 2^-11) would not: with a cap of 50 that one moves a score by up to 0.02 and
// its weight by 2 %.  In the polynomials, scale, cap and log2 e are folded into the
// coefficients, so that a score costs its square, the terms and one product; the fp32 pipe
// is what they load (two operations a score without a shape; 8, 10 and some 14 and a
// reciprocal with these), beside the exponential of the special-function unit.
// Which form a group of scores takes is decided by its largest magnitude, a warp at a
// time.  Measured, causal 8192 row, 16 / 4 heads, D 128: forward 292 us without a shape, 406,
// 473 and 716 us in the three forms; backward 1135 us in the 7 terms, 1478 in the last.  The
// backward leaves the 5 terms out: each form is four times in its code, and groups
// that alternate between three forms made it slower (1121 -> 1322 us at a cap that splits
// them, at the step that tried it) than the two terms saved.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace bfa {

constexpr float kLog2e = 1.4426950408889634f;

constexpr int kTanhTerms = 7, kTanhFew = 5;
constexpr float kTanhAnyMax = 9.f;

// What a call makes of its scores.
enum ScoreMode : int {
  kScorePlain = 0,
  kScoreCap = 1,
  kScoreSlopes = 2,
  kScoreCapSlopes = 3,
};

// Device view of a call's score shape (all zero: plain scores).
struct ScoreParams {
  float c0;             // scale / cap
  float c1;             // cap * log2(e)  (0: no cap)
  float ninv_c1_sq;     // -1 / c1^2
  float poly_max;       // largest |s| for the polynomial (negative: not to be used)
  float poly[kTanhTerms];  // its coefficients in s^2, times c1 c0
  float few_max;        // the same for the shorter one
  float few[kTanhFew];
  const float* slopes;  // [H] or nullptr
  __host__ __device__ int mode() const { return (c1 != 0.f ? kScoreCap : 0) | (slopes ? kScoreSlopes : 0); }
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * tanh(c0 s) * log2(e) of a pair: the folded polynomial
template <int kTerms>
__device__ __forceinline__ uint64_t capped_poly(uint64_t s, const float (&c)[kTerms]) {
  const uint64_t u = ptx::f2_mul(s, s);
  uint64_t p = ptx::f2_pack(c[kTerms - 1], c[kTerms - 1]);
#pragma unroll
  for (int i = kTerms - 2; i >= 0; --i) p = ptx::f2_fma(p, u, ptx::f2_pack(c[i], c[i]));
  return ptx::f2_mul(s, p);
}

// A constant pair made where it is used: the compiler would otherwise hold the pairs of
// the rarer forms in registers over the whole tile loop, which costs the common one.
__device__ __forceinline__ uint64_t f2_both(float c) {
  uint64_t r;
  asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(c));
  return r;
}

// x cut to |x| <= m; NaN stays NaN (fminf and fmaxf would make it a cap, and a row that
// attends it a finite one)
__device__ __forceinline__ float clamp_nan(float x, float m) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(-m));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(y) : "f"(m));
  return y;
}

// any x (infinities give the cap)
__device__ __forceinline__ uint64_t capped_any2(float s0, float s1, const ScoreParams& sp) {
  const float x0 = clamp_nan(s0 * sp.c0, kTanhAnyMax), x1 = clamp_nan(s1 * sp.c0, kTanhAnyMax);
  const uint64_t x = ptx::f2_pack(x0, x1), u = ptx::f2_mul(x, x);
  uint64_t p = f2_both(1.3353410699e-08f), q = f2_both(7.7760461556e-07f);
  p = ptx::f2_fma(p, u, f2_both(2.0608182991e-05f));
  q = ptx::f2_fma(q, u, f2_both(3.2855461444e-04f));
  p = ptx::f2_fma(p, u, f2_both(3.4955344269e-03f));
  q = ptx::f2_fma(q, u, f2_both(2.5876779672e-02f));
  p = ptx::f2_fma(p, u, f2_both(0.13380981060f));
  q = ptx::f2_fma(q, u, f2_both(0.46714296718f));
  p = ptx::f2_fma(p, u, f2_both(0.99999997963f));
  q = ptx::f2_fma(q, u, f2_both(1.f));
  float q0, q1;
  ptx::f2_unpack(q, q0, q1);
  return ptx::f2_mul(ptx::f2_mul(ptx::f2_mul(x, f2_both(sp.c1)), p), ptx::f2_pack(rcp_approx(q0), rcp_approx(q1)));
}

__device__ __forceinline__ float capped_any(float s, const ScoreParams& sp) {
  float a, b;
  ptx::f2_unpack(capped_any2(s, s, sp), a, b);
  return a;
}

// Natural-log LSE of a row from its reference maximum (log2 units) and its sum.  Only a row
// that attends nothing has the sum 0 and gets -inf; a NaN score makes the sum NaN, which must
// not pass for that (l > 0 would let it): the backward reads -inf as an empty row.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}

enum CapForm : int { kCapPoly = 0, kCapAny = 1, kCapFew = 2 };

template <int kForm>
__device__ __forceinline__ uint64_t capped_pair(float s0, float s1, const ScoreParams& sp) {
  if (kForm == kCapFew) return capped_poly(ptx::f2_pack(s0, s1), sp.few);
  if (kForm == kCapPoly) return capped_poly(ptx::f2_pack(s0, s1), sp.poly);
  return capped_any2(s0, s1, sp);
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

// The same where every attended entry of a row lies at or before the query (step -1, d0 - j
// >= 0): linear everywhere, and what it gives the masked entries does not matter.
__device__ __forceinline__ ScoreBias score_bias_causal(float slope, int d0) {
  ScoreBias r;
  r.slope = slope;
  r.d0 = static_cast<float>(d0);
  r.step = -1.f;
  r.linear = true;
  r.a = -slope * r.d0;
  r.b = slope;
  return r;
}

__device__ __forceinline__ float bias_at(const ScoreBias& r, int j) {
  return -r.slope * fabsf(fmaf(r.step, static_cast<float>(j), r.d0));
}

// a pair of products with the cap (or the scale) and a linear penalty: log2 units
template <int kMode, int kForm>
__device__ __forceinline__ uint64_t shaped_linear(float s0, float s1, int j, const ScoreBias& r, const ScoreParams& sp,
                                                  float scale_log2) {
  if (kMode == kScoreCap) return capped_pair<kForm>(s0, s1, sp);
  const uint64_t bias = ptx::f2_pack(fmaf(r.b, static_cast<float>(j), r.a), fmaf(r.b, static_cast<float>(j + 1), r.a));
  if (kMode == kScoreSlopes) return ptx::f2_fma(ptx::f2_pack(s0, s1), ptx::f2_pack(scale_log2, scale_log2), bias);
  return ptx::f2_add(capped_pair<kForm>(s0, s1, sp), bias);
}

template <int kMode, int kForm, bool kTurn>
__device__ __forceinline__ void shape_row_as(float* s, const ScoreParams& sp, float scale_log2, const ScoreBias& r) {
#pragma unroll
  for (int j = 0; j < 128; j += 2) {
    if (!kTurn) {
      ptx::f2_unpack(shaped_linear<kMode, kForm>(s[j], s[j + 1], j, r, sp, scale_log2), s[j], s[j + 1]);
    } else {  // the penalty changes direction in this tile
      float z0 = s[j] * scale_log2, z1 = s[j + 1] * scale_log2;
      if (kMode & kScoreCap) ptx::f2_unpack(capped_pair<kForm>(s[j], s[j + 1], sp), z0, z1);
      s[j] = z0 + bias_at(r, j);
      s[j + 1] = z1 + bias_at(r, j + 1);
    }
  }
}

// A row of 128 products s becomes shaped scores in log2 units, in place (the
// forward: one row a thread; `causal`: no later key is attended).  Called by whole warps.
template <int kMode>
__device__ __forceinline__ void shape_row(float* s, const ScoreParams& sp, float scale_log2, float slope, int d0,
                                          bool causal) {
  ScoreBias r = {};
  r.linear = true;
  if (kMode & kScoreSlopes) r = causal ? score_bias_causal(slope, d0) : score_bias(slope, d0, -1);
  if (!(kMode & kScoreCap)) {
    if (r.linear) shape_row_as<kMode, kCapPoly, false>(s, sp, scale_log2, r);
    else shape_row_as<kMode, kCapPoly, true>(s, sp, scale_log2, r);
    return;
  }
  float mx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 128; j += 2) mx[(j >> 1) & 3] = ptx::fmax3(mx[(j >> 1) & 3], fabsf(s[j]), fabsf(s[j + 1]));
  const float big = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  if (r.linear && __all_sync(0xffffffffu, big <= sp.few_max)) shape_row_as<kMode, kCapFew, false>(s, sp, scale_log2, r);
  else if (r.linear && __all_sync(0xffffffffu, big <= sp.poly_max)) shape_row_as<kMode, kCapPoly, false>(s, sp, scale_log2, r);
  else shape_row_as<kMode, kCapAny, (kMode & kScoreSlopes) != 0>(s, sp, scale_log2, r);
}

// The backward: a pair of products (entries j, j + 1) as the exponents x of their
// weights, log2(P) = z - LSE (nl: minus LSE log2 e of the two), and the cap's factor
// f = 1 - tanh^2 (untouched without a cap).  kSlow also takes the attend-bits of
// the group's 32 entries (bit jb for entry j: masked ones -inf, their products not
// looked at) and penalties that change direction in the tile.
template <int kMode, int kForm, bool kSlow>
__device__ __forceinline__ void shape_pair(float s0, float s1, int j, int jb, uint32_t bits, const ScoreBias& r,
                                           const ScoreParams& sp, float scale_log2, uint64_t nl, uint64_t& x,
                                           uint64_t& f) {
  if (kSlow) {
    if (!((bits >> jb) & 1u)) s0 = 0.f;
    if (!((bits >> (jb + 1)) & 1u)) s1 = 0.f;
  }
  if (kMode & kScoreSlopes) {
    const uint64_t bias = kSlow ? ptx::f2_pack(bias_at(r, j), bias_at(r, j + 1))
                                : ptx::f2_pack(fmaf(r.b, static_cast<float>(j), r.a),
                                               fmaf(r.b, static_cast<float>(j + 1), r.a));
    nl = ptx::f2_add(nl, bias);
  }
  if (kMode & kScoreCap) {
    const uint64_t z = capped_pair<kForm>(s0, s1, sp);
    x = ptx::f2_add(z, nl);
    f = ptx::f2_fma(ptx::f2_mul(z, ptx::f2_pack(sp.ninv_c1_sq, sp.ninv_c1_sq)), z, ptx::f2_pack(1.f, 1.f));
  } else {
    x = ptx::f2_fma(ptx::f2_pack(s0, s1), ptx::f2_pack(scale_log2, scale_log2), nl);
  }
  if (kSlow) {
    float x0, x1;
    ptx::f2_unpack(x, x0, x1);
    if (!((bits >> jb) & 1u)) x0 = -INFINITY;
    if (!((bits >> (jb + 1)) & 1u)) x1 = -INFINITY;
    x = ptx::f2_pack(x0, x1);
  }
}

// Run body(form tag, slow tag) for a group of 32 products: the cap's form by their largest
// magnitude (masked ones count too: they only cost the choice).  Called by whole warps.
template <int V>
struct ScoreTag {
  static constexpr int value = V;
};
template <int kMode, typename F>
__device__ __forceinline__ void score_dispatch(const uint32_t (&s)[32], const ScoreParams& sp, bool slow, F&& body) {
  if (kMode & kScoreCap) {
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < 32; j += 2)
      mx = ptx::fmax3(mx, fabsf(__uint_as_float(s[j])), fabsf(__uint_as_float(s[j + 1])));
    if (slow || !__all_sync(0xffffffffu, mx <= sp.poly_max)) body(ScoreTag<kCapAny>(), ScoreTag<1>());
    else body(ScoreTag<kCapPoly>(), ScoreTag<0>());
  } else {
    if (slow) body(ScoreTag<kCapPoly>(), ScoreTag<1>());
    else body(ScoreTag<kCapPoly>(), ScoreTag<0>());
  }
}

// f(mode tag) for a call's mode (host)
template <typename F>
inline auto for_score_mode(int mode, F&& f) {
  switch (mode) {
    case kScoreCap: return f(ScoreTag<kScoreCap>());
    case kScoreSlopes: return f(ScoreTag<kScoreSlopes>());
    case kScoreCapSlopes: return f(ScoreTag<kScoreCapSlopes>());
    default: return f(ScoreTag<kScorePlain>());
  }
}

}  // namespace bfa
