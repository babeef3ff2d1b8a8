// What may be done to a score before the softmax, in log2 units: a cap by tanh,
// x -> cap tanh(x / cap), then a bias by distance, x - slope |n - 1 - t|.
//
// tanh is odd: for |t| <= 1 it is t Q(t^2) with a polynomial Q, the minimax
// approximation (Remez exchange) of tanh(sqrt y) / sqrt y on [0, 1], relative
// error 7e-8; beyond, 1 - 2 / (1 + e^(2|t|)), whose terms are then of like size.
// A capped score is off by 2^-20 of itself at most, 2^-22 of the cap beyond it, most of
// it the coefficients left out below 1/2 (tanh_near). The hardware's one-instruction
// tanh is off by 2^-11 of the cap: half a percent of a weight.
#pragma once
#include <cstdint>

#include "sai_internal.h"

namespace sai {

// Tokens that row `row` of length n sees: [start, sinks_end) and [first, end),
// start <= sinks_end <= first <= end (sinks_end = start without a window). Not
// good: a start or prefix outside [0, max_len], or a length.
struct RowSpan {
  int start, sinks_end, first, end;
  bool good;
};
__device__ __forceinline__ RowSpan row_span(const AttnLaunch& p, int row, int n) {
  const int from = p.row_starts ? p.row_starts[row] : 0, prefix = p.prefix_lens ? p.prefix_lens[row] : 0;
  RowSpan r{0, 0, 0, 0, n >= 0 && n <= p.max_len && from >= 0 && from <= p.max_len && prefix >= 0 && prefix <= p.max_len};
  if (!r.good || n == 0) return r;
  r.end = max(n, prefix);
  r.start = min(from, r.end);
  r.first = p.window > 0 ? max(r.start, n - p.window) : r.start;
  r.sinks_end = r.start + min(p.sinks, r.first - r.start);
  return r;
}

// Q's coefficient of y^i.
__host__ __device__ constexpr float tanh_q(int i) {
  constexpr float q[7] = {0.9999999502f, -0.3333283915f, 0.1332520408f, -0.05345702955f,
                          0.02028998032f, -0.006203378982f, 0.001041022586f};
  return q[i];
}

// The same with four coefficients for |t| <= 1/2, where most scores lie
// (relative error 5.6e-7, 9.3 2^-24), and with three for |t| <= 1/4 (4.2e-7, 7.1
// 2^-24): a score is moved by 2^-20.7 of itself, which is below what an fp32 sum of
// 64 or 128 products may be off by (2^-17, 2^-16 of the sum of their sizes).
constexpr float kNear = 0.5f, kNearest = 0.25f;
__host__ __device__ constexpr float tanh_near(int i) {
  constexpr float q[4] = {0.9999994558f, -0.3332631794f, 0.1319029659f, -0.04440222584f};
  return q[i];
}
__host__ __device__ constexpr float tanh_nearest(int i) {
  constexpr float q[3] = {0.9999996043f, -0.3332190823f, 0.1284161343f};
  return q[i];
}

// tanh(t) for |t| > 1 (right to 2^-22 absolute below)
__device__ __forceinline__ float tanh_far(float t) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(t) * 2.885390081777927f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return copysignf(fmaf(-2.f, r, 1.f), t);
}

// x -> cap tanh(x / cap), inv = 1 / cap; NaN stays, infinities become +-cap
__device__ __forceinline__ float capped(float x, float cap, float inv) {
  const float t = x * inv, y = t * t;
  float q = tanh_q(6);
#pragma unroll
  for (int i = 5; i >= 0; --i) q = fmaf(q, y, tanh_q(i));
  return cap * (y <= 1.f ? t * q : tanh_far(t));
}

}  // namespace sai
