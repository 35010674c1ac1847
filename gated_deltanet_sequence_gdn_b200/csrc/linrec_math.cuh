// linrec_math.cuh -- the gates of the gated linear recurrence, for its scan, its
// backward and its one-token step:
//   z = a + dt_bias, g = -e^{A_log} softplus(z), alpha = e^g, beta = sigmoid(b),
//   f = 1, 1 - alpha or sqrt(1 - alpha^2) (the input scale), u = f beta x.
// float32 throughout.  Every exponential is one SFU ex2 of a rounded product and every
// quotient one SFU reciprocal (about 1e-7 relative each); 1 - alpha and softplus are
// evaluated so that they keep their relative accuracy where they are small (slow
// channels, whose alpha is next to 1).
#pragma once

#include "common.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

// Input scale of the recurrence (GDN_LINREC_TIED, GDN_LINREC_UNIT).
enum LinrecScale { kScaleNone = 0, kScaleTied = 1, kScaleUnit = 2 };

__device__ __forceinline__ float ex2_f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_f(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_f(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log(1 + y) for y in [0, 1]: 2 atanh(t), t = y / (2 + y) <= 1/3, by its odd series;
// the first term left out is t^14 / 15 < 1.4e-8 relative.
__device__ __forceinline__ float log1p_unit(float y, float inv_2py) {
  const float t = y * inv_2py, w = t * t;
  float p = fmaf(w, 1.f / 13.f, 1.f / 11.f);
  p = fmaf(w, p, 1.f / 9.f);
  p = fmaf(w, p, 1.f / 7.f);
  p = fmaf(w, p, 1.f / 5.f);
  p = fmaf(w, p, 1.f / 3.f);
  p = fmaf(w, p, 1.f);
  return 2.f * t * p;
}

// 1 - e^v for v <= 0: the exponential's series where it would cancel (v > -0.35: the
// first term left out is v^7 / 8! < 2e-8 relative), the difference elsewhere.
__device__ __forceinline__ float one_minus_exp(float v) {
  float p = fmaf(v, 1.f / 5040.f, 1.f / 720.f);
  p = fmaf(v, p, 1.f / 120.f);
  p = fmaf(v, p, 1.f / 24.f);
  p = fmaf(v, p, 1.f / 6.f);
  p = fmaf(v, p, 0.5f);
  p = fmaf(v, p, 1.f);
  return v > -0.35f ? -v * p : 1.f - ex2_f(v * kLog2e);
}

// The input scale f and, for the backward, df/dg = f' (alpha' = alpha with respect to g).
// sqrt(1 - alpha^2) has an infinite slope at g = 0; what reaches a is f' dg/da, which goes
// to 0 there with softplus, so f' is taken as 0 where f underflows.
template <int SCALE>
__device__ __forceinline__ float input_scale(float g) {
  if (SCALE == kScaleTied) return one_minus_exp(g);
  if (SCALE == kScaleUnit) return sqrt_f(one_minus_exp(2.f * g));
  return 1.f;
}
template <int SCALE>
__device__ __forceinline__ float input_scale_slope(float alpha, float f) {
  if (SCALE == kScaleTied) return -alpha;
  if (SCALE == kScaleUnit) return f > 0.f ? -alpha * alpha * rcp_f(f) : 0.f;
  return 0.f;
}

// Per-channel constants of the gates.
struct GateConst {
  float neg_A;  // -e^{A_log}
  float bias;   // dt_bias
};
__device__ __forceinline__ GateConst gate_const(const float* A_log, const float* dt_bias, int c) {
  return GateConst{-expf(A_log[c]), dt_bias[c]};
}

// The log-decay g of one element; `given`: a is g itself.
template <bool GIVEN>
__device__ __forceinline__ float log_decay(float a, const GateConst& k) {
  if (GIVEN) return a;
  const float z = a + k.bias;
  const float y = ex2_f(-fabsf(z) * kLog2e);
  return k.neg_A * (fmaxf(z, 0.f) + log1p_unit(y, rcp_f(2.f + y)));
}
// sigmoid by the exponential that does not overflow.
__device__ __forceinline__ float sigmoid_sfu(float b) {
  const float e = ex2_f(-fabsf(b) * kLog2e);
  const float r = rcp_f(1.f + e);
  return b >= 0.f ? r : e * r;
}
template <bool GIVEN>
__device__ __forceinline__ float write_gate(float b) {
  return GIVEN ? b : sigmoid_sfu(b);
}

}  // namespace gdn
