// linrec_math.cuh -- the gates of the gated linear recurrence, for its scan, its
// backward and its one-token step:
//   z = a + dt_bias, g = -e^{A_log} softplus(z), alpha = e^g, beta = sigmoid(b),
//   f = 1, 1 - alpha or sqrt(1 - alpha^2) (the input scale), u = f beta x.
// float32 throughout, two channels at a time (packed f32x2 arithmetic halves the
// instructions, which is what bounds these kernels).  Every exponential is one SFU ex2 of a
// rounded product and every quotient one SFU reciprocal (about 1e-7 relative each);
// 1 - alpha and softplus keep their relative accuracy where they are small (slow channels,
// whose alpha is next to 1).  The decay is carried as its base-2 exponent e = g log2(e).
#pragma once

#include "common.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// Two floats at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 ex2_2(float2 x) { return make_float2(ex2_f(x.x), ex2_f(x.y)); }
__device__ __forceinline__ float2 rcp_2(float2 x) { return make_float2(rcp_f(x.x), rcp_f(x.y)); }

// log(1 + y) / y for y in [0, 1]: the polynomial of degree 8 with the least relative error
// (Remez exchange on log1p(y) / y; 3.0e-8, 1.7e-7 with float32 rounding).  N tokens at once:
// a packed constant takes two moves into a register pair, so it is brought in once for all.
template <int N>
__device__ __forceinline__ void log1p_over(const float2* y, float2* p) {
  const float k[9] = {5.232694263e-03f, -2.950523877e-02f, 7.822595187e-02f,
                      -1.366324579e-01f, 1.910600676e-01f, -2.484298221e-01f,
                      3.331909681e-01f, -4.999949314e-01f, 9.999999699e-01f};
  const float2 k0 = both(k[0]), k1 = both(k[1]);
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = fma2(y[i], k0, k1);
#pragma unroll
  for (int j = 2; j < 9; ++j) {
    const float2 kj = both(k[j]);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = fma2(p[i], y[i], kj);
  }
}

// f[i] = 1 - 2^e for e <= 0.  Where the difference would cancel (e > -0.5): e times the polynomial
// of degree 4 with the least relative error on [-0.5, 0] (Remez exchange on (1 - 2^e) / e;
// 1.3e-8, 1.4e-7 with float32 rounding); 1 - pow elsewhere (pow = 2^e).
template <int N>
__device__ __forceinline__ void one_minus_ex2(const float2* e, const float2* pow, float2* f) {
  const float k[5] = {-1.15445233e-03f, -9.54128150e-03f, -5.54904081e-02f, -2.40225643e-01f,
                      -6.93147182e-01f};
  const float2 k0 = both(k[0]), k1 = both(k[1]);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = fma2(e[i], k0, k1);
#pragma unroll
  for (int j = 2; j < 5; ++j) {
    const float2 kj = both(k[j]);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = fma2(e[i], f[i], kj);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f[i] = mul2(e[i], f[i]);
    if (!(e[i].x > -0.5f)) f[i].x = 1.f - pow[i].x;
    if (!(e[i].y > -0.5f)) f[i].y = 1.f - pow[i].y;
  }
}

// Per-channel constants of the gates.
struct GateConst {
  float2 rate;  // -e^{A_log} log2(e): e = rate softplus(z)
  float2 bias;  // dt_bias
};
__device__ __forceinline__ GateConst gate_const(const float* A_log, const float* dt_bias, int c,
                                                int D) {
  GateConst k{both(0.f), both(0.f)};
  if (c < D) {
    k.rate.x = -expf(A_log[c]) * kLog2e;
    k.bias.x = dt_bias[c];
  }
  if (c + 1 < D) {
    k.rate.y = -expf(A_log[c + 1]) * kLog2e;
    k.bias.y = dt_bias[c + 1];
  }
  return k;
}

// e[i] in place of a[i], the base-2 exponents of alpha of N tokens; GIVEN: a is g itself.
// softplus(z) = max(z, 0) + log(1 + y) with y = e^{-|z|}.
template <bool GIVEN, int N>
__device__ __forceinline__ void decay_exponents(float2* a, const GateConst& k) {
  if (GIVEN) {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = mul2(a[i], both(kLog2e));
    return;
  }
  float2 y[N], q[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = add2(a[i], k.bias);
    y[i] = make_float2(ex2_f(-fabsf(a[i].x) * kLog2e), ex2_f(-fabsf(a[i].y) * kLog2e));
  }
  log1p_over<N>(y, q);
#pragma unroll
  for (int i = 0; i < N; ++i) {  // a NaN goes through y
    const float2 m = make_float2(fmaxf(a[i].x, 0.f), fmaxf(a[i].y, 0.f));
    a[i] = mul2(k.rate, fma2(y[i], q[i], m));
  }
}
// The same, and slope = -e^{A_log} sigmoid(z), the derivative of g with respect to a.
template <int N>
__device__ __forceinline__ void decay_exponents_slope(float2* a, const GateConst& k,
                                                      float2* slope) {
  float2 y[N], q[N];
  const float2 rate = mul2(k.rate, both(kLn2)), one = both(1.f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = add2(a[i], k.bias);
    y[i] = make_float2(ex2_f(-fabsf(a[i].x) * kLog2e), ex2_f(-fabsf(a[i].y) * kLog2e));
    const float2 r = rcp_2(add2(y[i], one));
    slope[i] = mul2(rate, make_float2(a[i].x >= 0.f ? r.x : r.x * y[i].x,
                                      a[i].y >= 0.f ? r.y : r.y * y[i].y));
  }
  log1p_over<N>(y, q);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 m = make_float2(fmaxf(a[i].x, 0.f), fmaxf(a[i].y, 0.f));
    a[i] = mul2(k.rate, fma2(y[i], q[i], m));
  }
}

// The input scales f of N tokens from alpha = 2^e (not called for kScaleNone).
template <int SCALE, int N>
__device__ __forceinline__ void input_scales(const float2* e, const float2* alpha, float2* f) {
  if (SCALE == kScaleTied) {
    one_minus_ex2<N>(e, alpha, f);
  } else {
    float2 e2[N], a2[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      e2[i] = add2(e[i], e[i]);
      a2[i] = mul2(alpha[i], alpha[i]);
    }
    one_minus_ex2<N>(e2, a2, f);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = make_float2(sqrt_f(f[i].x), sqrt_f(f[i].y));
  }
}
// df/dg.  sqrt(1 - alpha^2) has an infinite slope at g = 0; what reaches a is f' dg/da, which
// goes to 0 there with softplus, so f' is taken as 0 where f underflows.
template <int SCALE>
__device__ __forceinline__ float input_scale_slope(float alpha, float f) {
  if (SCALE == kScaleTied) return -alpha;
  return f > 0.f ? -alpha * alpha * rcp_f(f) : 0.f;
}

// beta[i] in place of b[i]; GIVEN: b is beta itself.
template <bool GIVEN, int N>
__device__ __forceinline__ void write_gates(float2* b) {
  if (GIVEN) return;
  const float2 one = both(1.f);
#pragma unroll
  for (int i = 0; i < N; ++i)
    b[i] = rcp_2(add2(make_float2(ex2_f(b[i].x * -kLog2e), ex2_f(b[i].y * -kLog2e)), one));
}
// 1 - beta = beta e^{-b}, without the cancellation (the exponent is kept below 2^126, where
// beta has underflowed).
__device__ __forceinline__ float2 write_gate_rest(float2 b, float2 beta) {
  return mul2(beta, make_float2(ex2_f(fminf(b.x * -kLog2e, 126.f)),
                                ex2_f(fminf(b.y * -kLog2e, 126.f))));
}

}  // namespace gdn
