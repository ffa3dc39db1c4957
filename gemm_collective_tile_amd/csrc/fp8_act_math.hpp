// Activations and their derivatives, in 32 bits.
#pragma once

#include "fp8_act.hpp"

namespace iris {

// z as a factor of what is 0 far out, where z may be infinite (fp16 holds a kept z of 65520 and
// more so): the slope there is its limit, 1 or 0. A NaN is in the other factor too.
__device__ __forceinline__ float held(float z) { return __builtin_amdgcn_fmed3f(z, -0x1p60f, 0x1p60f); }

// The normal distribution's upper tail Q(a) = erfc(a / sqrt 2) / 2, a >= 0, as
// exp(-a^2 / 2) t P(t) with t = 1 / (1 + 0.28 a): P of degree 8 fitted to the least
// relative error, 9.0e-8 over 0 <= a <= 40 (a weighted least-squares fit on Chebyshev
// points of t). A small value of gelu's negative side keeps its digits so, where 1 + erf
// would cancel. What 32 bits add grows with the exponent, whose roundings (of the square,
// of its product and of the constant) count |x^2| / 2 times 2^-24 and more: of the
// distribution 8e-7 for |x| up to 4, 2.0e-6 to 6, 7.4e-6 to 12.9, far below half a step of a
// 16-bit type. EXACT, for an fp32 C: the exponent's rest is carried along, 4.3e-7 anywhere
// (with an exact exp2 and reciprocal, in either form; theirs are good to an ulp).
// e: exp(-x^2 / 2). Returns the distribution at x.
template <bool EXACT>
__device__ __forceinline__ float normal_cdf(float x, float& e) {
  constexpr double kHalfLog2e = -0.72134752044448170;
  constexpr float c = (float)kHalfLog2e;
  const float a = __builtin_fabsf(x);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.28f, a, 1.0f));
  const float y = EXACT ? held(x) : x;   // no infinity among the rests
  const float square = y * y, power = square * c;
  e = __builtin_amdgcn_exp2f(power);
  if constexpr (EXACT) {
    constexpr float c_rest = (float)(kHalfLog2e - (double)c);
    const float rest = __builtin_fmaf(square, c_rest, __builtin_fmaf(__builtin_fmaf(y, y, -square), c, __builtin_fmaf(square, c, -power)));
    e = __builtin_fmaf(e, rest * 0.69314718055994531f, e);
  }
  float p = 0.025858724489808083f;
  p = __builtin_fmaf(p, t, -0.09804520010948181f);
  p = __builtin_fmaf(p, t, 0.09953682124614716f);
  p = __builtin_fmaf(p, t, -0.01241461280733347f);
  p = __builtin_fmaf(p, t, 0.0755930095911026f);
  p = __builtin_fmaf(p, t, 0.08288740366697311f);
  p = __builtin_fmaf(p, t, 0.10318596661090851f);
  p = __builtin_fmaf(p, t, 0.11169400811195374f);
  p = __builtin_fmaf(p, t, 0.11170392483472824f);
  const float q = p * t * e;
  return x < 0.0f ? q : 1.0f - q;
}

// gelu in its tanh form is z s(u), u = 2 sqrt(2 / pi) (z + 0.044715 z^3): the tanh of
// half an argument is a sigmoid. z^2 is held to 2^100, so that the derivative stays
// finite as z^2 leaves 32 bits.
constexpr float kGeluU = 1.5957691216057308f, kGelu3 = 0.044715f;
__device__ __forceinline__ float gelu_square(float z) { return __builtin_fminf(z * z, 0x1p100f); }
__device__ __forceinline__ float gelu_sigmoid(float z, float z2) {   // s(u), the constants and log2 e multiplied beforehand
  constexpr float c = -1.4426950408889634f * kGeluU;
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * __builtin_fmaf(c * kGelu3, z2, c)));
}

// EXACT: for an fp32 C
template <bool EXACT, int U, int N>
__device__ __forceinline__ void activate(int act, float (&v)[U][N]) {
  switch (act) {
    case ACT_RELU:
#pragma unroll
      for (int k = 0; k < U * N; ++k) v[k / N][k % N] = v[k / N][k % N] < 0.0f ? 0.0f : v[k / N][k % N];   // NaN stays
      break;
    case ACT_GELU:
#pragma unroll
      for (int k = 0; k < U * N; ++k) {
        float e;
        v[k / N][k % N] *= normal_cdf<EXACT>(v[k / N][k % N], e);
      }
      break;
    case ACT_GELU_TANH:
#pragma unroll
      for (int k = 0; k < U * N; ++k) v[k / N][k % N] *= gelu_sigmoid(v[k / N][k % N], v[k / N][k % N] * v[k / N][k % N]);
      break;
    case ACT_SILU:
#pragma unroll
      for (int k = 0; k < U * N; ++k) v[k / N][k % N] *= sigmoid(v[k / N][k % N]);
      break;
    default: break;
  }
}

// v *= act'(z)
template <bool EXACT, int U, int N>
__device__ __forceinline__ void times_slope(int act, const float (&z)[U][N], float (&v)[U][N]) {
  switch (act) {
    case ACT_RELU: {
#pragma unroll
      for (int k = 0; k < U * N; ++k) v[k / N][k % N] = z[k / N][k % N] > 0.0f ? v[k / N][k % N] : 0.0f;
      // NaN stays: looked for in all values at once (v_maximum3_f32 takes two and passes a NaN on),
      // for a comparison and a choice of each would cost 2.5 % at 4095 x 11008 x 4096
      float most = z[0][0];
#pragma unroll
      for (int k = 1; k < U * N; ++k) most = __builtin_elementwise_maximum(most, z[k / N][k % N]);
      if (most != most) {
#pragma unroll
        for (int k = 0; k < U * N; ++k) v[k / N][k % N] = z[k / N][k % N] != z[k / N][k % N] ? z[k / N][k % N] : v[k / N][k % N];
      }
      break;
    }
    case ACT_GELU:
#pragma unroll
      for (int k = 0; k < U * N; ++k) {
        float e;
        const float c = normal_cdf<EXACT>(z[k / N][k % N], e);
        v[k / N][k % N] *= __builtin_fmaf(held(z[k / N][k % N]) * 0.39894228040143268f, e, c);
      }
      break;
    case ACT_GELU_TANH:
#pragma unroll
      for (int k = 0; k < U * N; ++k) {
        const float z2 = gelu_square(z[k / N][k % N]), s = gelu_sigmoid(z[k / N][k % N], z2);
        v[k / N][k % N] *= __builtin_fmaf(held(z[k / N][k % N]) * s * (1.0f - s), __builtin_fmaf(3.0f * kGelu3 * kGeluU, z2, kGeluU), s);
      }
      break;
    case ACT_SILU:
#pragma unroll
      for (int k = 0; k < U * N; ++k) {
        const float s = sigmoid(z[k / N][k % N]);
        v[k / N][k % N] *= s * __builtin_fmaf(held(z[k / N][k % N]), 1.0f - s, 1.0f);
      }
      break;
    default: break;
  }
}

}  // namespace iris
