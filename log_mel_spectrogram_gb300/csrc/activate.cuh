// activate.cuh -- activations of the linear layers, in 32 bits, and their derivatives.
#pragma once

#include "f32x2.cuh"
#include "logmel.h"

namespace lm {

// max(x, 0), NaN for NaN.
__device__ __forceinline__ float relu(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// z Phi(z) = max(z, 0) - |z| Phi(-|z|), and log2 Phi(-a) is smooth enough for a
// polynomial: degree 7 in -a, fitted on [0, 10] for the least error of a Phi(-a),
// which is 1.3e-7 with the rounding of its evaluation (and at most 0.2% of a
// Phi(-a) itself); past 10 it falls as it should.  One exponential and no
// division: with a rational formula for erfc the special function unit bound
// the epilogue (windows of frames 14.1 us).  Past |z| = 20 the second term is 0.
__device__ __forceinline__ f32x2 gelu2(f32x2 z) {
  const float2 zz = unpair(z);
  const f32x2 b = pair(fmaxf(-fabsf(zz.x), -20.0f), fmaxf(-fabsf(zz.y), -20.0f));
  f32x2 q = fma2(both(1.39071039e-06f), b, both(5.31626938e-05f));
  q = fma2(q, b, both(0.000873087498f));
  q = fma2(q, b, both(0.00833543856f));
  q = fma2(q, b, both(0.0537305102f));
  q = fma2(q, b, both(-0.458572268f));
  q = fma2(q, b, both(1.15125668f));
  q = fma2(q, b, both(-0.999988258f));
  const float2 l = unpair(q);
  return fma2(b, pair(ex2(l.x), ex2(l.y)), pair(relu(zz.x), relu(zz.y)));
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == LM_ACT_RELU) return relu(z);
  if (ACT == LM_ACT_GELU) return unpair(gelu2(both(z))).x;
  if (ACT == LM_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
    const float u = fmaf(-2.0f * 0.79788456080286536f * kLog2e * 0.044715f * z * z, z,
                         -2.0f * 0.79788456080286536f * kLog2e * z);
    return z * rcp(1.0f + ex2(u));
  }
  if (ACT == LM_ACT_SILU) return z * rcp(1.0f + ex2(-kLog2e * z));
  return z;
}

template <int ACT>
__device__ __forceinline__ f32x2 activate2(f32x2 z) {
  if (ACT == LM_ACT_NONE) return z;
  if (ACT == LM_ACT_GELU) return gelu2(z);
  const float2 f = unpair(z);
  return pair(activate<ACT>(f.x), activate<ACT>(f.y));
}

// 1 / (1 + exp(-z)).
__device__ __forceinline__ float sigmoid(float z) { return rcp(1.0f + ex2(-kLog2e * z)); }

// The value and the derivative.  Products that may be 0 * infinity for large |z| are bounded;
// gelu takes the error function itself, because the polynomial above is fitted for z Phi(z)
// and 4e-6 off for Phi near 0.
template <int ACT>
__device__ __forceinline__ float activate_slope(float z, float &slope) {
  if (ACT == LM_ACT_RELU) {
    slope = z > 0.0f ? 1.0f : 0.0f;
    return relu(z);
  }
  if (ACT == LM_ACT_GELU) {
    const float phi = 0.5f * (1.0f + erff(0.70710678118654752f * z));
    slope = fmaf(z * 0.39894228040143268f, ex2(-0.5f * kLog2e * z * z), phi);
    return unpair(gelu2(both(z))).x;
  }
  if (ACT == LM_ACT_GELU_TANH) {
    const float c = 2.0f * 0.79788456080286536f, z2 = fminf(z * z, 1e30f);
    const float p = sigmoid(c * fmaf(0.044715f * z2, z, z));
    slope = fmaf(z * p * (1.0f - p), c * fmaf(3.0f * 0.044715f, z2, 1.0f), p);
    return z * p;
  }
  const float p = ACT == LM_ACT_NONE ? 1.0f : sigmoid(z);
  if (ACT == LM_ACT_SILU) {
    slope = p * fmaf(z, 1.0f - p, 1.0f);
    return z * p;
  }
  if (ACT == LM_ACT_SIGMOID) {
    slope = p * (1.0f - p);
    return p;
  }
  slope = 1.0f;
  return z;
}

// By a number that the whole warp shares.
__device__ __forceinline__ float activate_any(float z, int act) {
  switch (act) {
    case LM_ACT_RELU: return activate<LM_ACT_RELU>(z);
    case LM_ACT_GELU: return activate<LM_ACT_GELU>(z);
    case LM_ACT_GELU_TANH: return activate<LM_ACT_GELU_TANH>(z);
    case LM_ACT_SILU: return activate<LM_ACT_SILU>(z);
    case LM_ACT_SIGMOID: return sigmoid(z);
    default: return z;
  }
}

}  // namespace lm
