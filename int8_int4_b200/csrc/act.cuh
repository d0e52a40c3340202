// act.cuh -- the activations of the fused epilogues and their derivatives,
// in fp32.
//
// All are written in a form that keeps its RELATIVE accuracy where the
// result is small (negative z), because the result is rounded to fp16, whose
// steps shrink with it: sigmoid products instead of 1 + tanh, and the
// complementary error function's scaled form instead of 1 + erf. Measured on
// the host in fp32 against 64 bits the largest relative error of any of them
// is about 3e-6 for |z| <= 8, far below fp16's half step of 4.9e-4.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

namespace aria {

enum Act : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + exp(-z)). exp overflows to infinity below z = -88.7: the
// reciprocal is then 0, as it should be to fp16.
__device__ __forceinline__ float sigmoid(float z) { return fast_rcp(1.0f + __expf(-z)); }

// Upper tail of the normal distribution, Q(a) = erfc(a / sqrt(2)) / 2 for
// a >= 0, as exp(-a^2 / 2) * R(a): R = erfcx(a / sqrt(2)) / 2 is smooth and
// slowly decreasing, and t * polynomial(t) in t = 1 / (1 + 0.26 a) fits it
// to 2.8e-7 relative on [0, 8] (a least-squares fit reweighted toward equal
// error, made in 64 bits for this file; 5.6e-7 when evaluated in fp32) and
// keeps its a -> infinity limit. `gauss` returns exp(-a^2 / 2).
__device__ __forceinline__ float normal_tail(float a, float& gauss) {
  const float t = fast_rcp(fmaf(0.26f, a, 1.0f));
  float r = -0.07561299204826355f;
  r = fmaf(r, t, 0.23910772800445557f);
  r = fmaf(r, t, -0.12206314504146576f);
  r = fmaf(r, t, 0.17879557609558105f);
  r = fmaf(r, t, 0.06802142411470413f);
  r = fmaf(r, t, 0.10833492130041122f);
  r = fmaf(r, t, 0.10341634601354599f);
  gauss = __expf(-0.5f * a * a);
  return r * t * gauss;
}

constexpr float kTanhC0 = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhC1 = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == kActRelu) {
    return fmaxf(z, 0.0f);
  } else if constexpr (ACT == kActSilu) {
    return z * sigmoid(z);
  } else if constexpr (ACT == kActGelu) {
    // z Phi(z) = max(z, 0) - |z| Q(|z|): no cancellation on either side
    const float a = fabsf(z);
    float g;
    return fmaf(-a, normal_tail(a, g), fmaxf(z, 0.0f));
  } else if constexpr (ACT == kActGeluTanh) {
    // z (1 + tanh w) / 2 = z sigmoid(2 w)
    const float w2 = 2.0f * kTanhC0 * z * fmaf(kTanhC1 * z, z, 1.0f);
    return z * sigmoid(w2);
  } else {
    return z;
  }
}

// act(z) and act'(z)
template <int ACT>
__device__ __forceinline__ void act_fwd_bwd(float z, float& f, float& d) {
  if constexpr (ACT == kActRelu) {
    f = fmaxf(z, 0.0f);
    d = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    const float s = sigmoid(z);
    f = z * s;
    // 1 - s would cancel for large z; it multiplies z there, so the term's
    // absolute error stays below fp32's step of the sum
    d = s * fmaf(z, 1.0f - s, 1.0f);
  } else if constexpr (ACT == kActGelu) {
    const float a = fabsf(z);
    float g;
    const float q = normal_tail(a, g);
    f = fmaf(-a, q, fmaxf(z, 0.0f));
    // Phi(z) + z phi(z)
    d = fmaf(z * 0.3989422804014327f, g, z > 0.0f ? 1.0f - q : q);
  } else if constexpr (ACT == kActGeluTanh) {
    const float z2 = z * z;
    const float s = sigmoid(2.0f * kTanhC0 * z * fmaf(kTanhC1, z2, 1.0f));
    f = z * s;
    d = fmaf(f * (1.0f - s), 2.0f * kTanhC0 * fmaf(3.0f * kTanhC1, z2, 1.0f), s);
  } else {
    f = z;
    d = 1.0f;
  }
}

template <int A>
struct ActTag {
  static constexpr int value = A;
};

// Runs f(ActTag<ACT>) for the launch's activation: one uniform branch
// outside the element loop, so each loop body holds one activation only.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: f(ActTag<kActRelu>{}); break;
    case kActSilu: f(ActTag<kActSilu>{}); break;
    case kActGelu: f(ActTag<kActGelu>{}); break;
    case kActGeluTanh: f(ActTag<kActGeluTanh>{}); break;
    default: f(ActTag<kActNone>{}); break;
  }
}

}  // namespace aria
