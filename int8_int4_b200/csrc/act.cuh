// act.cuh -- the activations of the fused epilogues and their derivatives,
// in fp32.
//
// All are written in a form that keeps its RELATIVE accuracy where the
// result is small (negative z), because the result is rounded to fp16, whose
// steps shrink with it: sigmoid products instead of 1 + tanh, and the
// complementary error function's scaled form instead of 1 + erf. Measured
// against 64 bits on a million points, |z| <= 8: largest relative error silu
// 5e-7, gelu 3.3e-6, gelu_tanh 8e-6 (half a step of fp16 is 4.9e-4);
// derivatives 2e-6 absolute.
//
// At infinities and NaN each gives what its formula gives in IEEE arithmetic:
// a NaN stays one, act(+inf) is +inf, relu(-inf) is 0, and the others, which
// multiply -inf by 0 there, NaN.
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

// max(x, 0) that keeps a NaN (fmaxf would return the 0 and hide it)
__device__ __forceinline__ float relu1(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
  return r;
}

// Upper tail of the normal distribution, Q(a) = erfc(a / sqrt(2)) / 2 for
// a >= 0, as exp(-a^2 / 2) * R(a): R = erfcx(a / sqrt(2)) / 2 is smooth and
// slowly decreasing, and t * polynomial(t) in t = 1 / (1 + 0.26 a) fits it
// to 2.8e-7 relative on [0, 8] (a least-squares fit reweighted toward equal
// error, made in 64 bits for this file; 5.6e-7 when evaluated in fp32) and
// keeps its a -> infinity limit.
__host__ __device__ constexpr float tail_coeff(int i) {
  return i == 0 ? 0.10341634601354599f
       : i == 1 ? 0.10833492130041122f
       : i == 2 ? 0.06802142411470413f
       : i == 3 ? 0.17879557609558105f
       : i == 4 ? -0.12206314504146576f
       : i == 5 ? 0.23910772800445557f
                : -0.07561299204826355f;
}

constexpr float kTanhC0 = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhC1 = 0.044715f;

// Two fp32 values in one 64-bit register: one issue slot per pair for the
// sums and products. The epilogues of the wide tiles have as many
// instructions per output as the mainloop leaves room for, and the pairs
// halve their larger part.
struct F2 {
  uint64_t r;
};

__device__ __forceinline__ F2 f2(float x, float y) {
  F2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v.r) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 f2_get(F2 v) {
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(v.r));
  return o;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v.r) : "l"(a.r), "l"(b.r), "l"(c.r));
  return v;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v.r) : "l"(a.r), "l"(b.r));
  return v;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v.r) : "l"(a.r), "l"(b.r));
  return v;
}

__device__ __forceinline__ float fast_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ F2 f2_ex2(F2 x) {
  const float2 v = f2_get(x);
  return f2(fast_ex2(v.x), fast_ex2(v.y));
}
__device__ __forceinline__ F2 f2_rcp(F2 x) {
  const float2 v = f2_get(x);
  return f2(fast_rcp(v.x), fast_rcp(v.y));
}

constexpr float kLog2e = 1.4426950408889634f;

// Q(a), and exp(-a^2 / 2) in `gauss`
__device__ __forceinline__ F2 normal_tail2(F2 a, F2& gauss) {
  const F2 t = f2_rcp(f2_fma(a, f2(0.26f), f2(1.0f)));
  F2 r = f2(tail_coeff(6));
#pragma unroll
  for (int i = 5; i >= 0; --i) r = f2_fma(r, t, f2(tail_coeff(i)));
  gauss = f2_ex2(f2_mul(f2_mul(a, f2(-0.5f * kLog2e)), a));
  return f2_mul(f2_mul(r, t), gauss);
}

// z Phi(z) = max(z, 0) - |z| Q(|z|): no cancellation on either side. `m` holds
// -|z|, for positive z no lower than -64 (Q is 0 far before that): at
// +infinity, -infinity times 0 would make a NaN of a value that is +infinity.
__device__ __forceinline__ F2 gelu_of2(float2 v, F2 q) {
  const F2 m = f2(fminf(v.x, -fminf(v.x, 64.0f)), fminf(v.y, -fminf(v.y, 64.0f)));
  return f2_fma(m, q, f2(relu1(v.x), relu1(v.y)));
}

// 1 / (1 + exp(-z)), z scaled by -log2(e) already. exp overflows to infinity
// below z = -88.7: the reciprocal is then 0, as it should be to fp16.
__device__ __forceinline__ F2 f2_sigmoid_of(F2 neg_z_log2e) {
  return f2_rcp(f2_add(f2_ex2(neg_z_log2e), f2(1.0f)));
}

template <int ACT>
__device__ __forceinline__ F2 act_fwd2(F2 z) {
  if constexpr (ACT == kActRelu) {
    const float2 v = f2_get(z);
    return f2(relu1(v.x), relu1(v.y));
  } else if constexpr (ACT == kActSilu) {
    return f2_mul(z, f2_sigmoid_of(f2_mul(z, f2(-kLog2e))));
  } else if constexpr (ACT == kActGelu) {
    const float2 v = f2_get(z);
    F2 g;
    return gelu_of2(v, normal_tail2(f2(fabsf(v.x), fabsf(v.y)), g));
  } else if constexpr (ACT == kActGeluTanh) {
    // z (1 + tanh w) / 2 = z sigmoid(2 w), w = sqrt(2/pi) (z + 0.044715 z^3)
    constexpr float k = -2.0f * kTanhC0 * kLog2e;
    const F2 p = f2_fma(f2_mul(z, z), f2(k * kTanhC1), f2(k));
    return f2_mul(z, f2_sigmoid_of(f2_mul(z, p)));
  } else {
    return z;
  }
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  return f2_get(act_fwd2<ACT>(f2(z, z))).x;
}

// act(z) and act'(z)
template <int ACT>
__device__ __forceinline__ void act_fwd_bwd2(F2 z, F2& f, F2& d) {
  const F2 one = f2(1.0f), minus = f2(-1.0f);
  if constexpr (ACT == kActRelu) {
    const float2 v = f2_get(z);
    f = f2(relu1(v.x), relu1(v.y));
    d = f2(v.x > 0.0f ? 1.0f : 0.0f, v.y > 0.0f ? 1.0f : 0.0f);
  } else if constexpr (ACT == kActSilu) {
    // s + z s (1 - s): 1 - s cancels for large z, where it is a small part of
    // the sum
    const F2 s = f2_sigmoid_of(f2_mul(z, f2(-kLog2e)));
    f = f2_mul(z, s);
    d = f2_fma(f, f2_fma(s, minus, one), s);
  } else if constexpr (ACT == kActGelu) {
    // Phi(z) + z phi(z), Phi from the upper tail Q(|z|)
    const float2 v = f2_get(z);
    F2 g;
    const F2 q2 = normal_tail2(f2(fabsf(v.x), fabsf(v.y)), g);
    const float2 q = f2_get(q2);
    f = gelu_of2(v, q2);
    d = f2_fma(f2_mul(z, f2(0.3989422804014327f)), g, f2(v.x > 0.0f ? 1.0f - q.x : q.x, v.y > 0.0f ? 1.0f - q.y : q.y));
  } else if constexpr (ACT == kActGeluTanh) {
    constexpr float c = 2.0f * kTanhC0;
    const F2 z2 = f2_mul(z, z);
    const F2 s = f2_sigmoid_of(f2_mul(z, f2_fma(z2, f2(-c * kLog2e * kTanhC1), f2(-c * kLog2e))));
    f = f2_mul(z, s);
    d = f2_fma(f2_mul(f, f2_fma(s, minus, one)), f2_fma(z2, f2(3.0f * c * kTanhC1), f2(c)), s);
  } else {
    f = z;
    d = one;
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
