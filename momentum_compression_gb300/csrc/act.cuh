// The activations of the dense layer and their slopes, in fp32.
//
// GELU by Phi(z) = 1 - q(z) for z >= 0 and q(|z|) else, q(a) = erfc(a / sqrt 2) / 2.
// q(a) e^(a^2 / 2) falls slowly from 1/2 to 1/40 at a = 16; it is t P(t), t = 1 / (1 + 0.35 a),
// the form of Abramowitz and Stegun's 7.1.26.  That formula is off by 1.5e-7 whatever the
// value, which is 2% of q(10); P here was fitted (linear programming over 3000 points of
// [0, 16]) to be off by at most 4e-8 and 5e-6 of q(a) itself, fp32's roundings apart, so that
// a small y has its digits too: a step of bf16 is 4e-3 of a value, of fp16 5e-4.  One
// exponential, one reciprocal and ten multiply-adds; its slope has the same exponential.  The
// two multiply-adds more than 7.1.26's cost 16384 x 4096 x 1024 bf16 nothing forward (107 us)
// and make dz 74 us from 70.  The tanh form is z / (1 + e^(-2u)).
#pragma once

#include <type_traits>

#include "ob.h"
#include "tc.cuh"

namespace ob {

__device__ __forceinline__ float act_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float act_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A NaN in either comes out.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

constexpr float kActLog2e = 1.44269504f;

constexpr float kTailP = 0.35f;
constexpr float kTail0 = 0.139765867f, kTail1 = 0.137003896f, kTail2 = 0.142531257f,
                kTail3 = 0.0103732789f, kTail4 = 0.209318047f, kTail5 = -0.183337167f,
                kTail6 = 0.0443448548f;

// e^(-z^2 / 2) in *bell, erfc(|z| / sqrt 2) / 2 returned; |z| <= 16.
__device__ __forceinline__ float half_erfc(float size, float* bell) {
  const float t = act_rcp(__fmaf_rn(kTailP, size, 1.0f));
  float p = __fmaf_rn(t, kTail6, kTail5);
  p = __fmaf_rn(p, t, kTail4);
  p = __fmaf_rn(p, t, kTail3);
  p = __fmaf_rn(p, t, kTail2);
  p = __fmaf_rn(p, t, kTail1);
  p = __fmaf_rn(p, t, kTail0);
  *bell = act_ex2(size * size * (-0.5f * kActLog2e));
  return p * t * *bell;
}

constexpr float kTanhA = 0.7978845608f, kTanhB = 0.044715f;  // sqrt(2 / pi)

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if (ACT == OB_ACT_RELU) return max_nan(z, 0.0f);
  if (ACT == OB_ACT_GELU) {
    float bell;
    const float size = fminf(fabsf(z), 16.0f);  // further out the weight is 0 (of infinity too)
    return __fmaf_rn(-size, half_erfc(size, &bell), max_nan(z, 0.0f));
  }
  if (ACT == OB_ACT_GELU_TANH) {
    const float c = max_nan(z, -16.0f);
    const float u = c * __fmaf_rn(kTanhA * kTanhB, c * c, kTanhA);
    return c * act_rcp(1.0f + act_ex2(u * (-2.0f * kActLog2e)));
  }
  return z;
}

// Of two values at a time, two an instruction; the same bits as act_of's.
template <int ACT>
__device__ __forceinline__ void act_of2(float& z0, float& z1) {
  if (ACT == OB_ACT_GELU) {
    const float s0 = fminf(fabsf(z0), 16.0f), s1 = fminf(fabsf(z1), 16.0f);
    const uint64_t size = pair(s0, s1);
    auto both = [](float x) { return pair(x, x); };
    float t0, t1, e0, e1;
    unpair(fma2(both(kTailP), size, both(1.0f)), &t0, &t1);
    const uint64_t t = pair(act_rcp(t0), act_rcp(t1));
    uint64_t p = fma2(t, both(kTail6), both(kTail5));
    p = fma2(p, t, both(kTail4));
    p = fma2(p, t, both(kTail3));
    p = fma2(p, t, both(kTail2));
    p = fma2(p, t, both(kTail1));
    p = fma2(p, t, both(kTail0));
    unpair(mul2(mul2(size, size), both(-0.5f * kActLog2e)), &e0, &e1);
    const uint64_t tail = mul2(mul2(p, t), pair(act_ex2(e0), act_ex2(e1)));
    unpair(fma2(pair(-s0, -s1), tail, pair(max_nan(z0, 0.0f), max_nan(z1, 0.0f))), &z0, &z1);
    return;
  }
  z0 = act_of<ACT>(z0);
  z1 = act_of<ACT>(z1);
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == OB_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if (ACT == OB_ACT_GELU) {
    float bell;
    const float size = fminf(fabsf(z), 16.0f), tail = half_erfc(size, &bell);
    const float phi = z < 0.0f ? tail : 1.0f - tail;
    // a NaN stays one; size = 16 of an infinity has no bell left
    return z != z ? z : __fmaf_rn(copysignf(size, z) * 0.3989422804f, bell, phi);
  }
  if (ACT == OB_ACT_GELU_TANH) {
    const float c = max_nan(fminf(z, 16.0f), -16.0f);
    const float u = c * __fmaf_rn(kTanhA * kTanhB, c * c, kTanhA);
    const float s = act_rcp(1.0f + act_ex2(u * (-2.0f * kActLog2e)));
    const float du = __fmaf_rn(3.0f * kTanhA * kTanhB, c * c, kTanhA);
    return z != z ? z : __fmaf_rn(2.0f * c * s * (1.0f - s), du, s);
  }
  return 1.0f;
}

// f(std::integral_constant<int, act>) for the run-time code.
template <typename F>
__device__ __forceinline__ void by_act(int act, F f) {
  if (act == OB_ACT_NONE)
    f(std::integral_constant<int, OB_ACT_NONE>());
  else if (act == OB_ACT_RELU)
    f(std::integral_constant<int, OB_ACT_RELU>());
  else if (act == OB_ACT_GELU)
    f(std::integral_constant<int, OB_ACT_GELU>());
  else
    f(std::integral_constant<int, OB_ACT_GELU_TANH>());
}

}  // namespace ob
