// Activations of the layer operators and their derivatives, in fp32 (the
// formulas are in fp8bl_layers.h). Exponentials and quotients run on the
// hardware exp2 and reciprocal: a sigmoid is off by a relative
// (2 |v| + 4) 2^-23 at most (the product in the exponent is off by |v| times
// its roundings), far below the half step of the bf16 results (2^-8) and of
// the same size as the fp32 sums' own rounding.
#pragma once

#include <hip/hip_runtime.h>

namespace fp8bl {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

constexpr float kLog2E = 1.44269504088896341f;
__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2E));
}

constexpr float kTanhA2 = 1.59576912160573071f;       // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;
// The tanh form's p = 1 / (1 + e^-v), v = A2 t (1 + B t^2), with -A2 log2(e)
// folded into the polynomial: the epilogue of many rows is bound by these
// instructions.
__device__ __forceinline__ float tanh_cdf(float t) {
  constexpr double a = -1.59576912160573071 * 1.44269504088896341;
  const float e = t * __builtin_fmaf(t * t, (float)(a * 0.044715), (float)a);
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(e));
}
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// The normal distribution's tail Phi(-a), a >= 0, with e = e^(-a^2/2):
// Phi(-a) e^(a^2/2) is smooth and slowly varying, here a polynomial of degree
// 7 in 1 / (1 + 0.35 a), fitted by reweighted least squares to the smallest
// largest relative error on 0 <= a <= 14.5 (beyond, e is 0): 3.6e-7 with these
// coefficients, 6.0e-7 evaluated in fp32. e's exponent is rounded to fp32, which
// adds a^2 2^-24 to the tail's relative error (2.2e-6 in all at a = 6, 8e-6 at
// a = 13): still far inside the half step where Phi is small, as (1 + erf) / 2
// would not be. About 14 instructions with no branch; the library's erfcf took
// 150 us of 894 us in the epilogue of 8192 x 12288 x 4096.
__device__ __forceinline__ float normal_tail(float a, float& e) {
  e = __builtin_amdgcn_exp2f(a * a * (-0.5f * kLog2E));
  const float s = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35f, a, 1.0f));
  float p = 0.04890687018632889f;
  p = __builtin_fmaf(p, s, -0.2019839733839035f);
  p = __builtin_fmaf(p, s, 0.2404298037290573f);
  p = __builtin_fmaf(p, s, -0.016849324107170105f);
  p = __builtin_fmaf(p, s, 0.15587973594665527f);
  p = __builtin_fmaf(p, s, 0.1333768665790558f);
  p = __builtin_fmaf(p, s, 0.14026731252670288f);
  p = __builtin_fmaf(p, s, -2.7144789783051237e-05f);
  return e * p;
}
__device__ __forceinline__ float normal_cdf(float t, float& e) {
  const float tail = normal_tail(fabsf(t), e);
  return t < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_f32(float t) {
  if constexpr (ACT == kActRelu) return t > 0.0f ? t : (t != t ? t : 0.0f);
  if constexpr (ACT == kActSilu) return t * sigmoid_f32(t);
  if constexpr (ACT == kActGelu) {
    float e;
    return t * normal_cdf(t, e);
  }
  if constexpr (ACT == kActGeluTanh) return t * tanh_cdf(t);
  return t;
}

template <int ACT>
__device__ __forceinline__ float act_grad_f32(float t) {
  if constexpr (ACT == kActRelu) return t > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == kActSilu) {
    const float p = sigmoid_f32(t);
    return p * (1.0f + t * (1.0f - p));
  }
  if constexpr (ACT == kActGelu) {
    float e;
    const float c = normal_cdf(t, e);
    return c + t * (kInvSqrt2Pi * e);
  }
  if constexpr (ACT == kActGeluTanh) {
    // Past |t| = 30 the derivative is 0 or 1 in fp32; the clamp keeps t^2
    // finite there (0 * inf otherwise).
    const float c = fminf(fmaxf(t, -30.0f), 30.0f);
    const float p = tanh_cdf(c);
    const float dv = __builtin_fmaf(c * c, 3.0f * kTanhB * kTanhA2, kTanhA2);
    const float r = __builtin_fmaf(c * p, (1.0f - p) * dv, p);
    return t != t ? t : r;                              // fmin and fmax drop a NaN
  }
  return 1.0f;
}

// The activation chosen at run time (a wave-uniform value), for epilogues
// that finish a few outputs a lane.
__device__ __forceinline__ float act_any(int act, float t) {
  switch (act) {
    case kActRelu: return act_f32<kActRelu>(t);
    case kActSilu: return act_f32<kActSilu>(t);
    case kActGelu: return act_f32<kActGelu>(t);
    case kActGeluTanh: return act_f32<kActGeluTanh>(t);
    default: return t;
  }
}

// One call site per activation: `f` is a generic lambda called with the
// activation as a compile-time constant.
template <int A>
struct ActTag {
  static constexpr int value = A;
};
template <typename F>
auto with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: return f(ActTag<kActRelu>{});
    case kActSilu: return f(ActTag<kActSilu>{});
    case kActGelu: return f(ActTag<kActGelu>{});
    case kActGeluTanh: return f(ActTag<kActGeluTanh>{});
    default: return f(ActTag<kActNone>{});
  }
}

}  // namespace fp8bl
