// Activations of the layer operators and their derivatives, in fp32 (the
// formulas are in fp8bl_layers.h). Exponentials and quotients run on the
// hardware exp2 and reciprocal: a sigmoid is off by a relative
// (|v| + 4) 2^-23 at most, far below the half step of the bf16 results
// (2^-9) and of the same size as the fp32 sums' own rounding.
#pragma once

#include <hip/hip_runtime.h>

namespace fp8bl {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504088896341f));
}

constexpr float kTanhA2 = 1.59576912160573071f;       // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

template <int ACT>
__device__ __forceinline__ float act_f32(float t) {
  if constexpr (ACT == kActRelu) return t > 0.0f ? t : (t != t ? t : 0.0f);
  if constexpr (ACT == kActSilu) return t * sigmoid_f32(t);
  // Phi(t) = erfc(-t / sqrt 2) / 2 keeps its relative precision where Phi is
  // small; (1 + erf) / 2 would cancel there.
  if constexpr (ACT == kActGelu) return 0.5f * t * erfcf(-kSqrtHalf * t);
  if constexpr (ACT == kActGeluTanh) return t * sigmoid_f32(kTanhA2 * (t + kTanhB * t * t * t));
  return t;
}

template <int ACT>
__device__ __forceinline__ float act_grad_f32(float t) {
  if constexpr (ACT == kActRelu) return t > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == kActSilu) {
    const float p = sigmoid_f32(t);
    return p * (1.0f + t * (1.0f - p));
  }
  if constexpr (ACT == kActGelu)
    return 0.5f * erfcf(-kSqrtHalf * t) +
           t * (kInvSqrt2Pi * __builtin_amdgcn_exp2f(t * t * (-0.5f * 1.44269504088896341f)));
  if constexpr (ACT == kActGeluTanh) {
    // Past |t| = 30 the derivative is 0 or 1 in fp32; the clamp keeps t^2
    // finite there (0 * inf otherwise).
    const float c = fminf(fmaxf(t, -30.0f), 30.0f);
    const float p = sigmoid_f32(kTanhA2 * (c + kTanhB * c * c * c));
    const float r = p + c * p * (1.0f - p) * (kTanhA2 * (1.0f + 3.0f * kTanhB * c * c));
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
