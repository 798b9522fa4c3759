// Activations of the gated feed-forward product and their derivatives.
#pragma once

#include <cuda_runtime.h>

#include "nystrom.h"

namespace nys {
namespace act {

// FAST (bf16 results): special-function unit. The exponential is then off by up to
// 2 + 1.173 |x| units in its last place (CUDA's bound for __expf): 2^-18 of itself at
// |x| = 25, 2^-16 at 87.
template <bool FAST>
__device__ __forceinline__ float exponential(float x) {
  return FAST ? __expf(x) : expf(x);
}
// 1 / (1 + e^-x) and what it leaves of one, 1 / (1 + e^x), from the exponential of
// -|x|, which cannot overflow: the smaller of the two keeps its bits down to 2^-126,
// and below that is off by 2^-149 (from e^-x, it was 0 from x = -88 on).
struct Sigmoid {
  float s, rest;
};
template <bool FAST>
__device__ __forceinline__ Sigmoid sigmoid(float x) {
  const float e = exponential<FAST>(-fabsf(x));
  const float large = FAST ? __fdividef(1.f, 1.f + e) : 1.f / (1.f + e), small = e * large;
  return x < 0.f ? Sigmoid{small, large} : Sigmoid{large, small};
}

// tanh as 2 sigmoid(2 z) - 1: the factor (1 + tanh z) / 2 then loses no bits
// where it is small. 2 sqrt(2/pi) = 1.5957691...
constexpr float kTanh1 = 1.59576912160573f, kTanh3 = kTanh1 * 0.044715f;

template <int ACT, bool FAST>
__device__ __forceinline__ float value(float g) {
  if (ACT == NYS_ACT_SILU) return g * sigmoid<FAST>(g).s;
  if (ACT == NYS_ACT_GELU) return 0.5f * g * erfcf(-0.70710678118654752f * g);
  if (ACT == NYS_ACT_GELU_TANH) return g * sigmoid<FAST>(g * fmaf(kTanh3, g * g, kTanh1)).s;
  return fmaxf(g, 0.f) + (g != g ? g : 0.f);  // NaN stays NaN
}

// act(g) and act'(g).
template <int ACT, bool FAST>
__device__ __forceinline__ void with_slope(float g, float& a, float& slope) {
  if (ACT == NYS_ACT_SILU) {
    const Sigmoid y = sigmoid<FAST>(g);
    a = g * y.s;
    slope = y.s * fmaf(g, y.rest, 1.f);
  } else if (ACT == NYS_ACT_GELU) {
    const float p = 0.5f * erfcf(-0.70710678118654752f * g);
    a = g * p;
    slope = fmaf(0.39894228040143268f * g, exponential<FAST>(-0.5f * g * g), p);
  } else if (ACT == NYS_ACT_GELU_TANH) {
    const Sigmoid y = sigmoid<FAST>(g * fmaf(kTanh3, g * g, kTanh1));
    a = g * y.s;
    // from |g| = 16 on one of the factors is 0; g^2 itself would pass fp32's range
    slope = fmaf(g * y.s * y.rest, fmaf(3.f * kTanh3, fminf(g * g, 256.f), kTanh1), y.s);
  } else {
    a = value<NYS_ACT_RELU, FAST>(g);
    slope = g > 0.f ? 1.f : (g != g ? g : 0.f);
  }
}

// f(std::integral_constant<int, ACT>) for a run-time choice.
template <typename F>
__host__ __device__ __forceinline__ auto by_act(int a, F&& f) {
  switch (a) {
    case NYS_ACT_SILU: return f(std::integral_constant<int, NYS_ACT_SILU>{});
    case NYS_ACT_GELU: return f(std::integral_constant<int, NYS_ACT_GELU>{});
    case NYS_ACT_GELU_TANH: return f(std::integral_constant<int, NYS_ACT_GELU_TANH>{});
    default: return f(std::integral_constant<int, NYS_ACT_RELU>{});
  }
}

}  // namespace act
}  // namespace nys
