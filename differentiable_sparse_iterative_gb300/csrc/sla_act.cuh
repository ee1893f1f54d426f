// Activations of the gated feed-forward block and their derivatives, in float32.
//
//   silu       a = g s,            a' = s (1 + g (1 - s)),                 s = 1 / (1 + e^-g)
//   gelu       a = g Phi(g),       a' = Phi(g) + g phi(g),                 Phi, phi of the normal distribution
//   gelu_tanh  a = g (1 + t) / 2,  a' = (1 + t) / 2 + g (1 - t^2) z' / 2,  t = tanh z, z = sqrt(2/pi) (g + 0.044715 g^3)
//   relu       a = max(g, 0),      a' = [g > 0]
//
// Fast: the hardware's approximate exponential and division, for data of 16 bits (their error of
// a few 2^-22 disappears in the rounding to 2^-9 or 2^-12); float32 data takes expf, erff, tanhf.
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "sla.h"

namespace sla {

template <bool Fast>
__device__ __forceinline__ float sigmoid(float g) {
  return Fast ? __fdividef(1.f, 1.f + __expf(-g)) : 1.f / (1.f + expf(-g));
}

// 1 - 2 / (1 + e^2z): 1 and -1 at the ends, where e^2z is infinite or zero
template <bool Fast>
__device__ __forceinline__ float tanh_of(float z) {
  return Fast ? 1.f - 2.f * sigmoid<true>(-2.f * z) : tanhf(z);
}

struct ActValue {
  float a, da;
};

template <int Act, bool Fast>
__device__ __forceinline__ ActValue activate(float g) {
  if constexpr (Act == SLA_ACT_SILU) {
    const float s = sigmoid<Fast>(g);
    return {g * s, s * (1.f + g * (1.f - s))};
  } else if constexpr (Act == SLA_ACT_GELU) {
    const float phi = 0.5f * (1.f + erff(g * 0.7071067811865476f));
    const float e = Fast ? __expf(-0.5f * g * g) : expf(-0.5f * g * g);
    return {g * phi, phi + g * e * 0.3989422804014327f};
  } else if constexpr (Act == SLA_ACT_GELU_TANH) {
    const float z = 0.7978845608028654f * (g + 0.044715f * g * g * g);
    const float t = tanh_of<Fast>(z);
    return {0.5f * g * (1.f + t), 0.5f * (1.f + t) + 0.5f * g * (1.f - t * t) * 0.7978845608028654f *
                                                          (1.f + 3.f * 0.044715f * g * g)};
  } else {
    // written so that a NaN stays one
    return {g < 0.f ? 0.f : g, g > 0.f ? 1.f : 0.f};
  }
}

// Calls f with the activation as a constant: one branch for a whole loop, not one for each value.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F &&f) {
  switch (act) {
    case SLA_ACT_SILU: f(std::integral_constant<int, SLA_ACT_SILU>{}); break;
    case SLA_ACT_GELU: f(std::integral_constant<int, SLA_ACT_GELU>{}); break;
    case SLA_ACT_GELU_TANH: f(std::integral_constant<int, SLA_ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, SLA_ACT_RELU>{});
  }
}

}  // namespace sla
