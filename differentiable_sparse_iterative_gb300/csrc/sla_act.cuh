// Activations of the gated feed-forward block and their derivatives, in float32.
//
//   silu       a = g s,            a' = s (1 + g (1 - s)),                 s = 1 / (1 + e^-g)
//   gelu       a = g Phi(g),       a' = Phi(g) + g phi(g),                 Phi, phi of the normal distribution
//   gelu_tanh  a = g (1 + t) / 2,  a' = (1 + t) / 2 + g (1 - t^2) z' / 2,  t = tanh z, z = sqrt(2/pi) (g + 0.044715 g^3)
//   relu       a = max(g, 0),      a' = [g > 0]
//
// They are taken for pairs of values: packed float32 arithmetic, the approximate exponential and
// reciprocal.  (expf, erff and division cost the float32 epilogue three times the instructions.)  Every activation is
// right relative to its own value, at negative gates too, where it is small: to 2^-19, and 2^-22 of the exponential's
// argument, whose rounding the exponential multiplies; below the rounding of 16-bit data, and for float32 data below
// what its sums lose.
//   sigmoid: 1 / (1 + e^-x).  As 1/2 + tanh(x/2) / 2 with the approximate tanh it would cost one special function in
//     place of two (narrow blocks: 158 us in place of 168), but be off by 2^-12 of one: a tenth of the value at x = -6.
//   gelu: 1 - Phi(x) = e^(-x^2/2) t P(t), t = 1 / (1 + 0.3 x), for x >= 0.  P is the polynomial of degree 7 with the
//     least relative error on 0 <= x <= 13.5 (found by linear programming; 9.3e-8, 4.4e-7 evaluated in float32); beyond, the
//     exponential is zero.  It is the density's exponential too.
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "sla_net.cuh"

namespace sla {

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^-x) of both.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 m = mul2(x, f2(-1.4426950408889634f, -1.4426950408889634f));
  const float2 d = add2(f2(ex2_approx(m.x), ex2_approx(m.y)), f2(1.f, 1.f));
  return f2(rcp_approx(d.x), rcp_approx(d.y));
}

// The activation of a pair; da: also its derivative.
template <int Act, bool Derivative>
__device__ __forceinline__ void activate2(float2 g, float2 &a, float2 &da) {
  const float2 one = f2(1.f, 1.f);
  if constexpr (Act == SLA_ACT_SILU) {
    const float2 s = sigmoid2(g);
    a = mul2(g, s);
    if (Derivative) da = fma2(a, fma2(s, f2(-1.f, -1.f), one), s);  // s + a (1 - s)
  } else if constexpr (Act == SLA_ACT_GELU) {
    const float2 x = f2(fabsf(g.x), fabsf(g.y));
    const float2 den = fma2(x, f2(0.3f, 0.3f), one);
    const float2 t = f2(rcp_approx(den.x), rcp_approx(den.y));
    float2 q = fma2(t, f2(0.03592418f, 0.03592418f), f2(-0.15823323f, -0.15823323f));
    q = fma2(q, t, f2(0.20810671f, 0.20810671f));
    q = fma2(q, t, f2(-0.055270962f, -0.055270962f));
    q = fma2(q, t, f2(0.12938385f, 0.12938385f));
    q = fma2(q, t, f2(0.09967073f, 0.09967073f));
    q = fma2(q, t, f2(0.12079171f, 0.12079171f));
    q = fma2(q, t, f2(0.11962691f, 0.11962691f));
    const float2 m = mul2(mul2(g, g), f2(-0.7213475204444817f, -0.7213475204444817f));
    const float2 e = f2(ex2_approx(m.x), ex2_approx(m.y));
    q = mul2(mul2(q, t), e);  // 1 - Phi(|g|)
    const float2 phi = f2(g.x < 0.f ? q.x : 1.f - q.x, g.y < 0.f ? q.y : 1.f - q.y);
    a = mul2(g, phi);
    if (Derivative) da = fma2(mul2(g, e), f2(0.3989422804014327f, 0.3989422804014327f), phi);
  } else if constexpr (Act == SLA_ACT_GELU_TANH) {
    // (1 + tanh z) / 2 = 1 / (1 + e^-2z);  with s that: 1 - t^2 = 4 s (1 - s)
    constexpr float c = 0.7978845608028654f, k = 2.f * c;
    const float2 gg = mul2(g, g);
    const float2 s = sigmoid2(mul2(g, fma2(gg, f2(k * 0.044715f, k * 0.044715f), f2(k, k))));
    a = mul2(g, s);
    if (Derivative) {
      const float2 dz = fma2(gg, f2(2.f * c * 3.f * 0.044715f, 2.f * c * 3.f * 0.044715f), f2(2.f * c, 2.f * c));
      // a (1 - s) first: far from zero one of the two is zero, while a z' may pass the largest float32
      da = fma2(mul2(a, fma2(s, f2(-1.f, -1.f), one)), dz, s);
    }
  } else {
    a = f2(g.x < 0.f ? 0.f : g.x, g.y < 0.f ? 0.f : g.y);
    da = f2(g.x > 0.f ? 1.f : 0.f, g.y > 0.f ? 1.f : 0.f);
  }
}

// h = act(g) u from g and u.  Keep: g and u become the factors of the backward pass, dg = dh (u act'(g)) and
// du = dh act(g).  They are what a forward call leaves behind, in the place of g and u: as many bytes, one
// rounding to the data's type each, and the backward epilogue is two products.  (With the rounding of dg and du, which
// 16-bit tensor-core operands need, and of the result that makes three for dx and dw_in: 0.0029 in relative L2 in
// bfloat16, 0.00036 in float16, where one rounding is 0.0017 and 0.00021.  g and u kept in 16
// bits, from which the factors would be formed again, make 0.0030; factors in 32 bits 0.0023, for twice the bytes.)
template <int Act, bool Keep, int N>
__device__ __forceinline__ void gate(float (&g)[N], float (&u)[N], float (&h)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    constexpr int next = N > 1;
    float2 a, da;
    const float2 up = f2(u[i], u[i + next]);
    activate2<Act, Keep>(f2(g[i], g[i + next]), a, da);
    const float2 v = mul2(a, up);
    h[i + next] = v.y, h[i] = v.x;
    if (Keep) {
      da = mul2(da, up);
      g[i + next] = da.y, g[i] = da.x, u[i + next] = a.y, u[i] = a.x;
    }
  }
}

// From v = dh and the factors:  g = dg, u = du.
template <int N>
__device__ __forceinline__ void gate_gradients(const float (&v)[N], float (&g)[N], float (&u)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 dh = f2(v[i], v[i + 1]);
    const float2 a = mul2(dh, f2(g[i], g[i + 1])), b = mul2(dh, f2(u[i], u[i + 1]));
    g[i] = a.x, g[i + 1] = a.y, u[i] = b.x, u[i + 1] = b.y;
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
