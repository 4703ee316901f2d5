// Activations of the gated feed-forward block, a(g) and a'(g), in fp32.
//   silu       a = g s,  s = 1 / (1 + e^-g);                     a' = s (1 + g (1 - s))
//   gelu       a = g P,  P = erfc(-g / sqrt 2) / 2;              a' = P + g e^(-g^2/2) / sqrt(2 pi)
//   gelu_tanh  a = g s,  s = 1 / (1 + e^-2v) = (1 + tanh v) / 2, v = sqrt(2/pi) (g + 0.044715 g^3);
//              a' = s + 2 g s (1 - s) v'
// The erfc and logistic forms keep the relative accuracy of the small values at large negative
// g, where 1 + erf and 1 + tanh cancel; e^x overflowing to infinity gives s = 0, as it should.
// The logistic uses __expf and __fdividef: documented to within 2 + floor(1.173 |x|) and 2 units in the
// last place (2^-23 relative), so that s is off by at most (4 + 1.173 |x|) 2^-23 of itself, 2^-16 where
// e^x leaves fp32's range (and 0 below 2^-126): far inside the outputs' fp16 rounding of 2^-11.
// With expf and a division the epilogue of a 256-token tile took 3 us more.
#pragma once
#include <type_traits>

#include "owq_internal.cuh"

namespace owq {

__device__ __forceinline__ float logistic(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

template <int ACT>
__device__ __forceinline__ void act_eval(float g, float& a, float& da) {
  if constexpr (ACT == OWQ_ACT_SILU) {
    const float s = logistic(g);
    a = g * s;
    da = s * (1.f + g * (1.f - s));
  } else if constexpr (ACT == OWQ_ACT_GELU) {
    const float p = 0.5f * erfcf(-g * 0.70710678118654752f);
    a = g * p;
    da = p + g * (expf(-0.5f * g * g) * 0.39894228040143268f);
  } else {
    constexpr float c = 0.79788456080286536f, k = 0.044715f;
    const float g2 = g * g;
    const float s = logistic(2.f * c * (g + k * g2 * g));
    a = g * s;
    da = s + g * (s * (1.f - s)) * (2.f * c * (1.f + 3.f * k * g2));
  }
}
// f(std::integral_constant<int, act>): one copy of the code around an activation per kind, so that
// no element branches on it (inlined in every element of an unrolled epilogue, the three forms
// were more code than the instruction cache holds).
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == OWQ_ACT_SILU) f(std::integral_constant<int, OWQ_ACT_SILU>{});
  else if (act == OWQ_ACT_GELU) f(std::integral_constant<int, OWQ_ACT_GELU>{});
  else f(std::integral_constant<int, OWQ_ACT_GELU_TANH>{});
}

}  // namespace owq
