// The gates of the feed-forward block and their derivatives, in fp32.
//
// Both are act(g) = g * S(p(g)) with the logistic S(v) = 1 / (1 + exp(-v)):
//   silu  p(g) = g
//   gelu  p(g) = 2c (g + 0.044715 g^3), c = sqrt(2 / pi): the tanh form, as
//         (1 + tanh z) / 2 = S(2z), which keeps its relative precision where
//         1 + tanh z cancels
// so act'(g) = S + g S (1 - S) p'(g).
#pragma once

#include <hip/hip_runtime.h>

#include "moe_lora.h"

namespace moelora {

template <bool GRAD>
__device__ __forceinline__ float gate_act(int act, float g, float* grad) {
  float p = g, dp = 1.f;
  if (act == MOE_LORA_ACT_GELU) {
    // S(p) is exactly 0 or 1 from |g| = 30 on; the bound keeps g^3 finite
    const float t = fminf(fmaxf(g, -30.f), 30.f);
    constexpr float c2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float q = 0.044715f * t * t;
    p = c2 * t * (1.f + q);
    dp = c2 * (1.f + 3.f * q);
  }
  const float s = 1.f / (1.f + __expf(-p));
  if (GRAD) *grad = s + g * s * (1.f - s) * dp;
  return g * s;
}

}  // namespace moelora
