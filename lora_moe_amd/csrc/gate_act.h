// The gates of the feed-forward block and their derivatives, in fp32.
//
// Both are act(g) = g * S(p(g)) with the logistic S(v) = 1 / (1 + exp(-v)) and
//   p(g) = c g (1 + k g^2),  p'(g) = c (1 + 3 k g^2)
//   silu  c = 1, k = 0
//   gelu  c = 2 sqrt(2 / pi), k = 0.044715: the tanh form, as (1 + tanh z) / 2
//         = S(2z), which keeps its relative precision where 1 + tanh z cancels
// so act'(g) = S + g S (1 - S) p'(g).
#pragma once

#include <hip/hip_runtime.h>

#include "moe_lora.h"

namespace moelora {

template <bool GRAD>
__device__ __forceinline__ float gate_act(int act, float g, float* grad) {
  const bool gelu = act == MOE_LORA_ACT_GELU;
  const float c = gelu ? 1.5957691216057308f : 1.f, k = gelu ? 0.044715f : 0.f;
  // S is exactly 0 or 1 from these bounds on; they keep g^2 and g^3 finite
  const float bound = gelu ? 30.f : 1e18f;
  const float t = fminf(fmaxf(g, -bound), bound);
  const float q = k * t * t;
  // (the reciprocal instruction, 1 ulp: a correctly rounded division is ten)
  const float s = __builtin_amdgcn_rcpf(1.f + __expf(-c * t * (1.f + q)));
  if (GRAD) *grad = s + g * s * (1.f - s) * (c * (1.f + 3.f * q));
  return g * s;
}

}  // namespace moelora
