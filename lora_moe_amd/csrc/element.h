// Elements of the types that a caller names (MOE_LORA_F32, _BF16, _F16), 16
// bytes at a time, as fp32.
#pragma once

#include "device_util.h"
#include "moe_lora.h"

namespace moelora {

inline size_t element_size(int32_t dtype) { return dtype == MOE_LORA_F32 ? 4 : 2; }
inline bool is_element(int32_t dtype) {
  return dtype == MOE_LORA_F32 || dtype == MOE_LORA_BF16 || dtype == MOE_LORA_F16;
}

template <int DT>
struct Elements {
  static constexpr int N = DT == MOE_LORA_F32 ? 4 : 8;

  static __device__ __forceinline__ void load(u32x4_t q, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE_LORA_F32) {
        v[i] = __uint_as_float(q[i]);
      } else if constexpr (DT == MOE_LORA_BF16) {
        v[2 * i] = bf16_lo(q[i]);
        v[2 * i + 1] = bf16_hi(q[i]);
      } else {
        v[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)q[i]);
        v[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(q[i] >> 16));
      }
    }
  }

  // rounded to nearest even
  static __device__ __forceinline__ u32x4_t store(const float* v) {
    u32x4_t q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == MOE_LORA_F32) {
        q[i] = __float_as_uint(v[i]);
      } else if constexpr (DT == MOE_LORA_BF16) {
        q[i] = f32x2_to_bf16(v[2 * i], v[2 * i + 1]);
      } else {
        q[i] = __builtin_bit_cast(uint16_t, (_Float16)v[2 * i]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i + 1]) << 16;
      }
    }
    return q;
  }
};

}  // namespace moelora
