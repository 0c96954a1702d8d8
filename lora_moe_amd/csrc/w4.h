// Layout of a packed 4-bit matrix (w4.hip).  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "moe_lora.h"

namespace moelora {

struct W4Layout {
  int N, K, group, has_zeros;
  int tiles, chunks, G;  // 16-row tiles, 128-k chunks, groups along K
  size_t off_scales, off_zeros, total;
};

}  // namespace moelora
