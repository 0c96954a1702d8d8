// Host-side argument checks shared by the ABI sources.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moelora {

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

struct Range {
  const void* p;
  size_t bytes;
};

inline bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

// Whether an output shares memory with an input or with another output.
inline bool any_overlap(const Range* in, int n_in, const Range* out, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(out[i], in[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

}  // namespace moelora
