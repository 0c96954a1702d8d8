// bf16 weights as a stream for rows.h: rows of K values, k contiguous.  A load
// covers 16 rows x 64 bytes, two neighbouring ones whole lines.
#pragma once

#include "rows.h"

namespace moelora {

struct Bf16Stream {
  static constexpr int DEPTH = 2;
  static constexpr int LINES = 32;  // of 128 bytes, per chunk of a tile
  struct Tile {
    const uint16_t* base;
    uint32_t bytes;
  };
  struct Buf {
    u32x4_t v[4];
  };
  int K, kq;
  uint32_t off;
  __device__ __forceinline__ Bf16Stream(int K_, int lane)
      : K(K_), kq(lane >> 4), off(((uint32_t)(lane & 15) * (uint32_t)K_ + (uint32_t)(lane >> 4) * 8u) * 2u) {}
  __device__ __forceinline__ void load(Buf& b, const Tile& t, int c, bool real) const {
    const int left = real ? K - c * 128 : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t o = j * 32 + kq * 8 < left ? off + j * 64 : kBufNone;
      b.v[j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(t.base, t.bytes), (int)o,
                                                                                 c * 256, 2));  // non-temporal
    }
  }
  __device__ __forceinline__ u32x4_t operand(const Buf& b, int j) const { return b.v[j]; }

  template <int RF, int CT>
  struct Acc {
    f32x4_t a[RF][CT];
    __device__ __forceinline__ void clear() {
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int t = 0; t < CT; ++t) a[f][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    __device__ __forceinline__ void begin(const Bf16Stream&, const Buf*, int) {}
    __device__ __forceinline__ void rows(int, u32x4_t) {}
    __device__ __forceinline__ void mul(int f, int t, u32x4_t x, u32x4_t w) { a[f][t] = mfma_16x16x32(x, w, a[f][t]); }
    __device__ __forceinline__ void end(const Bf16Stream&, const Buf*, int) {}
    __device__ __forceinline__ f32x4_t sum(int f, int t) const { return a[f][t]; }
  };
};

}  // namespace moelora
