// The gated block's products for a few tokens (decode): see rows.h.
#include "ffn.h"
#include "rows.h"

namespace moelora {

namespace {

// bf16 weights [rows][K], k contiguous.  A load covers 16 rows x 64 bytes, two
// neighbouring ones whole lines.
struct Bf16Weights {
  struct Args {
    const uint16_t* w;  // gate: [2N][K], gate rows then up rows
  };
  static constexpr int DEPTH = 2;
  static constexpr int LINES = 32;  // of 128 bytes, per chunk of a tile
  static constexpr int MAX_FRAGMENTS = kRowsMax / 16;
  struct Tile {
    const uint16_t* base;
    uint32_t bytes;
  };
  struct Buf {
    u32x4_t v[4];
  };
  const uint16_t* w;
  int N, K, kq;
  uint32_t off;
  __device__ __forceinline__ Bf16Weights(const Args& a, int N_, int K_, int lane)
      : w(a.w), N(N_), K(K_), kq(lane >> 4), off(((uint32_t)(lane & 15) * (uint32_t)K_ + (uint32_t)(lane >> 4) * 8u) * 2u) {}
  // rows past N lie past the tile's bytes
  __device__ __forceinline__ Tile tile(int t, int half) const {
    const int rows = max(min(16, N - t * 16), 0);
    return Tile{w + (int64_t)(half * (int64_t)N + t * 16) * K, (uint32_t)rows * (uint32_t)K * 2u};
  }
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
    __device__ __forceinline__ void begin(const Bf16Weights&, const Buf*, int) {}
    __device__ __forceinline__ void rows(int, u32x4_t) {}
    __device__ __forceinline__ void mul(int f, int t, u32x4_t x, u32x4_t w) { a[f][t] = mfma_16x16x32(x, w, a[f][t]); }
    __device__ __forceinline__ void end(const Bf16Weights&, const Buf*, int) {}
    __device__ __forceinline__ f32x4_t sum(int f, int t) const { return a[f][t]; }
  };
};

}  // namespace

int launch_ffn_rows(const FfnGemm& g, FfnProduct product, const uint16_t* a_lo, uint16_t* out_lo, hipStream_t st) {
  const RowsArgs a{g.A, a_lo, g.out, out_lo, g.gu, g.M, g.N, g.K, g.act, g.slabs, 1, 0};
  const Bf16Weights::Args wa{g.B};
  if (product == FFN_GATE_UP) launch_rows<Bf16Weights, true, false>(a, wa, st);
  else if (a_lo) launch_rows<Bf16Weights, false, true>(a, wa, st);
  else launch_rows<Bf16Weights, false, false>(a, wa, st);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

size_t ffn_rows_slab_bytes(int T, int H, int I) {
  const int lines = Bf16Weights::LINES;
  return std::max(rows_slab_bytes(rows_plan(T, I, H, lines), T, I, true),
                  rows_slab_bytes(rows_plan(T, H, I, lines), T, H, false));
}

}  // namespace moelora
