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
  struct Tile {
    const uint16_t* row;  // this lane's row at its first k
  };
  struct Buf {
    u32x4_t v[4];
  };
  const uint16_t* w;
  int N, K, kq, l16;
  __device__ __forceinline__ Bf16Weights(const Args& a, const RowsArgs& p, int lane)
      : w(a.w), N(p.N), K(p.K), kq(lane >> 4), l16(lane & 15) {}
  __device__ __forceinline__ Tile tile(int t, int half) const {
    return Tile{w + (int64_t)(half * N + min(t * 16 + l16, N - 1)) * K + kq * 8};
  }
  __device__ __forceinline__ void load(Buf& b, const Tile& t, int c, bool masked) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = c * 128 + j * 32;
      b.v[j] = !masked || k + kq * 8 < K ? ld16_stream(t.row + k) : zero4();
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
    __device__ __forceinline__ void rows(int, const u32x4_t&) {}
    __device__ __forceinline__ void mul(int f, int t, u32x4_t x, u32x4_t w) { a[f][t] = mfma_16x16x32(x, w, a[f][t]); }
    __device__ __forceinline__ void step(const Bf16Weights&, const Tile*, const Buf*, int, int) {}
    __device__ __forceinline__ f32x4_t sum(int f, int t) const { return a[f][t]; }
  };
};

template <bool GATE, bool PAIR>
void launch(const RowsArgs& a, const uint16_t* w, hipStream_t st) {
  const Bf16Weights::Args wa{w};
  constexpr int CT1 = GATE ? 2 : 1;
  if (a.M <= 16) launch_rows_cfg<Bf16Weights, 1, CT1, GATE, PAIR>(a, wa, st);
  if constexpr (!PAIR) {
    if (a.M > 16 && a.M <= 32) launch_rows_cfg<Bf16Weights, 2, 2, GATE, false>(a, wa, st);
    if (a.M > 32) launch_rows_cfg<Bf16Weights, 4, 2, GATE, false>(a, wa, st);
  }
}

}  // namespace

int launch_ffn_rows(const FfnGemm& g, FfnProduct product, const uint16_t* a_lo, uint16_t* out_lo, hipStream_t st) {
  const RowsArgs a{g.A, a_lo, g.out, out_lo, g.M, g.N, g.K, g.act};
  if (product == FFN_GATE_UP) launch<true, false>(a, g.B, st);
  else if (a_lo) launch<false, true>(a, g.B, st);
  else launch<false, false>(a, g.B, st);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // namespace moelora
