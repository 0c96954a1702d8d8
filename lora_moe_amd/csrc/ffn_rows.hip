// The gated block's products for a few tokens (decode): see rows.h.
#include "ffn.h"
#include "rows_bf16.h"

namespace moelora {

namespace {

struct Bf16Weights : Bf16Stream {
  struct Args {
    const uint16_t* w;  // gate: [2N][K], gate rows then up rows
  };
  static constexpr bool RAW = false;
  static constexpr int MAX_FRAGMENTS = kRowsMax / 16;
  const uint16_t* w;
  int N;
  __device__ __forceinline__ Bf16Weights(const Args& a, int N_, int K_, int lane)
      : Bf16Stream(K_, lane), w(a.w), N(N_) {}
  // rows past N lie past the tile's bytes
  __device__ __forceinline__ Tile tile(int t, int half) const {
    const int rows = max(min(16, N - t * 16), 0);
    return Tile{w + (int64_t)(half * (int64_t)N + t * 16) * K, (uint32_t)rows * (uint32_t)K * 2u};
  }
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
