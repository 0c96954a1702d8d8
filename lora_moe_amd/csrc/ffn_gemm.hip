// Products of the gated feed-forward block: bf16 MFMA, fp32 sums.
#include "device_util.h"
#include "ffn.h"
#include "gate_act.h"

namespace moelora {

namespace {

// 128 x 128 outputs per workgroup of 2 x 2 wavefronts (64 x 64 each), K in
// steps of 32 through LDS rows padded to 40 elements.
constexpr int BM = 128, BN = 128, BK = 32, PAD = 40;

// Rows [r0, r0 + 128) x k [k0, k0 + 32) of an operand into LDS, k contiguous
// there.  KC: k is contiguous in memory.  row(i): memory row of tile row i
// (KC only).  What lies outside is zero.
template <bool KC, class RowOf>
__device__ __forceinline__ void stage(uint16_t* lds, const uint16_t* p, int64_t ld, int r0, int rows, int k0, int K,
                                      RowOf row) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = (int)threadIdx.x + 256 * j;
    if (KC) {
      const int r = c >> 2, k = (c & 3) * 8;
      const int64_t mr = row(r);
      const u32x4_t v = mr >= 0 && k0 + k < K ? ld16(p + mr * ld + k0 + k) : zero4();
      *reinterpret_cast<u32x4_t*>(lds + r * PAD + k) = v;
    } else {
      const int k = c >> 4, r = (c & 15) * 8;
      const u32x4_t v = k0 + k < K && r0 + r < rows ? ld16(p + (int64_t)(k0 + k) * ld + r0 + r) : zero4();
#pragma unroll
      for (int i = 0; i < 8; ++i) lds[(r + i) * PAD + k] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
  }
}

template <int PRODUCT>
__global__ __launch_bounds__(256) void ffn_gemm_kernel(FfnGemm p) {
  constexpr bool A_KC = PRODUCT != FFN_DW;
  constexpr bool B_KC = PRODUCT == FFN_GATE_UP || PRODUCT == FFN_DOWN;
  constexpr bool GATE = PRODUCT == FFN_GATE_UP;
  __shared__ __attribute__((aligned(16))) uint16_t As[BM * PAD], Bs[BN * PAD];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, l16 = lane & 15, kq = lane >> 4;
  const int m0 = blockIdx.y * BM;
  const int n0 = blockIdx.x * (GATE ? BN / 2 : BN);
  // gate_up: tile columns [64w, 64w + 64) are gate n0 + 32w + [0, 32), then
  // the up columns of the same outputs
  auto brow = [&](int c) -> int64_t {
    if (GATE) {
      const int n = n0 + (c >> 6) * 32 + (c & 31);
      return n < p.N ? ((c >> 5) & 1 ? p.N + n : n) : -1;
    }
    return n0 + c < p.N ? n0 + c : -1;
  };
  auto arow = [&](int r) -> int64_t { return m0 + r < p.M ? m0 + r : -1; };
  f32x4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < p.K; k0 += BK) {
    __syncthreads();
    stage<A_KC>(As, p.A, p.lda, m0, p.M, k0, p.K, arow);
    stage<B_KC>(Bs, p.B, p.ldb, n0, p.N, k0, p.K, brow);
    __syncthreads();
    u32x4_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = *reinterpret_cast<const u32x4_t*>(As + (wm * 64 + i * 16 + l16) * PAD + kq * 8);
      b[i] = *reinterpret_cast<const u32x4_t*>(Bs + (wn * 64 + i * 16 + l16) * PAD + kq * 8);
    }
    // B first: a lane ends with 4 neighbouring columns of one row
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = mfma_16x16x32(b[j], a[i], acc[i][j]);
  }
  auto pack4 = [](const float* v) {
    uint2 o;
    o.x = f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16);
    o.y = f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16);
    return o;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + wm * 64 + i * 16 + l16;
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < (GATE ? 2 : 4); ++j) {
      const int n = GATE ? n0 + wn * 32 + j * 16 + kq * 4 : n0 + wn * 64 + j * 16 + kq * 4;
      if (n >= p.N) continue;
      float v[4], w[4], h[4];
      if (GATE) {
        const f32x4_t g = acc[i][j], u = acc[i][j + 2];
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = gate_act<false>(p.act, g[q], nullptr) * u[q];
        *reinterpret_cast<uint2*>(p.out + (int64_t)m * p.N + n) = pack4(h);
        if (p.gu) {
          *reinterpret_cast<f32x4_t*>(p.gu + (int64_t)m * 2 * p.N + n) = g;
          *reinterpret_cast<f32x4_t*>(p.gu + (int64_t)m * 2 * p.N + p.N + n) = u;
        }
      } else if (PRODUCT == FFN_DH) {
        const f32x4_t g = *reinterpret_cast<const f32x4_t*>(p.gu + (int64_t)m * 2 * p.N + n);
        const f32x4_t u = *reinterpret_cast<const f32x4_t*>(p.gu + (int64_t)m * 2 * p.N + p.N + n);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float da;
          const float a = gate_act<true>(p.act, g[q], &da), dh = acc[i][j][q];
          h[q] = a * u[q];
          v[q] = dh * u[q] * da;
          w[q] = dh * a;
        }
        *reinterpret_cast<uint2*>(p.out + (int64_t)m * 2 * p.N + n) = pack4(v);
        *reinterpret_cast<uint2*>(p.out + (int64_t)m * 2 * p.N + p.N + n) = pack4(w);
        *reinterpret_cast<uint2*>(p.out2 + (int64_t)m * p.N + n) = pack4(h);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = acc[i][j][q];
        *reinterpret_cast<uint2*>(p.out + (int64_t)m * p.N + n) = pack4(v);
      }
    }
  }
}

template <int PRODUCT>
void launch(const FfnGemm& g, hipStream_t st) {
  const int bn = PRODUCT == FFN_GATE_UP ? BN / 2 : BN;
  ffn_gemm_kernel<PRODUCT><<<dim3((g.N + bn - 1) / bn, (g.M + BM - 1) / BM), 256, 0, st>>>(g);
}

}  // namespace

int launch_ffn_gemm(const FfnGemm& g, FfnProduct product, hipStream_t st) {
  if (g.M == 0 || g.N == 0) return MOE_LORA_OK;
  switch (product) {
    case FFN_GATE_UP: launch<FFN_GATE_UP>(g, st); break;
    case FFN_DOWN: launch<FFN_DOWN>(g, st); break;
    case FFN_DH: launch<FFN_DH>(g, st); break;
    case FFN_DX: launch<FFN_DX>(g, st); break;
    case FFN_DW: launch<FFN_DW>(g, st); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // namespace moelora
