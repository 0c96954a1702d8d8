// Products of a few rows with 4-bit weights and group scales, and the gated
// feed-forward block on such weights.  Contracts: include/moe_lora.h.
//
//   y[m][n] = sum over groups g of  s[n][g] * sum_{k in g} x[m][k] (q[n][k] - z[n][g])
//
// The weights meet the matrix cores as integers, so nothing of them is
// rounded: a nibble q put into the low mantissa bits of bf16 128 is exactly
// 128 + q (one AND and one OR for two weights), the MFMAs sum x (128 + q)
// per group in fp32, a further MFMA against ones gives the group's sum of x
// per row, and
//   y += s * (sum x (128 + q) - (128 + z) * sum x)
// once per group.  The cancelled part is at most ~30 times the result's size
// (136 against a spread of 4.6), so fp32 keeps 18 bits and more of it.
#include "abi_util.h"
#include "device_util.h"
#include "gate_act.h"
#include "w4.h"

namespace moelora {

namespace {

// Packed layout of an [N][K] matrix: tiles of 16 rows; per tile ceil(K / 128)
// chunks of 1 KB, 16 bytes for each lane of a wavefront: lane l holds row
// l % 16, and in word j the weights k = 128c + 32j + 8 (l / 16) + 0..7, even
// ones in the low half (k 2i at bits 4i) and odd ones in the high half (k
// 2i + 1 at bits 16 + 4i).  Then the scales [tile][group][16] bf16 and the
// zero points [tile][group][16] uint8 where the matrix has them.  Rows past N
// have scale 0, weights past K meet zeros of x.
__global__ __launch_bounds__(256) void w4_pack_kernel(W4Layout L, const uint8_t* __restrict__ q,
                                                      const uint16_t* __restrict__ scales,
                                                      const uint8_t* __restrict__ zeros, char* __restrict__ packed) {
  const int64_t words = (int64_t)L.tiles * L.chunks * 256;
  const int64_t groups = (int64_t)L.tiles * L.G * 16;
  const int64_t step = (int64_t)gridDim.x * 256;
  uint32_t* w = reinterpret_cast<uint32_t*>(packed);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += step) {
    const int j = (int)(i & 3), lane = (int)(i >> 2) & 63;
    const int64_t c = (i >> 8) % L.chunks, t = (i >> 8) / L.chunks;
    const int64_t n = t * 16 + (lane & 15), k = c * 128 + j * 32 + (lane >> 4) * 8;
    uint32_t v = 0;
    if (n < L.N && k < L.K) {
      const uint8_t* src = q + n * (L.K / 2) + k / 2;
#pragma unroll
      for (int b = 0; b < 4; ++b) v |= (uint32_t)(src[b] & 15u) << (4 * b) | (uint32_t)(src[b] >> 4) << (16 + 4 * b);
    }
    w[i] = v;
  }
  uint16_t* s = reinterpret_cast<uint16_t*>(packed + L.off_scales);
  uint8_t* z = reinterpret_cast<uint8_t*>(packed + L.off_zeros);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < groups; i += step) {
    const int64_t g = (i >> 4) % L.G, n = (i >> 4) / L.G * 16 + (i & 15);
    s[i] = n < L.N ? scales[n * L.G + g] : (uint16_t)0;
    if (L.has_zeros) {
      const uint8_t v = n < L.N ? zeros[n * L.G + g] : (uint8_t)0;
      z[i] = v < 15 ? v : (uint8_t)15;
    }
  }
}

struct W4Args {
  const uint16_t* x;  // [M][K]
  const char* w[2];   // packed; w[1]: the up weights (gated)
  W4Layout L;
  uint16_t* out;      // [M][N]
  int M, act;
};

// One workgroup: 16 rows x 16 columns; its four wavefronts take every fourth
// chunk of K and add up through LDS.
template <bool GATED>
__global__ __launch_bounds__(256) void w4_kernel(W4Args p) {
  constexpr int NW = 4, NP = GATED ? 2 : 1;
  __shared__ f32x4_t part[NW][NP][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, kq = lane >> 4;
  const int tile = blockIdx.x, m0 = blockIdx.y * 16;
  const W4Layout& L = p.L;
  const int mr = min(m0 + l16, p.M - 1);  // rows past M repeat the last one; their results are dropped
  const uint16_t* xr = p.x + (int64_t)mr * L.K;
  const u32x4_t ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
  f32x4_t tot[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) tot[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int spg = L.group / 32;  // MFMA steps per group
  for (int c = wave; c < L.chunks; c += NW) {
    u32x4_t q[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i)
      q[i] = ld16_stream(p.w[i] + ((int64_t)tile * L.chunks + c) * 1024 + lane * 16);
    f32x4_t acc[NP], xs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NP; ++i) acc[i] = xs;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = c * 128 + j * 32 + kq * 8;
      const u32x4_t a = k < L.K ? ld16(xr + k) : zero4();
      xs = mfma_16x16x32(a, ones, xs);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        u32x4_t b;
#pragma unroll
        for (int h = 0; h < 4; ++h) b[h] = ((q[i][j] >> (4 * h)) & 0x000f000fu) | 0x43004300u;
        acc[i] = mfma_16x16x32(a, b, acc[i]);
      }
      if ((j + 1) % spg == 0) {  // the group ends (the last one of K may be short: the rest met zeros)
        const int g = min((c * 128 + j * 32) / L.group, L.G - 1);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int64_t at = ((int64_t)tile * L.G + g) * 16 + l16;
          const float s = bf16_to_f32(reinterpret_cast<const uint16_t*>(p.w[i] + L.off_scales)[at]);
          const float z =
              128.f + (L.has_zeros ? (float)reinterpret_cast<const uint8_t*>(p.w[i] + L.off_zeros)[at] : 8.f);
#pragma unroll
          for (int v = 0; v < 4; ++v) tot[i][v] += s * (acc[i][v] - z * xs[v]);
          acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        xs = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) part[wave][i][lane] = tot[i];
  __syncthreads();
  if (wave) return;
  const int n = tile * 16 + l16;
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int w = 1; w < NW; ++w) tot[i] += part[w][i][lane];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int m = m0 + kq * 4 + v;
    if (m < p.M && n < L.N) {
      const float o = GATED ? gate_act<false>(p.act, tot[0][v], nullptr) * tot[NP - 1][v] : tot[0][v];
      p.out[(int64_t)m * L.N + n] = f32_to_bf16(o);
    }
  }
}

int check_matrix(const moe_lora_w4* w, W4Layout* L) {
  if (!w || w->N <= 0 || w->K <= 0) return MOE_LORA_EINVAL;
  if (w->group != 32 && w->group != 64 && w->group != 128) return MOE_LORA_EINVAL;
  if (w->has_zeros != 0 && w->has_zeros != 1) return MOE_LORA_EINVAL;
  if (w->K % 8) return MOE_LORA_EALIGN;
  if (w->N > (1 << 24) || w->K > (1 << 24)) return MOE_LORA_EUNSUPPORTED;
  L->N = w->N;
  L->K = w->K;
  L->group = w->group;
  L->has_zeros = w->has_zeros;
  L->tiles = (w->N + 15) / 16;
  L->chunks = (w->K + 127) / 128;
  L->G = (w->K + w->group - 1) / w->group;
  L->off_scales = (size_t)L->tiles * L->chunks * 1024;
  L->off_zeros = L->off_scales + round256((size_t)L->tiles * L->G * 32);
  L->total = L->off_zeros + (w->has_zeros ? round256((size_t)L->tiles * L->G * 16) : 0);
  return MOE_LORA_OK;
}

void launch_product(const W4Args& a, bool gated, hipStream_t st) {
  const dim3 grid(a.L.tiles, (a.M + 15) / 16);
  if (gated) w4_kernel<true><<<grid, 256, 0, st>>>(a);
  else w4_kernel<false><<<grid, 256, 0, st>>>(a);
}

constexpr int32_t kMaxRows = 1 << 16;

}  // namespace

}  // namespace moelora

using namespace moelora;

extern "C" {

size_t moe_lora_w4_bytes(const moe_lora_w4* w) {
  W4Layout L;
  return check_matrix(w, &L) ? 0 : L.total;
}

int moe_lora_w4_pack(const moe_lora_w4* w, const uint8_t* q, const uint16_t* scales, const uint8_t* zeros,
                     void* packed, size_t packed_bytes, void* stream) {
  W4Layout L;
  const int rc = check_matrix(w, &L);
  if (rc) return rc;
  if (!q || !scales || !packed || (zeros != nullptr) != (L.has_zeros != 0)) return MOE_LORA_EINVAL;
  if (packed_bytes < L.total) return MOE_LORA_EWORKSPACE;
  if (!aligned16(packed) || (uintptr_t)scales % 2) return MOE_LORA_EALIGN;
  const size_t ng = (size_t)L.N * L.G;
  const Range in[] = {{q, (size_t)L.N * (L.K / 2)}, {scales, 2 * ng}, {zeros, zeros ? ng : 0}};
  const Range out[] = {{packed, L.total}};
  if (any_overlap(in, 3, out, 1)) return MOE_LORA_EINVAL;
  w4_pack_kernel<<<2048, 256, 0, (hipStream_t)stream>>>(L, q, scales, zeros, (char*)packed);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

int moe_lora_w4_matmul(const moe_lora_w4* w, int32_t M, const uint16_t* x, uint16_t* y, void* stream) {
  W4Args a = {};
  const int rc = check_matrix(w, &a.L);
  if (rc) return rc;
  if (M < 0) return MOE_LORA_EINVAL;
  if (M > kMaxRows) return MOE_LORA_EUNSUPPORTED;
  if (M == 0) return MOE_LORA_OK;
  if (!x || !y || !w->data) return MOE_LORA_EINVAL;
  if (!aligned16(x) || (uintptr_t)y % 2 || !aligned16(w->data)) return MOE_LORA_EALIGN;
  const Range in[] = {{x, (size_t)M * a.L.K * 2}, {w->data, a.L.total}};
  const Range out[] = {{y, (size_t)M * a.L.N * 2}};
  if (any_overlap(in, 2, out, 1)) return MOE_LORA_EINVAL;
  a.x = x;
  a.w[0] = (const char*)w->data;
  a.out = y;
  a.M = M;
  launch_product(a, false, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

size_t moe_lora_w4_ffn_workspace_bytes(int32_t M, int32_t I) {
  if (M < 0 || I <= 0 || M > kMaxRows) return 0;
  const size_t n = round256((size_t)M * I * 2);
  return n ? n : 256;
}

int moe_lora_w4_ffn_forward(const moe_lora_w4* gate, const moe_lora_w4* up, const moe_lora_w4* down, int32_t M,
                            int32_t act, const uint16_t* x, void* workspace, size_t ws_bytes, uint16_t* y,
                            void* stream) {
  W4Args a = {};
  W4Layout Lu, Ld;
  int rc;
  if ((rc = check_matrix(gate, &a.L)) || (rc = check_matrix(up, &Lu)) || (rc = check_matrix(down, &Ld))) return rc;
  // the two halves of gate_up walk together
  if (Lu.N != a.L.N || Lu.K != a.L.K || Lu.group != a.L.group || Lu.has_zeros != a.L.has_zeros ||
      Ld.N != a.L.K || Ld.K != a.L.N || M < 0)
    return MOE_LORA_EINVAL;
  if (act != MOE_LORA_ACT_SILU && act != MOE_LORA_ACT_GELU) return MOE_LORA_EINVAL;
  if (M > kMaxRows) return MOE_LORA_EUNSUPPORTED;
  if (M == 0) return MOE_LORA_OK;
  if (!x || !y || !gate->data || !up->data || !down->data) return MOE_LORA_EINVAL;
  const size_t h_bytes = (size_t)M * Ld.K * 2;
  if (!workspace || ws_bytes < h_bytes) return MOE_LORA_EWORKSPACE;
  if (!aligned16(x) || (uintptr_t)y % 2 || !aligned16(workspace) || !aligned16(gate->data) || !aligned16(up->data) ||
      !aligned16(down->data))
    return MOE_LORA_EALIGN;
  const Range in[] = {
      {x, (size_t)M * a.L.K * 2}, {gate->data, a.L.total}, {up->data, Lu.total}, {down->data, Ld.total}};
  const Range out[] = {{y, (size_t)M * Ld.N * 2}, {workspace, h_bytes}};
  if (any_overlap(in, 4, out, 2)) return MOE_LORA_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  a.x = x;
  a.w[0] = (const char*)gate->data;
  a.w[1] = (const char*)up->data;
  a.out = (uint16_t*)workspace;
  a.M = M;
  a.act = act;
  launch_product(a, true, st);
  a.x = (const uint16_t*)workspace;
  a.w[0] = (const char*)down->data;
  a.w[1] = nullptr;
  a.L = Ld;
  a.out = y;
  launch_product(a, false, st);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // extern "C"
