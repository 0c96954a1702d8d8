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
#include <type_traits>

#include "abi_util.h"
#include "device_util.h"
#include "rows.h"
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

// The stream's policy for packed weights (rows.h): a chunk of a tile is one
// contiguous KB.  SPG: 32-deep steps per group.
template <int SPG, bool ZEROS>
struct PackedWeights {
  struct Args {
    const char* w[2];  // w[1]: the up weights (gate)
    W4Layout L;
  };
  static constexpr int GPC = 4 / SPG;  // groups of a chunk
  struct Tile {
    const char* q;      // this lane's piece of chunk 0
    const uint16_t* s;  // the scale and zero point of this lane's row, group 0
    const uint8_t* z;
  };
  struct Buf {
    u32x4_t q;
    uint16_t s[GPC];
    uint8_t z[GPC];
  };
  Args a;
  int lane;
  __device__ __forceinline__ PackedWeights(const Args& a_, const RowsArgs&, int lane_) : a(a_), lane(lane_) {}
  __device__ __forceinline__ Tile tile(int t, int half) const {
    const int64_t i = min(t, a.L.tiles - 1);
    const char* w = a.w[half];
    Tile r;
    r.q = w + i * a.L.chunks * 1024 + lane * 16;
    r.s = reinterpret_cast<const uint16_t*>(w + a.L.off_scales) + i * a.L.G * 16 + (lane & 15);
    r.z = reinterpret_cast<const uint8_t*>(w + a.L.off_zeros) + i * a.L.G * 16 + (lane & 15);
    return r;
  }
  __device__ __forceinline__ void load(Buf& b, const Tile& t, int c, bool masked) const {
    b.q = ld16_stream(t.q + (int64_t)c * 1024);
#pragma unroll
    for (int g = 0; g < GPC; ++g) {
      // a masked chunk's groups past the last one met zeros of x only
      const int at = masked ? min(c * GPC + g, a.L.G - 1) : c * GPC + g;
      b.s[g] = t.s[at * 16];
      if (ZEROS) b.z[g] = t.z[at * 16];
    }
  }
  // the weights of step j as bf16 128 + q
  __device__ __forceinline__ u32x4_t operand(const Buf& b, int j) const {
    u32x4_t v;
#pragma unroll
    for (int h = 0; h < 4; ++h) v[h] = ((b.q[j] >> (4 * h)) & 0x000f000fu) | 0x43004300u;
    return v;
  }

  template <int RF, int CT>
  struct Acc {
    f32x4_t tot[RF][CT], a[RF][CT], xs[RF];
    __device__ __forceinline__ void clear() {
      const f32x4_t z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        xs[f] = z;
#pragma unroll
        for (int t = 0; t < CT; ++t) tot[f][t] = a[f][t] = z;
      }
    }
    // the rows' sums, in every column
    __device__ __forceinline__ void rows(int f, const u32x4_t& x) {
      const u32x4_t ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
      xs[f] = mfma_16x16x32(x, ones, xs[f]);
    }
    __device__ __forceinline__ void mul(int f, int t, u32x4_t x, u32x4_t w) { a[f][t] = mfma_16x16x32(x, w, a[f][t]); }
    __device__ __forceinline__ void step(const PackedWeights&, const Tile*, const Buf* b, int, int j) {
      if ((j + 1) % SPG) return;
      const int g = j / SPG;
      const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        const float s = bf16_to_f32(b[t].s[g]);
        const float z = ZEROS ? 128.f + (float)b[t].z[g] : 136.f;
#pragma unroll
        for (int f = 0; f < RF; ++f) {
#pragma unroll
          for (int v = 0; v < 4; ++v) tot[f][t][v] += s * (a[f][t][v] - z * xs[f][v]);
          a[f][t] = zero;
        }
      }
#pragma unroll
      for (int f = 0; f < RF; ++f) xs[f] = zero;
    }
    __device__ __forceinline__ f32x4_t sum(int f, int t) const { return tot[f][t]; }
  };
};

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

template <class W>
void launch_format(const RowsArgs& a, const typename W::Args& wa, bool gated, hipStream_t st) {
  if (gated) {
    if (a.M <= 16) launch_rows_cfg<W, 1, 2, true, false>(a, wa, st);
    else if (a.M <= 32) launch_rows_cfg<W, 2, 2, true, false>(a, wa, st);
    else launch_rows_cfg<W, 4, 2, true, false>(a, wa, st);
  } else if (a.x_lo) {
    launch_rows_cfg<W, 1, 1, false, true>(a, wa, st);
  } else {
    if (a.M <= 16) launch_rows_cfg<W, 1, 1, false, false>(a, wa, st);
    else if (a.M <= 32) launch_rows_cfg<W, 2, 2, false, false>(a, wa, st);
    else launch_rows_cfg<W, 4, 2, false, false>(a, wa, st);
  }
}

// up: the second matrix of a gated product, or NULL
void launch_product(const RowsArgs& a, const W4Layout& L, const void* w, const void* up, hipStream_t st) {
  auto go = [&](auto spg, auto zeros) {
    typedef PackedWeights<decltype(spg)::value, decltype(zeros)::value> W;
    typename W::Args wa;
    wa.w[0] = (const char*)w;
    wa.w[1] = (const char*)up;
    wa.L = L;
    launch_format<W>(a, wa, up != nullptr, st);
  };
  auto with = [&](auto spg) {
    if (L.has_zeros) go(spg, std::true_type());
    else go(spg, std::false_type());
  };
  if (L.group == 32) with(std::integral_constant<int, 1>());
  else if (L.group == 64) with(std::integral_constant<int, 2>());
  else with(std::integral_constant<int, 4>());
}

constexpr int32_t kPairRows = 16;  // up to here h goes on as a bf16 pair, which costs nothing beside the weights
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
  W4Layout L;
  const int rc = check_matrix(w, &L);
  if (rc) return rc;
  if (M < 0) return MOE_LORA_EINVAL;
  if (M > kMaxRows) return MOE_LORA_EUNSUPPORTED;
  if (M == 0) return MOE_LORA_OK;
  if (!x || !y || !w->data) return MOE_LORA_EINVAL;
  if (!aligned16(x) || (uintptr_t)y % 2 || !aligned16(w->data)) return MOE_LORA_EALIGN;
  const Range in[] = {{x, (size_t)M * L.K * 2}, {w->data, L.total}};
  const Range out[] = {{y, (size_t)M * L.N * 2}};
  if (any_overlap(in, 2, out, 1)) return MOE_LORA_EINVAL;
  launch_product(RowsArgs{x, nullptr, y, nullptr, M, L.N, L.K, 0}, L, w->data, nullptr, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

size_t moe_lora_w4_ffn_workspace_bytes(int32_t M, int32_t I) {
  if (M < 0 || I <= 0 || M > kMaxRows) return 0;
  const size_t n = round256((size_t)M * I * 2) * (M <= kPairRows ? 2 : 1);
  return n ? n : 256;
}

int moe_lora_w4_ffn_forward(const moe_lora_w4* gate, const moe_lora_w4* up, const moe_lora_w4* down, int32_t M,
                            int32_t act, const uint16_t* x, void* workspace, size_t ws_bytes, uint16_t* y,
                            void* stream) {
  W4Layout Lg, Lu, Ld;
  int rc;
  if ((rc = check_matrix(gate, &Lg)) || (rc = check_matrix(up, &Lu)) || (rc = check_matrix(down, &Ld))) return rc;
  // the two halves of gate_up walk together
  if (Lu.N != Lg.N || Lu.K != Lg.K || Lu.group != Lg.group || Lu.has_zeros != Lg.has_zeros || Ld.N != Lg.K ||
      Ld.K != Lg.N || M < 0)
    return MOE_LORA_EINVAL;
  if (act != MOE_LORA_ACT_SILU && act != MOE_LORA_ACT_GELU) return MOE_LORA_EINVAL;
  if (M > kMaxRows) return MOE_LORA_EUNSUPPORTED;
  if (M == 0) return MOE_LORA_OK;
  if (!x || !y || !gate->data || !up->data || !down->data) return MOE_LORA_EINVAL;
  const size_t need = moe_lora_w4_ffn_workspace_bytes(M, Ld.K);
  if (!workspace || ws_bytes < need) return MOE_LORA_EWORKSPACE;
  if (!aligned16(x) || (uintptr_t)y % 2 || !aligned16(workspace) || !aligned16(gate->data) || !aligned16(up->data) ||
      !aligned16(down->data))
    return MOE_LORA_EALIGN;
  const Range in[] = {
      {x, (size_t)M * Lg.K * 2}, {gate->data, Lg.total}, {up->data, Lu.total}, {down->data, Ld.total}};
  const Range out[] = {{y, (size_t)M * Ld.N * 2}, {workspace, need}};
  if (any_overlap(in, 4, out, 2)) return MOE_LORA_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  uint16_t* h = (uint16_t*)workspace;
  uint16_t* h_lo = M <= kPairRows ? (uint16_t*)((char*)workspace + round256((size_t)M * Ld.K * 2)) : nullptr;
  launch_product(RowsArgs{x, nullptr, h, h_lo, M, Lg.N, Lg.K, act}, Lg, gate->data, up->data, st);
  launch_product(RowsArgs{h, h_lo, y, nullptr, M, Ld.N, Ld.K, 0}, Ld, down->data, nullptr, st);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // extern "C"
