// Products of a few rows with 4-bit weights and group scales, and the gated
// feed-forward block on such weights.  Contracts: include/moe_lora.h.
//
//   y[m][n] = sum over groups g of  s[n][g] * sum_{k in g} x[m][k] (q[n][k] - z[n][g])
//
// The weights meet the matrix cores as integers, so nothing of them is
// rounded: a nibble q put into the low mantissa bits of bf16 128 is exactly
// 128 + q (one AND-OR for two weights), 128 + z is exact in bf16 as well, and
// the MFMAs sum x (128 + q) and -x (128 + z) into the same fp32 accumulator,
// once per 32-deep step each.  A group's sum, sum x (q - z), is then scaled
// and added to the row's.  The two sums cancel: each has terms of up to 143
// |x| where the result's have 4.6 on the mean.  For x of mixed signs that is 30
// times the result's size and fp32 keeps 19 bits of it; x of one sign makes it
// about 170 times over a step, and 16 bits.  In all the result is off by at
// most (K + 8) 2^-24 sum |x| s (256 + q + z).
//
// Measured: one row, 5120 x 25600 and back (gate and up 135 MB, down 68): 25
// and 20 us, 5.2 TB/s where tiles are many (1600 pairs), 3.4 where 320 tiles
// meet 256 CUs.  32 rows, 4096 x 11008: 22 us gate and up (49 MB), 13 down,
// 4 for each join of the slabs: there decoding bounds it, 16 bits of every
// weight by VALU for each 16 x 32 x 16 step of the matrix cores, and a join
// is as long as a launch.
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
// 2i + 1 at bits 16 + 4i).  Then the scales [tile][chunk][16][groups of a
// chunk] bf16 and, where the matrix has them, the zero points in the same
// order, uint8: a lane has a chunk's in one load.  Rows past N and groups
// past the last have scale 0, weights past K meet zeros of x.
__global__ __launch_bounds__(256) void w4_pack_kernel(W4Layout L, const uint8_t* __restrict__ q,
                                                      const uint16_t* __restrict__ scales,
                                                      const uint8_t* __restrict__ zeros, char* __restrict__ packed) {
  const int64_t words = (int64_t)L.tiles * L.chunks * 256;
  const int gpc = 128 / L.group;
  const int64_t groups = (int64_t)L.tiles * L.chunks * 16 * gpc;
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
    const int64_t tc = i / (16 * gpc);  // tile, chunk
    const int64_t g = tc % L.chunks * gpc + i % gpc, n = tc / L.chunks * 16 + i / gpc % 16;
    const bool ok = n < L.N && g < L.G;
    s[i] = ok ? scales[n * L.G + g] : (uint16_t)0;
    if (L.has_zeros) {
      const uint8_t v = ok ? zeros[n * L.G + g] : (uint8_t)0;
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
  static constexpr int LINES = 8;
  static constexpr int MAX_FRAGMENTS = 4;
  // 4 starts later and gains nothing; 1 is up to 9 % faster in some products
  // and 9 to 15 % slower in others.  us with 1, 2 and 4,
  // N x K, one row: 11008 x 4096 7.5, 8.2, 9.0; 4096 x 11008 8.7, 8.0, 9.0;
  // 25600 x 5120 21, 18, 18; 5120 x 25600 17.7, 18.6, 20.3; 32 rows: 4096 x
  // 11008 16.6, 17.0, 18.1; 25600 x 5120 30, 30, 31.  The block, 2 and 4: one
  // row, H 5120, I 25600 47.5 and 51; 32 rows, 4096, 11008 43 and 45.  (The
  // shared form takes turns in two buffers of rows, so that a gated product
  // needs 2.)
  static constexpr int DEPTH = 2;
  struct Tile {  // chunk 0 of the tile's weights, scales and zero points
    const char* q;
    const char* s;
    const char* z;
  };
  struct Buf {
    u32x4_t q;
    uint32_t s[2], z;  // the words with the chunk's scales and zero points of this lane's row
  };
  const Args& a;
  int lane;
  uint32_t mask = 0x000f000fu, magic = 0x43004300u;
  __device__ __forceinline__ PackedWeights(const Args& a_, int, int, int lane_) : a(a_), lane(lane_) {
    // in registers, so that AND and OR are one instruction
    asm("" : "+s"(mask));
    asm("" : "+v"(magic));
  }
  // tiles past the last repeat it, their sums are dropped
  __device__ __forceinline__ Tile tile(int t, int half) const {
    const int64_t i = (int64_t)min(t, a.L.tiles - 1) * a.L.chunks;
    const char* w = a.w[half];
    return Tile{w + i * 1024, w + a.L.off_scales + i * (32 * GPC), w + a.L.off_zeros + i * (16 * GPC)};
  }
  __device__ __forceinline__ void load(Buf& b, const Tile& t, int c, bool real) const {
    const uint32_t n = real ? (uint32_t)a.L.chunks : 0u;
    const buf_rsrc_t q = make_rsrc(t.q, n * 1024u);
    b.q = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(q, lane * 16, c * 1024, 2));
    // whole words, of which a lane picks its part when it uses them
    const buf_rsrc_t s = make_rsrc(t.s, n * (32u * GPC));
    const int row = lane & 15, sc = c * (32 * GPC);
    if (GPC == 4) {
      const uint2 v = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(s, row * 8, sc, 0));
      b.s[0] = v.x;
      b.s[1] = v.y;
    } else {
      b.s[0] = __builtin_amdgcn_raw_buffer_load_b32(s, (row * GPC >> 1) * 4, sc, 0);
    }
    if (ZEROS) b.z = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(t.z, n * (16u * GPC)), (row * GPC >> 2) * 4,
                                                          c * (16 * GPC), 0);
  }
  __device__ __forceinline__ float scale(const Buf& b, int g) const {
    uint32_t v = b.s[GPC == 4 ? g >> 1 : 0];
    if (GPC == 1) v <<= lane & 1 ? 0 : 16;
    return (GPC == 1 || g & 1) ? bf16_hi(v) : bf16_lo(v);
  }
  // -(128 + z) as bf16, twice
  __device__ __forceinline__ uint32_t zero(const Buf& b, int g) const {
    if (!ZEROS) return 0xc308c308u;
    const int shift = 8 * ((lane * GPC & 3) + g);
    const uint32_t z = (b.z >> shift) & 255u;
    return 0xc300c300u + z * 0x00010001u;
  }
  // the weights of step j as bf16 128 + q
  __device__ __forceinline__ u32x4_t operand(const Buf& b, int j) const {
    u32x4_t v;
#pragma unroll
    for (int h = 0; h < 4; ++h) v[h] = ((b.q[j] >> (4 * h)) & mask) | magic;
    return v;
  }

  template <int RF, int CT>
  struct Acc {
    f32x4_t tot[RF][CT], a[RF][CT];
    u32x4_t z[CT];
    __device__ __forceinline__ void clear() {
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int t = 0; t < CT; ++t) tot[f][t] = a[f][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    // before step j: the zero points of its group
    __device__ __forceinline__ void begin(const PackedWeights& w, const Buf* b, int j) {
      if (j % SPG) return;
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        const uint32_t v = w.zero(b[t], j / SPG);
        z[t] = u32x4_t{v, v, v, v};
      }
    }
    // the zero points' share of a step
    __device__ __forceinline__ void rows(int f, u32x4_t x) {
#pragma unroll
      for (int t = 0; t < CT; ++t) a[f][t] = mfma_16x16x32(x, z[t], a[f][t]);
    }
    __device__ __forceinline__ void mul(int f, int t, u32x4_t x, u32x4_t w) { a[f][t] = mfma_16x16x32(x, w, a[f][t]); }
    // after step j: a group's sum is scaled where it ends
    __device__ __forceinline__ void end(const PackedWeights& w, const Buf* b, int j) {
      if ((j + 1) % SPG) return;
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        const float s = w.scale(b[t], j / SPG);
#pragma unroll
        for (int f = 0; f < RF; ++f) {
#pragma unroll
          for (int v = 0; v < 4; ++v) tot[f][t][v] += s * a[f][t][v];
          a[f][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
      }
    }
    __device__ __forceinline__ f32x4_t sum(int f, int t) const { return tot[f][t]; }
  };
};

int check_matrix(const moe_lora_w4* w, W4Layout* L) {
  if (!w || w->N <= 0 || w->K <= 0) return MOE_LORA_EINVAL;
  if (w->group != 32 && w->group != 64 && w->group != 128) return MOE_LORA_EINVAL;
  if (w->has_zeros != 0 && w->has_zeros != 1) return MOE_LORA_EINVAL;
  if (w->K % 8) return MOE_LORA_EALIGN;
  if (w->N > (1 << 22) || w->K > (1 << 22)) return MOE_LORA_EUNSUPPORTED;
  L->N = w->N;
  L->K = w->K;
  L->group = w->group;
  L->has_zeros = w->has_zeros;
  L->tiles = (w->N + 15) / 16;
  L->chunks = (w->K + 127) / 128;
  L->G = (w->K + w->group - 1) / w->group;
  L->off_scales = (size_t)L->tiles * L->chunks * 1024;
  const size_t groups = (size_t)L->tiles * L->chunks * 16 * (128 / w->group);
  L->off_zeros = L->off_scales + round256(groups * 2);
  L->total = L->off_zeros + (w->has_zeros ? round256(groups) : 0);
  return MOE_LORA_OK;
}

// up: the second matrix of a gated product, or NULL
void launch_product(const RowsArgs& a, const W4Layout& L, const void* w, const void* up, hipStream_t st) {
  auto go = [&](auto spg, auto zeros) {
    typedef PackedWeights<decltype(spg)::value, decltype(zeros)::value> W;
    typename W::Args wa;
    wa.w[0] = (const char*)w;
    wa.w[1] = (const char*)up;
    wa.L = L;
    if (up) launch_rows<W, true, false>(a, wa, st);
    else if (a.x_lo) launch_rows<W, false, true>(a, wa, st);
    else launch_rows<W, false, false>(a, wa, st);
  };
  auto with = [&](auto spg) {
    if (L.has_zeros) go(spg, std::true_type());
    else go(spg, std::false_type());
  };
  if (L.group == 32) with(std::integral_constant<int, 1>());
  else if (L.group == 64) with(std::integral_constant<int, 2>());
  else with(std::integral_constant<int, 4>());
}

size_t slab_bytes(const W4Layout& L, int M) { return rows_slab_bytes(rows_plan(M, L.N, L.K, 8), M, L.N, false); }

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

size_t moe_lora_w4_workspace_bytes(const moe_lora_w4* w, int32_t M) {
  W4Layout L;
  if (check_matrix(w, &L) || M < 0 || M > kMaxRows) return 0;
  // 256 says that nothing is needed, so slabs of a few bytes count as more
  const size_t n = M ? slab_bytes(L, M) : 0;
  return n ? std::max<size_t>(round256(n), 512) : 256;
}

int moe_lora_w4_matmul(const moe_lora_w4* w, int32_t M, const uint16_t* x, void* workspace, size_t ws_bytes,
                       uint16_t* y, void* stream) {
  W4Layout L;
  const int rc = check_matrix(w, &L);
  if (rc) return rc;
  if (M < 0) return MOE_LORA_EINVAL;
  if (M > kMaxRows) return MOE_LORA_EUNSUPPORTED;
  if (M == 0) return MOE_LORA_OK;
  if (!x || !y || !w->data) return MOE_LORA_EINVAL;
  const size_t need = slab_bytes(L, M);
  if (need && (!workspace || ws_bytes < need)) return MOE_LORA_EWORKSPACE;
  if (!aligned16(x) || (uintptr_t)y % 2 || !aligned16(w->data) || (need && !aligned16(workspace)))
    return MOE_LORA_EALIGN;
  const Range in[] = {{x, (size_t)M * L.K * 2}, {w->data, L.total}};
  const Range out[] = {{y, (size_t)M * L.N * 2}, {workspace, need}};
  if (any_overlap(in, 2, out, 2)) return MOE_LORA_EINVAL;
  launch_product(RowsArgs{x, nullptr, y, nullptr, nullptr, M, L.N, L.K, 0, (float*)workspace, 1, 0}, L, w->data, nullptr, (hipStream_t)stream);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

// h (and its remainder), then the slabs of either product
static size_t ffn_h_bytes(int32_t M, int32_t I) { return round256((size_t)M * I * 2) * (M <= kPairRows ? 2 : 1); }

size_t moe_lora_w4_ffn_workspace_bytes(int32_t M, int32_t I) {
  if (M < 0 || I <= 0 || M > kMaxRows || I > (1 << 22)) return 0;
  return M ? ffn_h_bytes(M, I) + rows_slab_bound(M) : 256;
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
  float* slabs = (float*)((char*)workspace + ffn_h_bytes(M, Ld.K));
  launch_product(RowsArgs{x, nullptr, h, h_lo, nullptr, M, Lg.N, Lg.K, act, slabs, 1, 0}, Lg, gate->data, up->data, st);
  launch_product(RowsArgs{h, h_lo, y, nullptr, nullptr, M, Ld.N, Ld.K, 0, slabs, 1, 0}, Ld, down->data, nullptr, st);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // extern "C"
