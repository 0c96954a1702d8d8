// The adapters' gradients: dA_l = sum u[t] x[t]^T, dB_l = s_l sum dy[t] z[t]^T.
//
// Both are a few columns (u's or z's, 3r of them as parts) against all columns
// of x or dy, summed over the rows of one adapter: the wide side is read once
// and bounds the product.  A workgroup takes 128 of its columns and one piece
// of a run, 64 rows a stage, gathered on their way into LDS; both sides have
// their output index contiguous and are transposed on the way to registers
// (ds_read_b64_tr_b16).  An adapter without tokens is an empty piece.  A run of
// several pieces puts fp32 sums into slabs, which a second kernel adds in their
// order.  What is left of a value behind its first part may be 0 or of the other
// sign, so an infinity or NaN of x or dy meets the first part alone, whose
// product with it is the value's; the others meet 0 there.  8192
// tokens, 4096 x 4096, rank 16: 30 us (156 MB at 5.3 TB/s) and 5 for the slabs;
// 1001 tokens, 2880 x 2880, rank 32: 9.6 us.
#include "internal.h"
#include "proj.h"
#include "tile.h"

namespace moelora {

namespace {

constexpr int WT = 128;               // wide columns of a workgroup
constexpr int NW = 4, NT = 64 * NW;
constexpr int kMostRows = 1024;       // of a piece

struct GradArgs {
  ProjArgs p;
  ProjGrads g;
  int tiles_a;          // workgroups along x's columns (0: no dA)
  int slabs;            // at most
};

// PW: columns of a narrow row's part, 16 or a multiple of 32.
template <int PW>
struct Grad {
  // Blocks of 32 narrow columns.  The values rounded have blocks of their own,
  // half of one with PW = 16, where the other two parts share the next.
  static constexpr int NB = PW == 16 ? 2 : 3 * PW / 32, FIRST = PW == 16 ? 1 : PW / 32;
  static constexpr int ROWB = NB * 64;                      // bytes of a narrow LDS row
  static constexpr int WIDE = BK * WT * 2, STAGE = WIDE + BK * ROWB;
  static constexpr int RING = NB <= 2 ? 3 : 2;              // (two workgroups on a CU up to PW = 32)
  static constexpr int NC = WIDE / 1024 / NW + NB;          // copies of a wavefront and stage
  static constexpr int LDS = RING * STAGE + kMostRows * 4;
  // 64-byte parts of a narrow row are swizzled so that the four rows that a
  // transposing read takes side by side lie in different banks
  static __device__ __forceinline__ int swizzle(int k) {
    return ROWB % 256 == 0 ? 64 * (k & 3) : ROWB % 128 == 0 ? 64 * ((k >> 1) & 1) : 0;
  }
  // of an LDS row's column: its part, and which of the part's; a part's first
  static __device__ __forceinline__ int part_of(int col) { return PW == 16 ? (col + 16) / 32 : col / PW; }
  static constexpr int first(int part) { return PW == 16 ? part * 16 + (part > 0) * 16 : part * PW; }
};

__device__ __forceinline__ u32x4_t transposed(const char* p, int four_rows) {
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + four_rows));
  const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
  return u32x4_t{a.x, a.y, b.x, b.y};
}

template <int PW>
__global__ __launch_bounds__(NT, PW <= 32 ? 2 : 1) void proj_grads_kernel(GradArgs a) {
  typedef Grad<PW> C;
  constexpr int NB = C::NB;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  int* token = reinterpret_cast<int*>(smem + C::RING * C::STAGE);
  const ProjArgs& p = a.p;
  if ((int)blockIdx.y >= p.o.count[1]) return;
  const ProjItem item = p.o.grad[blockIdx.y];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool is_a = (int)blockIdx.x < a.tiles_a;
  const int w0 = ((int)blockIdx.x - (is_a ? 0 : a.tiles_a)) * WT;
  const int width = is_a ? p.K : p.N, r = p.r;
  const u32x4_t rw = rsrc_of(is_a ? a.g.x : a.g.dy, 0x7fffffffu);
  const u32x4_t rn = rsrc_of(is_a ? a.g.us : a.g.zs, 0x7fffffffu);
  for (int i = threadIdx.x; i < item.n; i += NT) token[i] = p.o.perm[item.row + i];
  lds_barrier();

  const uint32_t smem_at = (uint32_t)(uintptr_t)(lds_char*)smem;
  const int stages = (item.n + BK - 1) / BK;
  auto bring = [&](int s, int slot) __attribute__((always_inline)) {
    const uint32_t to = smem_at + slot * C::STAGE;
    for_each<C::NC - NB>([&](auto i_c) __attribute__((always_inline)) {
      constexpr int i = decltype(i_c)::value;
      const int k = (wave * (C::NC - NB) + i) * 4 + (lane >> 4), ch = (lane & 15) ^ (4 * (k & 3));
      const int m = s * BK + k;
      const uint32_t off = m < item.n && w0 + ch * 8 < width
                               ? ((uint32_t)token[m] * (uint32_t)width + w0 + ch * 8u) * 2u : kBufNone;
      copy16<i * 1024>(rw, to + wave * ((C::NC - NB) * 1024), off, 0);
    });
    for_each<NB>([&](auto i_c) __attribute__((always_inline)) {
      constexpr int i = decltype(i_c)::value;
      const int at = (wave * NB + i) * 1024 + lane * 16, k = at / C::ROWB;
      const int col = ((at % C::ROWB) ^ C::swizzle(k)) / 2;       // of the LDS row
      const int part = C::part_of(col), j = col - C::first(part), m = s * BK + k;
      const uint32_t off = m < item.n && j >= 0 && j < r
                               ? ((uint32_t)((item.row + m) * kParts + part) * (uint32_t)r + j) * 2u : kBufNone;
      copy16<i * 1024>(rn, to + C::WIDE + wave * (NB * 1024), off, 0);
    });
  };

  f32x16_t acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[b][v] = 0.f;
  const int g = lane >> 4, sub = (lane >> 2) & 3;
  constexpr int AHEAD = C::RING - 1;
#pragma unroll
  for (int s = 0; s < AHEAD; ++s) bring(s, s);
  int slot = 0;
  for (int s = 0; s < stages; ++s) {
    // this stage's copies have landed (with three slots the next one's may
    // still be on their way), and everybody is done with the slot before it
    if constexpr (AHEAD == 2) __builtin_amdgcn_s_waitcnt((C::NC & 15) | ((C::NC >> 4) << 14) | (7 << 4) | (15 << 8));
    else __builtin_amdgcn_s_waitcnt(wait_vm0);
    bare_barrier();
    const int to = slot + AHEAD >= C::RING ? slot + AHEAD - C::RING : slot + AHEAD;
    bring(s + AHEAD, to);
    const char* at = smem + slot * C::STAGE;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const u32x4_t wide = Operand<false, WT, 1, false>::frag(at, wave * 32, 0, kk);
      u32x4_t finite = wide;
      if (__ballot(not_finite_bits(wide) & 0x80008000u)) finite = only_finite(wide);
      const int k = kk * 16 + 8 * (g >> 1) + sub;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int col = ((b * 32 + (g & 1) * 16) * 2 + (lane & 3) * 8) ^ C::swizzle(k);
        acc[b] = mfma_32x32x16(transposed(at + C::WIDE + k * C::ROWB + col, 4 * C::ROWB), b < C::FIRST ? wide : finite,
                              acc[b]);
      }
    }
    __builtin_amdgcn_s_waitcnt(wait_lgkm0);
    slot = slot + 1 == C::RING ? 0 : slot + 1;
  }
  __builtin_amdgcn_s_waitcnt(wait_vm0);  // no copy outlives the workgroup

  // element 4 q + i of the blocks: narrow column 8 q + 4 (l / 32) + i, wide
  // column l % 32; of a value its three parts' sums
  const int c = w0 + wave * 32 + (lane & 31), kh = lane >> 5;
  if (c >= width) return;
#pragma unroll
  for (int q = 0; q < PW / 8; ++q) {
    const int j = 8 * q + 4 * kh;
    if (8 * q >= r) break;
    constexpr int MID = C::first(1) / 8, LOW = C::first(2) / 8;
    f32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = acc[q / 4][q % 4 * 4 + i] +
             (acc[(q + MID) / 4][(q + MID) % 4 * 4 + i] + acc[(q + LOW) / 4][(q + LOW) % 4 * 4 + i]);
    if (item.slab >= 0) {
      if (is_a) {
        float* to = a.g.slabs + ((int64_t)item.slab * r + j) * width + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) to[(int64_t)i * width] = v[i];
      } else {
        float* to = a.g.slabs + (a.tiles_a ? (int64_t)a.slabs * r * p.K : 0) + ((int64_t)item.slab * width + c) * r + j;
        *reinterpret_cast<f32x4_t*>(to) = v;
      }
    } else if (is_a) {
      uint16_t* to = a.g.dA + ((int64_t)item.adapter * r + j) * width + c;
#pragma unroll
      for (int i = 0; i < 4; ++i) to[(int64_t)i * width] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
    } else {
      uint16_t* to = a.g.dB + ((int64_t)item.adapter * width + c) * r + j;
      *reinterpret_cast<uint2*>(to) = uint2{f32x2_to_bf16(v[0], v[1]), f32x2_to_bf16(v[2], v[3])};
    }
  }
}

// Gradients of adapters in several pieces: their slabs, added in order.
__global__ __launch_bounds__(256) void proj_grads_join_kernel(GradArgs a) {
  const ProjArgs& p = a.p;
  const int l = blockIdx.y, first = p.o.slabs[2 * l], n = p.o.slabs[2 * l + 1];
  if (n == 0) return;  // written already
  const int64_t in_a = a.g.dA ? (int64_t)p.r * p.K : 0, in_b = a.g.dB ? (int64_t)p.r * p.N : 0;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < in_a + in_b; i += (int64_t)gridDim.x * 2048) {
    const bool is_a = i < in_a;
    const int64_t size = is_a ? in_a : in_b, at = is_a ? i : i - in_a;
    const float* src = a.g.slabs + (is_a ? 0 : a.slabs * in_a) + first * size + at;
    float v[8];
    for (int z = 0; z < n; ++z) {
      const f32x4_t* s = reinterpret_cast<const f32x4_t*>(src + z * size);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = z ? v[q] + s[q >> 2][q & 3] : s[q >> 2][q & 3];
    }
    store8((is_a ? a.g.dA : a.g.dB) + l * size + at, v);
  }
}

template <int PW>
int launch_cfg(const GradArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> attr_done;
  const void* fn = reinterpret_cast<const void*>(&proj_grads_kernel<PW>);
  const int rc = ensure_dynamic_lds(fn, Grad<PW>::LDS, attr_done);
  if (rc) return rc;
  const int tiles = a.tiles_a + (a.g.dB ? (a.p.N + WT - 1) / WT : 0);
  const dim3 grid(tiles, (unsigned)proj_grad_items(a.p));
  proj_grads_kernel<PW><<<grid, NT, Grad<PW>::LDS, st>>>(a);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

int slabs_of(int T, int rows) { return 2 * (T / rows); }

}  // namespace

// Enough pieces to fill the chip with four rounds of workgroups, but at least 8r
// rows each (a slab of r columns costs as much as 4r rows to write and read
// again).  Few tokens beside a stack of more than four adapters are not split at
// all, which spares the join where the batch has several of them.  L counts those
// of the stack: how many are met is known on the device alone.  A backward for dA
// and dB, us, unsplit and split, 16 adapters of rank 32, 2880 x 2880, 1001 tokens
// of 16, 5, 2 and 1 of them: 24.3 and 25.9, 23.4 and 25.1, 26.5 and 27.0, 33.1 and
// 28.1; 500 tokens of 16, 5 and 1: 23.8 and 25.3, 21.5 and 23.3, 26.2 and 26.3.
int proj_grad_rows(int T, int K, int N, int L, int r) {
  if (T <= kMostRows && L > 4) return kMostRows;
  const int64_t rows = (int64_t)T * ((K + N) / WT + 1) / 1024;
  return (int)std::min<int64_t>(kMostRows, std::max<int64_t>((rows + BK - 1) / BK * BK, std::max(256, 8 * r)));
}

size_t proj_grad_slab_bytes(const ProjArgs& p) {
  return (size_t)slabs_of(p.T, p.grad_rows) * p.r * ((size_t)p.K + p.N) * sizeof(float);
}

int launch_proj_grads(const ProjArgs& p, const ProjGrads& g, hipStream_t st) {
  const GradArgs a{p, g, g.dA ? (p.K + WT - 1) / WT : 0, slabs_of(p.T, p.grad_rows)};
  const int rc = p.r <= 16 ? launch_cfg<16>(a, st) : p.r <= 32 ? launch_cfg<32>(a, st)
                 : p.r <= 64 ? launch_cfg<64>(a, st) : launch_cfg<128>(a, st);
  if (rc || p.T <= p.grad_rows) return rc;  // no run has several pieces
  const int64_t pieces = ((int64_t)(g.dA ? p.K : 0) + (g.dB ? p.N : 0)) * p.r / 8;
  const dim3 grid((unsigned)std::min<int64_t>(64, (pieces + 255) / 256), p.L);
  proj_grads_join_kernel<<<grid, 256, 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // namespace moelora
