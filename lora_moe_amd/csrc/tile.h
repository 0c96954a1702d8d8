// Pieces of the LDS-tiled bf16 MFMA products (ffn_gemm.hip, proj_gemm.hip):
// asynchronous copies into LDS, an operand's side of a stage, waits.
#pragma once

#include <algorithm>
#include <type_traits>

#include "device_util.h"

namespace moelora {

typedef __attribute__((address_space(3))) char lds_char;
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

constexpr int BK = 64;  // K depth of a stage

// 16 bytes per lane from the resource's base + soff + voff (zeros where voff
// is past the resource's end) to LDS byte lds + IMM + 16 * lane.  In assembly,
// without a register that a load in flight could write: through the builtin
// the compiler takes every later LDS read for a read of this copy's target
// and waits for the copy first.  Callers wait themselves.  Resource, offset
// and m0 come from scalar arithmetic, which needs no wait states before a
// vector memory operation, and one between m0 and a copy into LDS.  m0 is
// named as overwritten; that the compiler never keeps values of its own in it
// (a "reserved" register, says its warning) is what lets the block set it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int IMM>
__device__ __forceinline__ void copy16(u32x4_t rsrc, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff), "n"(IMM)
               : "memory", "scc", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ u32x4_t rsrc_of(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)base;
  return u32x4_t{(uint32_t)b, (uint32_t)(b >> 32), bytes, 0x00020000u};
}

template <int BM_, int BN_, int WM_, int WN_>
struct FfnCfg {
  static constexpr int BM = BM_, BN = BN_;            // tile
  static constexpr int WM = WM_, WN = WN_;            // wavefronts along m and n
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int MI = BM / WM / 32, NI = BN / WN / 32;  // 32 x 32 blocks of a wavefront
  static constexpr int ABYTES = BM * BK * 2, BBYTES = BN * BK * 2, STAGE = ABYTES + BBYTES;
  static constexpr int LDS = 2 * STAGE;
  static constexpr int LDS_ONE = std::max(STAGE, NW * 32 * (BN / WN + 4) * 4);  // one stage, or the epilogue's rows
  static constexpr int NCA = ABYTES / 1024 / NW, NCB = BBYTES / 1024 / NW;  // 1 KB copies per wavefront and stage
};

// f(0), f(1), .. with compile-time indices
template <int N, int I = 0, class F>
__device__ __forceinline__ void for_each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    for_each<N, I + 1>(static_cast<F&&>(f));
  }
}

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// One operand's side of a stage: ROWS x 64 (rows: the output index).
//
// KC, k contiguous: LDS row r holds 64 k (128 bytes) of output row r, its 16
// byte pieces XOR-swizzled by (r / 2) % 8 so that the 32 rows of a fragment
// read meet every bank equally.
// Else: LDS row k holds ROWS outputs; its 64-byte quarters of every 256
// bytes are XOR-swizzled by k % 4, the four k rows that a transposing read
// takes side by side.
// The swizzle is applied to the global address (a copy fills LDS in order).
// Rows past the end get an offset past the buffer's and copy zeros.
//
// Stages count from the end of K: where K is no multiple of 64 the FIRST
// stage begins before k = 0, and its lanes that lie there copy zeros; the
// loop's copies are whole ones.
template <bool KC, int ROWS, int NC, bool SPLIT>
struct Operand {
  const uint16_t* base;  // KC: row 0 of the tile at stage 0's first k; else stage 0's first k row, column 0
  int64_t odd;           // SPLIT: elements from there to the rows of the odd 32-row blocks (gate_up's up rows)
  int64_t ld;
  uint32_t off[NC];
  u32x4_t rs, rs2;       // the stage's resources, set by at()
  uint32_t soff;

  // p: the tile's first output at k = 0; rows_left: outputs from there on;
  // kfirst: stage 0's first k, in (-64, 0]; wrap (else 0; one stage): k from
  // there on are rows 0.. again
  __device__ __forceinline__ void init(const uint16_t* p, int64_t odd_, int64_t ld_, int rows_left, int kfirst,
                                       int wave, int wrap) {
    base = p + kfirst * (KC ? (int64_t)1 : ld_);
    odd = odd_;
    ld = ld_;
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = wave * NC + i;
      if (KC) {
        const int r = c * 8 + (lane >> 3);
        const int ch = (lane & 7) ^ ((r >> 1) & 7);
        // SPLIT: blocks of 32 alternate between the two row sets
        const int mr = SPLIT ? (r >> 6) * 32 + (r & 31) : r;
        off[i] = mr < rows_left ? (uint32_t)(mr * (int)ld + ch * 8) * 2u : kBufNone;
      } else {
        constexpr int PER = 1024 / (ROWS * 2), LPR = ROWS / 8;  // k rows per copy, lanes per row
        const int k = c * PER + lane / LPR;
        const int ch = (lane % LPR) ^ (4 * (k & 3));
        const int r = wrap && k + kfirst >= wrap ? k - wrap : k;
        off[i] = ch * 8 < rows_left ? (uint32_t)(r * (int)ld + ch * 8) * 2u : kBufNone;
      }
    }
  }

  // makes stage s the one that copy() fills from; behind the last one (!real)
  // copies bring zeros
  __device__ __forceinline__ void at(int s, bool real) {
    const uint32_t bytes = real ? 0x7fffffffu : 0u;
    if (KC) {
      rs = rsrc_of(base, bytes);
      if (SPLIT) rs2 = rsrc_of(base + odd, bytes);
      soff = (uint32_t)s * (BK * 2);
    } else {
      rs = rsrc_of(base + (int64_t)s * BK * ld, bytes);
      soff = 0;
    }
  }

  // copy I of the stage into the operand's part of a stage at LDS byte lds;
  // FIRST: stage 0, whose k below 0 are zeros
  template <int I, bool FIRST>
  __device__ __forceinline__ void copy(uint32_t lds, int wave, int kfirst) const {
    uint32_t o = off[I];
    if (FIRST) {
      const int lane = lane_id(), c = wave * NC + I;
      int k;
      if (KC) k = ((lane & 7) ^ (((c * 8 + (lane >> 3)) >> 1) & 7)) * 8;
      else k = c * (1024 / (ROWS * 2)) + lane / (ROWS / 8);
      if (kfirst + k < 0) o = kBufNone;
    }
    constexpr bool WIDE = NC >= 8;  // the row set alternates within a wavefront's copies, else with the wavefront
    if (SPLIT && (WIDE ? ((I >> 2) & 1) : (wave & 1))) copy16<I * 1024>(rs2, lds + wave * (NC * 1024), o, soff);
    else copy16<I * 1024>(rs, lds + wave * (NC * 1024), o, soff);
  }

  // fragment of 32 outputs from w0 + 32 * blk on, K slice kk of the stage:
  // lane l holds output l % 32, k = 16 kk + 8 (l / 32) + 0..7
  static __device__ __forceinline__ u32x4_t frag(const char* lds, int w0, int blk, int kk) {
    const int lane = lane_id();
    if (KC) {
      const int r = lane & 31, ch = (2 * kk + (lane >> 5)) ^ ((r >> 1) & 7);
      return *reinterpret_cast<const u32x4_t*>(lds + (w0 + blk * 32 + r) * 128 + ch * 16);
    }
    const int g = lane >> 4, s = (lane >> 2) & 3;
    const int col = ((w0 + blk * 32 + (g & 1) * 16) * 2 + (lane & 3) * 8) ^ (64 * s);
    const char* p = lds + (kk * 16 + 8 * (g >> 1) + s) * (ROWS * 2) + col;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * ROWS * 2));
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return u32x4_t{a.x, a.y, b.x, b.y};
  }
};

constexpr int wait_vm0 = (7 << 4) | (15 << 8);
constexpr int wait_lgkm0 = 15 | (3 << 14) | (7 << 4);

__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Bits 15 and 31 of the result: whether one of the two bf16 of a word of v is an
// infinity or NaN (the exponent's ones carry into the sign's place).
__device__ __forceinline__ uint32_t not_finite_bits(u32x4_t v) {
  uint32_t b = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) b |= (v[i] & 0x7f807f80u) + 0x00800080u;
  return b;
}

// such values to 0
__device__ __forceinline__ u32x4_t only_finite(u32x4_t v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & 0x7f80u) == 0x7f80u) v[i] &= 0xffff0000u;
    if ((v[i] & 0x7f800000u) == 0x7f800000u) v[i] &= 0xffffu;
  }
  return v;
}

__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f32x2_to_bf16(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<u32x4_t*>(p) = o;
}

}  // namespace moelora
