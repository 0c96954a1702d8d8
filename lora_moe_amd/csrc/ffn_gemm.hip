// Products of the gated feed-forward block: LDS-tiled bf16 MFMA.
//
//   C[m][n] = sum_k A(m, k) B(n, k), fp32 sums, gate and its gradient in the
// epilogue.  An operand lies either with k contiguous (x, h, dy, the weights
// of a forward) or with its output index contiguous (the weights of dh and
// dx, both sides of a weight gradient): the transposes that a backward pass
// needs are never written out, they happen on the way from LDS to registers
// (ds_read_b64_tr_b16).
#include <algorithm>
#include <type_traits>

#include "device_util.h"
#include "ffn.h"
#include "internal.h"
#include "gate_act.h"

namespace moelora {

namespace {

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

__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f32x2_to_bf16(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<u32x4_t*>(p) = o;
}

// 8 values as sums of two bf16
__device__ __forceinline__ void store8_pair(uint16_t* hi, uint16_t* lo, const float* v) {
  u32x4_t a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t h[2], l[2];
    f32_to_bf16_pair(v[2 * i], h, l);
    f32_to_bf16_pair(v[2 * i + 1], h + 1, l + 1);
    a[i] = h[0] | (uint32_t)h[1] << 16;
    b[i] = l[0] | (uint32_t)l[1] << 16;
  }
  *reinterpret_cast<u32x4_t*>(hi) = a;
  *reinterpret_cast<u32x4_t*>(lo) = b;
}

// g and u of 8 neighbouring outputs, as the forward kept them
__device__ __forceinline__ void load_kept(const FfnGemm& p, int m, int n, f32x4_t* g, f32x4_t* u) {
  const f32x4_t* src = reinterpret_cast<const f32x4_t*>(p.gu + (int64_t)m * 2 * p.N + n);
  g[0] = src[0];
  g[1] = src[1];
  u[0] = src[p.N / 4];
  u[1] = src[p.N / 4 + 1];
}

// What becomes of 8 neighbouring sums a (gate_up: gate sums a and up sums u;
// dh: kept g and u in kg and ku).
template <int PRODUCT>
__device__ __forceinline__ void finish(const FfnGemm& p, int m, int n, const f32x4_t* a, const f32x4_t* u,
                                       const f32x4_t* kg, const f32x4_t* ku) {
  float v[8], w[8], h[8];
  if (PRODUCT == FFN_GATE_UP) {
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = gate_act<false>(p.act, a[q >> 2][q & 3], nullptr) * u[q >> 2][q & 3];
    store8(p.out + (int64_t)m * p.N + n, h);
    if (p.gu) {
      f32x4_t* dst = reinterpret_cast<f32x4_t*>(p.gu + (int64_t)m * 2 * p.N + n);
      __builtin_nontemporal_store(a[0], dst);
      __builtin_nontemporal_store(a[1], dst + 1);
      __builtin_nontemporal_store(u[0], dst + p.N / 4);
      __builtin_nontemporal_store(u[1], dst + p.N / 4 + 1);
    }
  } else if (PRODUCT == FFN_DH) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float g = kg[q >> 2][q & 3], k = ku[q >> 2][q & 3], dh = a[q >> 2][q & 3];
      float da;
      const float act = gate_act<true>(p.act, g, &da);
      h[q] = act * k;
      v[q] = dh * k * da;
      w[q] = dh * act;
    }
    uint16_t* dg = p.out + (int64_t)m * 2 * p.N + n;
    uint16_t* ho = p.out2 + (int64_t)m * p.N + n;
    if (p.pair) {
      const int64_t lo = (int64_t)p.M * p.N;
      store8_pair(dg, dg + 2 * lo, v);
      store8_pair(dg + p.N, dg + 2 * lo + p.N, w);
      store8_pair(ho, ho + lo, h);
    } else {
      store8(dg, v);
      store8(dg + p.N, w);
      store8(ho, h);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = a[q >> 2][q & 3];
    store8(p.out + (int64_t)m * p.N + n, v);
  }
}

// SPLIT: this split's sums go to the slabs.  ONE: K is one stage, and the ring
// that single stage, so that twice as many workgroups share a CU: a weight
// gradient of few tokens is bound by its own stores and by how many tiles'
// first copies are in flight (22016 x 4096 of 64 tokens: 48 us so, 79
// without).
//
// Workgroup `block` of the product's ncol x nrow tiles (times its splits).
template <int PRODUCT, class C, bool SPLIT, bool ONE>
__device__ __forceinline__ void ffn_tile(const FfnGemm& p, int ncol, int nrow, int block) {
  constexpr bool A_KC = PRODUCT != FFN_DW;
  constexpr bool B_KC = PRODUCT == FFN_GATE_UP || PRODUCT == FFN_DOWN;
  constexpr bool GATE = PRODUCT == FFN_GATE_UP;
  constexpr int MI = C::MI, NI = C::NI;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;

  // Workgroup i runs on XCD i % 8: each XCD takes a contiguous eighth of the
  // tiles (of each K split in turn), in panels of 4 row tiles, column by
  // column, so that the 32 tiles that an XCD works on at a time share 4 row
  // and 8 column panels in its L2.
  int t;
  {
    const int total = ncol * nrow * (SPLIT ? p.splits : 1), x = block & 7, j = block >> 3;
    const int per = total >> 3, rest = total & 7;
    t = x * per + min(x, rest) + j;
  }
  const int split = SPLIT ? t / (ncol * nrow) : 0;
  t -= split * (ncol * nrow);
  constexpr int GM = 4;
  const int panel = t / (GM * ncol), in = t - panel * GM * ncol;
  const int gm = min(GM, nrow - panel * GM);
  const int tn = in / gm, tm = panel * GM + in - tn * gm;
  const int m0 = tm * C::BM, n0 = tn * (GATE ? C::BN / 2 : C::BN);

  const int rows = PRODUCT == FFN_DX && p.pair ? 2 * p.M : p.M;  // of A
  Operand<A_KC, C::BM, C::NCA, false> A;
  Operand<B_KC, C::BN, C::NCB, GATE> B;
  const int all = (p.K + BK - 1) / BK, kfirst = p.K - all * BK;
  // this split's stages
  const int s0 = SPLIT ? (int)((int64_t)all * split / p.splits) : 0;
  const int nst = SPLIT ? (int)((int64_t)all * (split + 1) / p.splits) : all;
  A.init(A_KC ? p.A + (int64_t)m0 * p.lda : p.A + m0, 0, p.lda, rows - m0, kfirst, wave, PRODUCT == FFN_DW ? p.wrap_a : 0);
  B.init(B_KC ? p.B + (int64_t)n0 * p.ldb : p.B + n0, (int64_t)p.N * p.ldb, p.ldb, p.N - n0, kfirst, wave,
         PRODUCT == FFN_DW ? p.wrap_b : 0);

  f32x16_t acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  const uint32_t smem_at = (uint32_t)(uintptr_t)(lds_char*)smem;
  u32x4_t af[2][MI], bf[2][NI];
  auto read = [&](int slot, int kk, int set, int i) __attribute__((always_inline)) {  // fragment i of a slice
    const char* at = smem + slot * C::STAGE;
    // the first MFMAs' first: one of A, all of B, the rest of A
    if (i == 0) af[set][0] = A.frag(at, wm * (C::BM / C::WM), 0, kk);
    else if (i <= NI) bf[set][i - 1] = B.frag(at + C::ABYTES, wn * (C::BN / C::WN), i - 1, kk);
    else af[set][i - NI] = A.frag(at, wm * (C::BM / C::WM), i - NI, kk);
  };
  constexpr int NM = MI * NI, NF = MI + NI, NC = C::NCA + C::NCB;
  // MFMA n of a slice; the next slice's fragment reads go out between the
  // first ones, so that they have landed when the slice ends, and after the
  // stage's barrier the copies of the stage after next, one or two at a time
  auto slice = [&](int set, int slot, int kk, auto issue_c) __attribute__((always_inline)) {
    constexpr bool ISSUE = decltype(issue_c)::value;
    for_each<NM>([&](auto n_c) __attribute__((always_inline)) {
      constexpr int n = decltype(n_c)::value, i = n / NI, j = n % NI;
      // B first: a lane ends with runs of 4 neighbouring columns of one row
      acc[i][j] = mfma_32x32x16(bf[set][j], af[set][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (n < NF) read(slot, kk, set ^ 1, n);
      if constexpr (ISSUE) {
        for_each<(n + 1) * NC / NM - n * NC / NM>([&](auto q_c) __attribute__((always_inline)) {
          constexpr int q = n * NC / NM + decltype(q_c)::value;
          const uint32_t to = smem_at + (slot ^ 1) * C::STAGE;
          if constexpr (q < C::NCA) A.template copy<q, false>(to, wave, 0);
          else B.template copy<q - C::NCA, false>(to + C::ABYTES, wave, 0);
        });
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  typedef std::integral_constant<bool, true> yes;
  typedef std::integral_constant<bool, false> no;
  // Every stage runs the same code: the copies behind the last stage bring
  // zeros without touching memory, and the last reads take what is never
  // used (or, where the number of stages is odd, zeros).
  A.at(s0, s0 < nst);
  B.at(s0, s0 < nst);
  if (s0 == 0) {
    for_each<C::NCA>([&](auto i) { A.template copy<decltype(i)::value, true>(smem_at, wave, kfirst); });
    for_each<C::NCB>([&](auto i) { B.template copy<decltype(i)::value, true>(smem_at + C::ABYTES, wave, kfirst); });
  } else {
    for_each<C::NCA>([&](auto i) { A.template copy<decltype(i)::value, false>(smem_at, wave, 0); });
    for_each<C::NCB>([&](auto i) { B.template copy<decltype(i)::value, false>(smem_at + C::ABYTES, wave, 0); });
  }
  if constexpr (!ONE) {
    A.at(s0 + 1, s0 + 1 < nst);
    B.at(s0 + 1, s0 + 1 < nst);
    for_each<C::NCA>([&](auto i) { A.template copy<decltype(i)::value, false>(smem_at + C::STAGE, wave, 0); });
    for_each<C::NCB>(
        [&](auto i) { B.template copy<decltype(i)::value, false>(smem_at + C::STAGE + C::ABYTES, wave, 0); });
  }
  __builtin_amdgcn_s_waitcnt(wait_vm0);
  bare_barrier();
#pragma unroll
  for (int i = 0; i < NF; ++i) read(0, 0, 0, i);
  if constexpr (ONE) {
    slice(0, 0, 1, no());
    slice(1, 0, 2, no());
    slice(0, 0, 3, no());
    slice(1, 0, 0, no());
  } else {
    for (int s = s0; s < nst; s += 2) {
      for_each<2>([&](auto h_c) __attribute__((always_inline)) {
        constexpr int slot = decltype(h_c)::value;
        slice(0, slot, 1, no());
        slice(1, slot, 2, no());
        A.at(s + slot + 2, s + slot + 2 < nst);
        B.at(s + slot + 2, s + slot + 2 < nst);
        slice(0, slot, 3, no());
        // own copies of the next stage have landed, own reads of this one are done
        __builtin_amdgcn_s_waitcnt(wait_vm0 & wait_lgkm0);
        bare_barrier();
        slice(1, slot ^ 1, 0, yes());
      });
    }
  }
  __builtin_amdgcn_s_waitcnt(wait_vm0);  // no copy outlives the workgroup

  // Epilogue, 32 rows of the wavefront at a time through its own part of the
  // LDS (the ring is done with: every wavefront is past the last stage's
  // barrier and reads, see above), so that memory sees whole lines: a lane
  // takes 8 neighbouring outputs of one row, a row's lanes lie side by side.
  // Straight from the accumulators a row's 16-byte pieces went to memory one
  // by one: dh with its gate at T = 8192, H = 4096, I = 11008 took 1550 us
  // that way and 1200 with this (four wavefronts, both).
  constexpr int WC = C::BN / C::WN;          // the wavefront's tile columns
  constexpr int ROWF = WC + 4;               // floats of a staged row (padded by 16 bytes against bank conflicts)
  constexpr int OUT = GATE ? WC / 2 : WC;    // its outputs per row
  constexpr int LPR = OUT / 8, RPI = 64 / LPR;  // lanes per row, rows per step
  float* mine = reinterpret_cast<float*>(smem) + wave * 32 * ROWF;
  static_assert(C::NW * 32 * ROWF * 4 <= (ONE ? C::LDS_ONE : C::LDS), "staged rows must fit the ring");
  bare_barrier();
  const int l32 = lane & 31, kh = lane >> 5;
  const int oc = (lane % LPR) * 8;           // first of this lane's outputs in the wavefront's columns
  const int n = n0 + wn * OUT + oc;
  // A runtime loop over the row blocks: all unrolled, the gate's code came to
  // 70 KB, more than the instruction cache.  What dh reads of the forward is a
  // step ahead (dh at T = 8192, H = 4096, I = 11008: 873 us with a block's loads
  // at its start, 805 so).
  constexpr int STEPS = 32 / RPI;
  const int mb = m0 + wm * (C::BM / C::WM) + lane / LPR, rows_here = SPLIT ? rows : p.M;
  constexpr bool KEPT = PRODUCT == FFN_DH && !SPLIT;
  f32x4_t kg[2], ku[2], ng[2], nu[2];
  if (KEPT && mb < p.M && n < p.N) load_kept(p, mb, n, ng, nu);
  auto one = [&](int i, int r) __attribute__((always_inline)) {
    const int step = i * STEPS + r;
    const int m = mb + i * 32 + r * RPI;
    if (KEPT) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        kg[h] = ng[h];
        ku[h] = nu[h];
      }
      const int next = mb + (step + 1) / STEPS * 32 + (step + 1) % STEPS * RPI;
      if (step + 1 < MI * STEPS && next < p.M && n < p.N) load_kept(p, next, n, ng, nu);
    }
    if (m < rows_here && n < p.N) {
      const float* row = mine + (r * RPI + lane / LPR) * ROWF;
      // gate_up: 32-column blocks alternate, gate, up
      const f32x4_t* src = reinterpret_cast<const f32x4_t*>(row + (GATE ? (oc >> 5) * 64 + (oc & 31) : oc));
      const f32x4_t a[2] = {src[0], src[1]}, u[2] = {src[GATE ? 8 : 0], src[GATE ? 9 : 1]};
      if constexpr (SPLIT) {
        constexpr int W = GATE ? 2 : 1;
        f32x4_t* dst = reinterpret_cast<f32x4_t*>(p.slabs + ((int64_t)split * rows + m) * (W * p.N) + n);
        dst[0] = a[0];
        dst[1] = a[1];
        if (GATE) {
          dst[p.N / 4] = u[0];
          dst[p.N / 4 + 1] = u[1];
        }
      } else {
        finish<PRODUCT>(p, m, n, a, u, kg, ku);
      }
    }
  };
#pragma unroll 1
  for (int i = 0; i < MI; ++i) {
    // element v of a 32 x 32 block: row l % 32, column 8 (v / 4) + 4 (l / 32) + v % 4
    for_each<MI>([&](auto b_c) __attribute__((always_inline)) {
      constexpr int b = decltype(b_c)::value;
      if (i != b) return;
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4_t*>(mine + l32 * ROWF + j * 32 + 8 * q + 4 * kh) =
              f32x4_t{acc[b][j][4 * q], acc[b][j][4 * q + 1], acc[b][j][4 * q + 2], acc[b][j][4 * q + 3]};
    });
    asm volatile("" ::: "memory");  // a wavefront's LDS accesses run in order
#pragma unroll
    for (int r = 0; r < STEPS; ++r) one(i, r);
    asm volatile("" ::: "memory");
  }
}

template <int PRODUCT, class C, bool SPLIT, bool ONE>
__global__ __launch_bounds__(C::NT, ONE ? 4 : 2) void ffn_gemm_kernel(FfnGemm p, int ncol, int nrow) {
  ffn_tile<PRODUCT, C, SPLIT, ONE>(p, ncol, nrow, blockIdx.x);
}

// The three products of a backward that follow dh, none of which needs
// another, as one grid: dx, whose tiles take longest, then the weight
// gradients, so that no product ends in a round of its own (backward of 1001
// tokens, H = I = 2880: 130 us so, 174 as three grids; 4096 x 11008: 150 tokens
// 225 and 238, 2048 tokens 999 and 1140, 8192 tokens 3723 and 3759).
struct FfnGrads {
  FfnGemm g[3];  // dx, dW_gu, dW_down
  int ncol[3], nrow[3];
  int first[3];  // workgroup
};

template <class C, bool SPLIT>
__global__ __launch_bounds__(C::NT, 2) void ffn_grads_kernel(FfnGrads p) {
  const int block = blockIdx.x;
  if (block < p.first[1]) {
    ffn_tile<FFN_DX, C, SPLIT, false>(p.g[0], p.ncol[0], p.nrow[0], block);
  } else {
    const int i = block < p.first[2] ? 1 : 2;
    ffn_tile<FFN_DW, C, false, false>(p.g[i], p.ncol[i], p.nrow[i], block - p.first[i]);
  }
}

// Adds the slabs in their order and finishes 8 neighbouring outputs.  DX of a
// pair: a row's remainder is row M + m of the slabs.
template <int PRODUCT>
__global__ __launch_bounds__(256) void ffn_join_kernel(FfnGemm p) {
  constexpr int W = PRODUCT == FFN_GATE_UP ? 2 : 1;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = p.N / 8;
  if (i >= per * p.M) return;
  const int m = (int)(i / per), n = (int)(i % per) * 8;
  const int halves = PRODUCT == FFN_DX && p.pair ? 2 : 1;
  f32x4_t kg[2], ku[2];
  if (PRODUCT == FFN_DH) load_kept(p, m, n, kg, ku);
  f32x4_t s[W][2];
  for (int z = 0; z < p.splits * halves; ++z)
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const f32x4_t* src =
          reinterpret_cast<const f32x4_t*>(p.slabs + ((int64_t)z * p.M + m) * (W * p.N) + w * p.N + n);
#pragma unroll
      for (int h = 0; h < 2; ++h) s[w][h] = z ? s[w][h] + src[h] : src[h];
    }
  finish<PRODUCT>(p, m, n, s[0], s[W - 1], kg, ku);
}

template <int PRODUCT>
void launch_join(const FfnGemm& g, hipStream_t st) {
  const int64_t n = (int64_t)g.M * (g.N / 8);
  ffn_join_kernel<PRODUCT><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(g);
}

template <int PRODUCT, class C, bool SPLIT, bool ONE = false>
int launch_cfg(const FfnGemm& g, hipStream_t st) {
  static std::atomic<uint64_t> attr_done;
  constexpr int bn = PRODUCT == FFN_GATE_UP ? C::BN / 2 : C::BN;
  constexpr int lds = ONE ? C::LDS_ONE : C::LDS;
  const int rows = PRODUCT == FFN_DX && g.pair ? 2 * g.M : g.M;
  const int64_t ncol = (g.N + bn - 1) / bn, nrow = (rows + C::BM - 1) / C::BM, grid = ncol * nrow * g.splits;
  if (grid * C::NT > 0xffffffff) return MOE_LORA_EUNSUPPORTED;
  const void* fn = reinterpret_cast<const void*>(&ffn_gemm_kernel<PRODUCT, C, SPLIT, ONE>);
  const int rc = ensure_dynamic_lds(fn, lds, attr_done);
  if (rc) return rc;
  ffn_gemm_kernel<PRODUCT, C, SPLIT, ONE><<<(unsigned)grid, C::NT, lds, st>>>(g, (int)ncol, (int)nrow);
  if (SPLIT) launch_join<PRODUCT>(g, st);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

// 256 x 256 tiles on 8 wavefronts of 128 x 64, one workgroup per CU (128 KB
// of LDS).  T = 8192, H = 4096, I = 11008 (0.74 TFLOP, the gate_up pair 1.48,
// the gradients that follow dh 3.69), us: down 586, gate_up with its kept gu
// 1445, dh with its gate 843, the gradients 2951, i.e. 1.25 PFLOP/s where the
// epilogue is only a store.  What bounds them is power: at 75 % of the MFMA
// slots the clock is 1.5 to 1.85 GHz of 2.4, and a copy of the loop that waits
// less reached 87 % at 1.59 GHz and the same time within 4 %.  Four wavefronts
// of 128 x 128 read less LDS but stall the only wavefront of a SIMD while it
// issues its copies (dx 1250 us against 1177, alternating runs).
typedef FfnCfg<256, 256, 2, 4> Big;
// 128 x 128 tiles on 4 wavefronts, two workgroups per CU, where there are too
// few large ones to fill the chip.
typedef FfnCfg<128, 128, 2, 2> Small;

// Tile, and K splits of the small one, by the time that they would take: full
// rounds of workgroups (256 large ones, or 512 small ones, two to a CU) and
// their stages; a last round of small ones with a CU each is shorter; splits
// cost a launch and the slabs' way to memory and back.  The constants (us)
// are fitted to 2189 times of 386 products of 65 to 8192 tokens, H 1024 to
// 5120, I 2816 to 25600: the choice is 1.6 % above the best one on the mean, and
// furthest off, by 47 %, for dh of 256 tokens at H 1024, I 2816.
struct FfnPlan {
  bool big;
  int splits;
  double us;
};

FfnPlan plan(int M, int N, int K, FfnProduct product) {
  const int64_t stages = std::max(1, (K + BK - 1) / BK), cols = (int64_t)N * (product == FFN_GATE_UP ? 2 : 1);
  FfnPlan best{true, 1, 0.};
  int64_t tiles = (int64_t)((M + 255) / 256) * ((cols + 255) / 256);
  double least = (double)((tiles + 255) / 256) * (stages * 1.19 + 4.0);
  tiles = (int64_t)((M + 127) / 128) * ((cols + 127) / 128);
  for (int64_t s = 1; s <= 16 && s * 3 <= std::max<int64_t>(3, stages); ++s) {
    if (s > 1 && (tiles > 512 || tiles * s > 2048)) break;  // less than a round to begin with
    const int64_t each = (stages + s - 1) / s, full = tiles * s / 512, rest = tiles * s % 512;
    const double round_us = each * 0.81 + 0.8;
    double us = (full + (rest > 256)) * round_us + (rest > 0 && rest <= 256 ? each * 0.57 : 0.);
    if (s > 1) us += 3.5 + s * (double)M * cols * 8 * 0.16e-6;
    if (us < least) {
      least = us;
      best = FfnPlan{false, (int)s};
    }
  }
  best.us = least;
  return best;
}

int64_t tiles_of(int M, int N, int tile) { return (int64_t)((M + tile - 1) / tile) * ((N + tile - 1) / tile); }

// Up to BK tokens: one grid up to this many tiles of the weight gradients,
// beyond it their one-stage form in grids of their own gains more than the
// launches cost.  33 tokens, one grid and three, us: 256 x 512 (24 tiles) 18
// and 25, 1024 x 2816 (528) 30 and 35, 2880 x 2880 (1564) 46 and 49, 2880 x
// 5760 (3105) 65 and 63, 4096 x 11008 (8256) 174 and 153.
constexpr int64_t kGradsFew = 2048;

// The same for the three products as one grid: all stages share the chip, and
// on the mean half a weight gradient's tile is what the last workgroups wait
// for.  us = 0: three grids.
FfnPlan grads_plan(int T, int H, int I) {
  FfnPlan best{false, 1, 0.};
  if (T <= BK) {
    const bool pair = T <= kRowsPair;
    const int64_t s = plan(pair ? 2 * T : T, H, 2 * I, FFN_DX).splits;
    if (tiles_of(2 * I, H, 128) + tiles_of(H, I, 128) <= kGradsFew) best = FfnPlan{false, (int)s, 1.};
    return best;
  }
  double least = plan(T, H, 2 * I, FFN_DX).us + plan(2 * I, H, T, FFN_DW).us + plan(H, I, T, FFN_DW).us;
  const int sx = (2 * I + BK - 1) / BK, sw = (T + BK - 1) / BK;
  auto take = [&](bool big, int s, double us) {
    if (us < least) best = FfnPlan{big, s, us}, least = us;
  };
  {
    const int64_t x = tiles_of(T, H, 256), w = tiles_of(2 * I, H, 256) + tiles_of(H, I, 256);
    const double all = (x * (sx * 1.19 + 4.) + w * (sw * 1.19 + 4.)) / 256, last = sw * 1.19 + 4.;
    take(true, 1, std::max(all + last / 2, sx * 1.19 + 4.));
  }
  const int64_t x = tiles_of(T, H, 128), w = tiles_of(2 * I, H, 128) + tiles_of(H, I, 128);
  for (int s = 1; s <= 16 && s * 3 <= std::max(3, sx); ++s) {
    if (s > 1 && x * s > 2048) break;
    const int each = (sx + s - 1) / s;
    const double all = (x * s * (each * 0.81 + 0.8) + w * (sw * 0.81 + 0.8)) / 512, last = sw * 0.81 + 0.8;
    take(false, s, std::max(all + last / 2, each * 0.81 + 0.8) + (s > 1 ? 3.5 + s * (double)T * H * 8 * 0.16e-6 : 0.));
  }
  return best;
}

template <class C, bool SPLIT>
int launch_grads_cfg(FfnGrads g, hipStream_t st) {
  static std::atomic<uint64_t> attr_done;
  int64_t n = 0;
  for (int i = 0; i < 3; ++i) {
    g.ncol[i] = (g.g[i].N + C::BN - 1) / C::BN;
    g.nrow[i] = ((i == 0 && g.g[0].pair ? 2 : 1) * g.g[i].M + C::BM - 1) / C::BM;
    g.first[i] = (int)n;
    n += (int64_t)g.ncol[i] * g.nrow[i] * g.g[i].splits;
    if (n * C::NT > 0xffffffff) return MOE_LORA_EUNSUPPORTED;
  }
  const int rc = ensure_dynamic_lds(reinterpret_cast<const void*>(&ffn_grads_kernel<C, SPLIT>), C::LDS, attr_done);
  if (rc) return rc;
  ffn_grads_kernel<C, SPLIT><<<(unsigned)n, C::NT, C::LDS, st>>>(g);
  if (SPLIT) launch_join<FFN_DX>(g.g[0], st);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

template <int PRODUCT>
int launch(FfnGemm g, hipStream_t st) {
  g.splits = 1;
  if constexpr (PRODUCT == FFN_DW)
    if (g.K <= BK) return launch_cfg<PRODUCT, Small, false, true>(g, st);
  const bool pair = PRODUCT == FFN_DX && g.pair;
  const FfnPlan f = plan(pair ? 2 * g.M : g.M, g.N, g.K, (FfnProduct)PRODUCT);
  g.splits = f.splits;
  if (pair || f.splits > 1) return launch_cfg<PRODUCT, Small, true>(g, st);
  return f.big ? launch_cfg<PRODUCT, Big, false>(g, st) : launch_cfg<PRODUCT, Small, false>(g, st);
}

}  // namespace

size_t ffn_gemm_slab_bytes(int M, int N, int K, FfnProduct product, bool pair) {
  const int s = plan(pair ? 2 * M : M, N, K, product).splits;
  return s > 1 || pair ? (size_t)s * M * N * (product == FFN_GATE_UP || pair ? 2 : 1) * sizeof(float) : 0;
}

size_t ffn_grads_slab_bytes(int T, int H, int I) {
  const FfnPlan f = grads_plan(T, H, I);
  const bool pair = T <= kRowsPair;
  return f.us > 0. && (f.splits > 1 || pair) ? (size_t)f.splits * (pair ? 2 : 1) * T * H * sizeof(float) : 0;
}

int launch_ffn_grads(const FfnGemm& dx, const FfnGemm& dw_gu, const FfnGemm& dw_down, hipStream_t st) {
  const FfnPlan f = grads_plan(dx.M, dx.N, dx.K / 2);
  if (f.us > 0.) {
    FfnGrads g = {{dx, dw_gu, dw_down}, {}, {}, {}};
    g.g[0].splits = f.splits;
    g.g[1].splits = g.g[2].splits = 1;
    if (f.splits > 1 || dx.pair) return launch_grads_cfg<Small, true>(g, st);
    return f.big ? launch_grads_cfg<Big, false>(g, st) : launch_grads_cfg<Small, false>(g, st);
  }
  int r = launch_ffn_gemm(dx, FFN_DX, st);
  if (!r) r = launch_ffn_gemm(dw_gu, FFN_DW, st);
  return r ? r : launch_ffn_gemm(dw_down, FFN_DW, st);
}

int launch_ffn_gemm(const FfnGemm& g, FfnProduct product, hipStream_t st) {
  if (g.M == 0 || g.N == 0) return MOE_LORA_OK;
  switch (product) {
    case FFN_GATE_UP: return launch<FFN_GATE_UP>(g, st);
    case FFN_DOWN: return launch<FFN_DOWN>(g, st);
    case FFN_DH: return launch<FFN_DH>(g, st);
    case FFN_DX: return launch<FFN_DX>(g, st);
    case FFN_DW: return launch<FFN_DW>(g, st);
  }
  return MOE_LORA_EINVAL;
}

}  // namespace moelora
