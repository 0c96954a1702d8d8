// The projection's products: LDS-tiled bf16 MFMA.
//
//   forward   y[t]  = W x[t]    + B_l (s_l z[t])
//   backward  dx[t] = W^T dy[t] + A_l^T u[t]
//
// One product each, over the tokens sorted by adapter: a tile's K loop runs
// over the shared weights first, then over the ranks of the adapters whose
// rows the tile holds, 64 deep like the rest (a rank takes 3r: a value is the
// sum of three bf16).  A row takes part in its own adapter's share and is
// zeros in another's, so a tile of one long request has one share and a tile
// of a decode batch as many as it has adapters, while W is met once by all.
// The sorted order exists only in the addresses: rows of x (dy) are gathered
// on their way into LDS, rows of y (dx) scattered from the epilogue.
//
// Zeros times an infinity or NaN would carry one adapter's broken weights into
// another request's rows.  So the adapters' weights go into the products with
// 0 in place of such values, and so do the rows' own in that slice of K, and a
// tile that met one adds the terms of both to the rows that they belong to, one
// by one, in its epilogue.
//
// The loop is that of ffn_gemm.hip, with a ring of two to four slots: filled by
// asynchronous copies that go out between the MFMAs of the stage before.  The
// adapters' shares are further stages of the same loop, whose copies get their
// addresses when their turn comes.
//
// What bounds it: with large tiles the matrix cores at the clock that the
// card's power leaves them (8192 tokens, 4096 x 4096, rank 16: 219 us, 1.29
// PFLOP/s with the adapters' stages; 7168 x 7168, rank 64: 743 us, 1.17, of
// which 50 to 60 us are theirs where the flops would take 25: their first touch
// of B comes late from memory).  With a workgroup per CU the copies (0.34 us a
// stage of 32 KB, 100 GB/s to a CU), and up to 201 tokens a first trip through
// memory and the weights behind it.  (BOTH, a decode batch's x [W; A]^T without
// an order, is described in proj_few.hip.)
#include "ffn.h"
#include "internal.h"
#include "proj.h"
#include "tile.h"

namespace moelora {

namespace {

struct TileArgs {
  ProjArgs p;
  ProjGemm g;
  int in_cols, out_cols;  // K and N of a forward
  int ncol, nrow;
  int ncol_w, slots;      // BOTH: column tiles of W, then those of so many adapters
};

// A tile whose wavefronts share the stage's K slices too: KS groups of WM x WN
// wavefronts, each with 4 / KS of the four slices, whose sums meet in LDS at the
// end.  A wavefront's blocks are larger for it, and fewer bytes come out of LDS.
template <int BM, int BN, int WM, int WN, int KS>
struct SliceCfg : FfnCfg<BM, BN, WM, WN> {
  typedef FfnCfg<BM, BN, WM, WN> Base;
  static constexpr int NW = Base::NW * KS, NT = 64 * NW;
  static constexpr int NCA = Base::ABYTES / 1024 / NW, NCB = Base::BBYTES / 1024 / NW;
};

// RING: slots of the ring, of which all but one are filled ahead.
template <class C, int RING>
constexpr int tile_lds() { return RING * C::STAGE + (2 * C::BM + std::max(C::BM, 64)) * 4 + 16; }

// The terms of a row that only_finite took out, for 8 neighbouring outputs: those
// of which a factor is not finite.  Some may be in the sum already (a tile's
// wavefronts and K splits take out what they meet themselves); such a term is an
// infinity or NaN, and once more of it changes nothing.
// z: the row's parts; w: the adapter's weight of the first output and rank 0,
// `rank` apart along the rank and `out` along the outputs.
struct Eight {
  f32x4_t v[2];
};
__device__ __noinline__ Eight add_not_finite(Eight e, const uint16_t* z, const uint16_t* w, int64_t rank, int64_t out,
                                             int r) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float s = e.v[q >> 2][q & 3];
    for (int j = 0; j < r; ++j) {
      const uint16_t b = w[j * rank + q * out];
      if ((b & 0x7f80u) == 0x7f80u || (z[j] & 0x7f80u) == 0x7f80u)
        s += (bf16_to_f32(z[j]) + bf16_to_f32(z[r + j]) + bf16_to_f32(z[2 * r + j])) * bf16_to_f32(b);
    }
    e.v[q >> 2][q & 3] = s;
  }
  return e;
}

// BOTH (forward, SPLIT): x [W; A]^T instead, adapters' A behind W as further
// columns, tokens in their own order, all of it fp32 into the slabs [splits][T][N
// + slots r].  With fewer slots than adapters those are the ones that the batch
// (of at most 64 tokens) meets.
template <bool BACK, class C, int RING, bool SPLIT, bool BOTH>
__global__ __launch_bounds__(C::NT, 2) void proj_tile_kernel(TileArgs a) {
  constexpr bool B_KC = !BACK;
  constexpr int MI = C::MI, NI = C::NI;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  int* token = reinterpret_cast<int*>(smem + RING * C::STAGE);  // [BM] of the tile's rows, -1 past the last
  int* share = token + C::BM;                          // [BM] which of the tile's adapters, -1: none
  int* adapter = share + C::BM;                        // [BM, at least 64] the tile's adapters
  int* not_finite = adapter + std::max(C::BM, 64);
  const ProjArgs& p = a.p;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int KS = C::NW / (C::WM * C::WN), KK = 4 / KS;  // groups, and slices of a stage each
  static_assert(RING * KK % 2 == 0 && MI * NI % KS == 0, "fragments' sets alternate, blocks are shared out");
  const int group = wave / (C::WM * C::WN), in_group = wave % (C::WM * C::WN);
  const int wm = in_group / C::WN, wn = in_group % C::WN;
  const int T = p.T, K = a.in_cols, r = p.r, ncol = a.ncol, nrow = a.nrow;

  // workgroups to tiles as in ffn_gemm.hip: each XCD a contiguous eighth, in
  // panels of 4 row tiles
  int t;
  {
    const int total = ncol * nrow * (SPLIT ? a.g.splits : 1), x = blockIdx.x & 7, j = blockIdx.x >> 3;
    const int per = total >> 3, rest = total & 7;
    t = x * per + min(x, rest) + j;
  }
  const int split = SPLIT ? t / (ncol * nrow) : 0;
  t -= split * (ncol * nrow);
  constexpr int GM = 4;
  const int panel = t / (GM * ncol), in = t - panel * GM * ncol;
  const int gm = min(GM, nrow - panel * GM);
  const int tn = in / gm, tm = panel * GM + in - tn * gm;
  const bool is_w = !BOTH || tn < a.ncol_w;
  const int m0 = tm * C::BM, n0 = (is_w ? tn : tn - a.ncol_w) * C::BN;
  const int N = is_w ? a.out_cols : a.slots * r;
  auto token_of = [&](int m) { return BOTH ? m : p.o.perm[m]; };

  // Stages: those of the shared weights, then those of the tile's shares;
  // column kx of the latter's part of K is value kx % 3r of share kx / 3r.
  const int last = min(m0 + C::BM, T) - 1, deep = kParts * r;
  const int run0 = BOTH ? 0 : p.o.run[m0], with = BOTH ? 0 : p.o.count[2];  // runs from `with` on: without an adapter
  const int shares = BOTH ? 0 : max(0, min(p.o.run[last] + 1, with) - run0);
  const int base = (K + BK - 1) / BK, kfirst = K - base * BK;
  const int total = base + (shares * deep + BK - 1) / BK;
  // this split's
  const int s0 = SPLIT ? (int)((int64_t)total * split / a.g.splits) : 0;
  const int nst = SPLIT ? (int)((int64_t)total * (split + 1) / a.g.splits) : total;

  Operand<true, C::BM, C::NCA, false> A;
  Operand<B_KC, C::BN, C::NCB, false> B;
  A.init(a.g.in, 0, K, 0, kfirst, wave, 0);
  int my_share[C::NCA];  // of this lane's rows
  const uint32_t a_row = (uint32_t)(m0 + wave * C::NCA * 8 + (lane >> 3)) * deep * 2u;
  const float inv_deep = 1.f / (float)deep;
#pragma unroll
  for (int i = 0; i < C::NCA; ++i) {  // its rows from anywhere
    const int rr = (wave * C::NCA + i) * 8 + (lane >> 3), ch = (lane & 7) ^ ((rr >> 1) & 7);
    const int run = !BOTH && m0 + rr < T ? p.o.run[m0 + rr] : with;
    my_share[i] = run < with ? run - run0 : -1;
    A.off[i] = m0 + rr < T ? ((uint32_t)token_of(m0 + rr) * (uint32_t)K + ch * 8u) * 2u : kBufNone;
  }
  const int64_t ldw = BACK ? N : K;
  const uint16_t* w = is_w ? a.g.W : a.g.weights;
  const bool met = BOTH && !is_w && a.slots < p.L;  // columns of the adapters that are met
  const int64_t first = met ? 0 : B_KC ? n0 * ldw : n0;
  B.init(w + first, 0, ldw, N - n0, kfirst, wave, 0);
  if (met) {
    // a lane a token (64 at most): adapters in the order of their first tokens
    int id = lane < T ? p.ids[lane] : -1, place = -1, count = 0;
    if (id >= p.L) id = -1;
    for (uint64_t left = __ballot(id >= 0); left; ++count) {
      const int one = __builtin_ctzll(left), l = __builtin_amdgcn_readlane(id, one);
      if (id == l) place = count;
      if (lane == one) adapter[count] = l;  // (every wavefront the same)
      left &= ~__ballot(id == l);
    }
    if (tn == a.ncol_w && tm == 0 && split == 0 && wave == 0 && lane < T) a.g.place[lane] = place;
    lds_barrier();
#pragma unroll
    for (int i = 0; i < C::NCB; ++i) {
      const int rr = (wave * C::NCB + i) * 8 + (lane >> 3), ch = (lane & 7) ^ ((rr >> 1) & 7);
      const int q = (n0 + rr) / r, j = n0 + rr - q * r;
      B.off[i] = q < count ? (((uint32_t)adapter[q] * r + j) * (uint32_t)K + ch * 8u) * 2u : kBufNone;
    }
  }

  // the tile's rows and adapters
  for (int i = threadIdx.x; i < C::BM; i += C::NT) {
    const int m = m0 + i;
    int tok = -1, sh = -1;
    if (m < T) {
      tok = token_of(m);
      const int run = BOTH ? 0 : p.o.run[m];
      if (run < with) {
        sh = run - run0;
        if (i == 0 || p.o.run[m - 1] != run) adapter[sh] = p.o.adapter[run];
      }
    }
    token[i] = tok;
    share[i] = sh;
  }
  if (threadIdx.x == 0) *not_finite = 0;

  // what copy() brings next: stage s, or, behind the split's last, zeros
  auto at = [&](int s) __attribute__((always_inline)) {
    if (s < base || s >= nst) {
      A.at(s, s < nst);
      B.at(s, s < nst);
      return;
    }
    A.rs = rsrc_of(a.g.parts, 0x7fffffffu);
    B.rs = rsrc_of(a.g.weights, 0x7fffffffu);
    A.soff = B.soff = 0;
    const int k0 = (s - base) * BK;
    // of column kx: its share q and value w
    auto split_k = [&](int kx, int& q, int& w) {
      // exact: with kx < 2^17, deep < 2^9 and q <= 2^8 the product is off by less
      // than 2^-14, its distance from a whole number at least 2^-10
      q = (int)(((float)kx + 0.5f) * inv_deep);
      w = kx - q * deep;
    };
    auto rank_of = [&](int w) { return w < r ? w : w < 2 * r ? w - r : w - 2 * r; };
    // a lane's 16-byte piece of an even and of an odd copy's rows
    int q[2], w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) split_k(k0 + ((lane & 7) ^ ((lane >> 4) + 4 * h)) * 8, q[h], w[h]);
#pragma unroll
    for (int i = 0; i < C::NCA; ++i) {
      const bool odd = (wave * C::NCA + i) & 1;
      A.off[i] = my_share[i] == (odd ? q[1] : q[0]) ? a_row + (uint32_t)(i * 8 * deep + (odd ? w[1] : w[0])) * 2u : kBufNone;
    }
    if (B_KC) {
      uint32_t at_q[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        at_q[h] = kBufNone;
        if (q[h] < shares) at_q[h] = ((uint32_t)adapter[q[h]] * N * r + rank_of(w[h])) * 2u;
      }
#pragma unroll
      for (int i = 0; i < C::NCB; ++i) {
        const int c = wave * C::NCB + i, nn = n0 + c * 8 + (lane >> 3);
        const uint32_t of_q = c & 1 ? at_q[1] : at_q[0];
        B.off[i] = of_q != kBufNone && nn < N ? of_q + (uint32_t)(nn * r) * 2u : kBufNone;
      }
    } else {
#pragma unroll
      for (int i = 0; i < C::NCB; ++i) {
        constexpr int PER = 1024 / (C::BN * 2), LPR = C::BN / 8;
        const int k = (wave * C::NCB + i) * PER + lane / LPR, n = n0 + ((lane % LPR) ^ (4 * (k & 3))) * 8;
        int qk, wk;
        split_k(k0 + k, qk, wk);
        B.off[i] = qk < shares && n < N ? (((uint32_t)adapter[qk] * r + rank_of(wk)) * N + n) * 2u : kBufNone;
      }
    }
  };

  f32x16_t acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  const uint32_t smem_at = (uint32_t)(uintptr_t)(lds_char*)smem;
  u32x4_t af[2][MI], bf[2][NI];
  bool bad = false;
  auto read = [&](int slot, int kk, int set, int i) __attribute__((always_inline)) {
    const char* from = smem + slot * C::STAGE;
    kk += group * KK;
    if (i == 0) af[set][0] = A.frag(from, wm * (C::BM / C::WM), 0, kk);
    else if (i <= NI) bf[set][i - 1] = B.frag(from + C::ABYTES, wn * (C::BN / C::WN), i - 1, kk);
    else af[set][i - NI] = A.frag(from, wm * (C::BM / C::WM), i - NI, kk);
  };
  constexpr int NM = MI * NI, NF = MI + NI, NC = C::NCA + C::NCB;
  // shared: the stage is one of the shared weights'; MIXED: it need not be
  auto slice = [&](bool shared, int set, int slot, int kk, int to_slot, auto issue_c, auto mixed_c) __attribute__((always_inline)) {
    constexpr bool ISSUE = decltype(issue_c)::value;
    if (decltype(mixed_c)::value && !shared) {
      uint32_t b = 0;
#pragma unroll
      for (int j = 0; j < NI; ++j) b |= not_finite_bits(bf[set][j]);
      if (__ballot(b & 0x80008000u)) {
        bad = true;
#pragma unroll
        for (int j = 0; j < NI; ++j) bf[set][j] = only_finite(bf[set][j]);
#pragma unroll
        for (int i = 0; i < MI; ++i) af[set][i] = only_finite(af[set][i]);  // (an infinity times the 0 would be NaN)
      }
    }
    for_each<NM>([&](auto n_c) __attribute__((always_inline)) {
      constexpr int n = decltype(n_c)::value, i = n / NI, j = n % NI;
      acc[i][j] = mfma_32x32x16(bf[set][j], af[set][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      constexpr int PER = (NF + NM - 1) / NM;  // all of them, also where there are more than MFMAs
      for_each<PER>([&](auto f_c) __attribute__((always_inline)) {
        constexpr int f = n * PER + decltype(f_c)::value;
        if constexpr (f < NF) read(slot, kk, set ^ 1, f);
      });
      if constexpr (ISSUE) {
        for_each<(n + 1) * NC / NM - n * NC / NM>([&](auto q_c) __attribute__((always_inline)) {
          constexpr int q = n * NC / NM + decltype(q_c)::value;
          const uint32_t to = smem_at + to_slot * C::STAGE;
          if constexpr (q < C::NCA) A.template copy<q, false>(to, wave, 0);
          else B.template copy<q - C::NCA, false>(to + C::ABYTES, wave, 0);
        });
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  typedef std::integral_constant<bool, true> yes;
  typedef std::integral_constant<bool, false> no;
  if (!SPLIT || s0 < base) {
    A.at(s0, true);
    B.at(s0, true);
  } else {
    lds_barrier();  // share and adapter are written
    at(s0);
  }
  if (s0 == 0) {
    for_each<C::NCA>([&](auto i) { A.template copy<decltype(i)::value, true>(smem_at, wave, kfirst); });
    for_each<C::NCB>([&](auto i) { B.template copy<decltype(i)::value, true>(smem_at + C::ABYTES, wave, kfirst); });
  } else {
    for_each<C::NCA>([&](auto i) { A.template copy<decltype(i)::value, false>(smem_at, wave, 0); });
    for_each<C::NCB>([&](auto i) { B.template copy<decltype(i)::value, false>(smem_at + C::ABYTES, wave, 0); });
  }
  lds_barrier();
  for_each<RING - 1>([&](auto d_c) __attribute__((always_inline)) {
    constexpr int d = decltype(d_c)::value + 1;
    at(s0 + d);
    const uint32_t to = smem_at + d * C::STAGE;
    for_each<C::NCA>([&](auto i) { A.template copy<decltype(i)::value, false>(to, wave, 0); });
    for_each<C::NCB>([&](auto i) { B.template copy<decltype(i)::value, false>(to + C::ABYTES, wave, 0); });
  });
  // the next stage's copies have landed, those of the stages after it may be on
  // their way; own LDS reads are done
  constexpr int ON = (RING - 2) * NC;
  static_assert(ON < 64, "six bits count them");
  constexpr int wait_next = (ON & 15) | (ON >> 4 << 14) | (7 << 4);
  __builtin_amdgcn_s_waitcnt((((RING - 1) * NC) & 15) | ((RING - 1) * NC >> 4 << 14) | (7 << 4));
  bare_barrier();
#pragma unroll
  for (int i = 0; i < NF; ++i) read(0, 0, 0, i);
  // Two loops of the same steps: one that meets and brings nothing but the
  // shared weights, and one for the stages around their end and behind it (as
  // one loop with its branches 242 us where this takes 218: 8192 tokens, 4096 x
  // 4096, rank 16).
  auto round = [&](int s, auto mixed_c) __attribute__((always_inline)) {
    constexpr bool MIXED = decltype(mixed_c)::value;
    for_each<RING>([&](auto h_c) __attribute__((always_inline)) {
      constexpr int slot = decltype(h_c)::value, next = (slot + 1) % RING;
      if (MIXED && RING > 2 && s + slot >= nst) return;
      constexpr int set = slot * KK & 1;  // of the stage's first slice
      const bool shared = s + slot < base;
      for_each<KK - 1>([&](auto k_c) __attribute__((always_inline)) {
        constexpr int k = decltype(k_c)::value;
        if (k < KK - 2) slice(shared, set ^ (k & 1), slot, k + 1, 0, no(), mixed_c);
      });
      if constexpr (MIXED) {
        at(s + slot + RING);
      } else {
        A.at(s + slot + RING, true);
        B.at(s + slot + RING, true);
      }
      if (KK > 1) slice(shared, set ^ (KK & 1), slot, KK - 1, 0, no(), mixed_c);
      __builtin_amdgcn_s_waitcnt(wait_next);
      bare_barrier();
      slice(shared, set ^ (KK - 1 & 1), next, 0, slot, yes(), mixed_c);
    });
  };
  int s = s0;
#pragma unroll 1
  for (; s + 2 * RING - 1 < min(base, nst); s += RING) round(s, no());
#pragma unroll 1
  for (; s < nst; s += RING) round(s, yes());
  if (bad) *not_finite = 1;
  __builtin_amdgcn_s_waitcnt(wait_vm0 & wait_lgkm0);  // no copy outlives the loop
  bare_barrier();
  const bool mend = *not_finite;

  // A wavefront's blocks, by group: a group hands the others theirs and adds
  // what it gets, in a fixed order.
  constexpr int NB = MI * NI, PER = NB / KS;
  if constexpr (KS > 1) {
    static_assert(C::WM * C::WN * (KS - 1) * NB * 4096 <= RING * C::STAGE, "they must fit the ring");
    f32x4_t* sums = reinterpret_cast<f32x4_t*>(smem) + in_group * (KS - 1) * NB * 256 + lane;
    auto place = [&](int from, int to) { return (to * (KS - 1) + (from - to + KS) % KS - 1) * PER; };
    for_each<NB>([&](auto f_c) __attribute__((always_inline)) {
      constexpr int f = decltype(f_c)::value, to = f / PER;
      if (to == group) return;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16_t& v = acc[f / NI][f % NI];
        sums[((place(group, to) + f % PER) * 4 + q) * 64] = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
    });
    lds_barrier();
    for_each<NB>([&](auto f_c) __attribute__((always_inline)) {
      constexpr int f = decltype(f_c)::value, to = f / PER;
      if (to != group) return;
#pragma unroll
      for (int d = 1; d < KS; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4_t v = sums[((place((to + d) % KS, to) + f % PER) * 4 + q) * 64];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[f / NI][f % NI][4 * q + e] += v[e];
        }
    });
    lds_barrier();
  }

  // Epilogue, 32 rows of the wavefront at a time through its own part of the
  // LDS, so that memory sees whole lines (as in ffn_gemm.hip).
  constexpr int EC = NI < PER ? NI : PER;  // blocks side by side
  constexpr int WC = EC * 32, ROWF = WC + 4;
  constexpr int LPR = WC / 8, RPI = 64 / LPR, STEPS = 32 / RPI;
  float* mine = reinterpret_cast<float*>(smem) + wave * 32 * ROWF;
  static_assert(C::NW * 32 * ROWF * 4 <= RING * C::STAGE, "staged rows must fit the ring");
  const int l32 = lane & 31, kh = lane >> 5;
  const int oc = (lane % LPR) * 8, n = n0 + wn * (C::BN / C::WN) + group * PER % NI * 32 + oc;
#pragma unroll 1
  for (int i = group * PER / NI; i < group * PER / NI + PER / EC; ++i) {
    for_each<NB>([&](auto f_c) __attribute__((always_inline)) {
      constexpr int f = decltype(f_c)::value, b = f / NI, j = f % NI;
      if (i != b || f / PER != group) return;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4_t*>(mine + l32 * ROWF + j % EC * 32 + 8 * q + 4 * kh) =
            f32x4_t{acc[b][j][4 * q], acc[b][j][4 * q + 1], acc[b][j][4 * q + 2], acc[b][j][4 * q + 3]};
    });
    asm volatile("" ::: "memory");  // a wavefront's LDS accesses run in order
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int rr = wm * (C::BM / C::WM) + i * 32 + s * RPI + lane / LPR;
      const int tok = token[rr];
      if (tok < 0 || n >= N) continue;
      const f32x4_t* src = reinterpret_cast<const f32x4_t*>(mine + (s * RPI + lane / LPR) * ROWF + oc);
      Eight e = {{src[0], src[1]}};
      // (with K split the shares' terms are added by the split that met them)
      if (mend && share[rr] >= 0) {
        const int64_t first = (int64_t)adapter[share[rr]] * N * r;
        e = add_not_finite(e, a.g.parts + (int64_t)(m0 + rr) * deep, a.g.weights + first + (BACK ? n : (int64_t)n * r),
                           BACK ? N : 1, BACK ? 1 : r, r);
      }
      const f32x4_t* v = e.v;
      if (SPLIT) {
        const int cols = BOTH ? a.out_cols + a.slots * r : N, c = is_w ? n : a.out_cols + n;
        f32x4_t* dst = reinterpret_cast<f32x4_t*>(a.g.slabs + ((int64_t)split * T + m0 + rr) * cols + c);
        dst[0] = v[0];
        dst[1] = v[1];
      } else {
        const float o[8] = {v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]};
        store8(a.g.out + (int64_t)tok * N + n, o);
      }
    }
    asm volatile("" ::: "memory");
  }
}

// Adds the slabs in their order and scatters the rows.
__global__ __launch_bounds__(256) void proj_join_kernel(TileArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = a.out_cols / 8;
  if (i >= per * a.p.T) return;
  const int m = (int)(i / per), n = (int)(i % per) * 8;
  f32x4_t s[2];
  for (int z = 0; z < a.g.splits; ++z) {
    const f32x4_t* src = reinterpret_cast<const f32x4_t*>(a.g.slabs + ((int64_t)z * a.p.T + m) * a.out_cols + n);
#pragma unroll
    for (int h = 0; h < 2; ++h) s[h] = z ? s[h] + src[h] : src[h];
  }
  const float o[8] = {s[0][0], s[0][1], s[0][2], s[0][3], s[1][0], s[1][1], s[1][2], s[1][3]};
  store8(a.g.out + (int64_t)a.p.o.perm[m] * a.out_cols + n, o);
}

typedef FfnCfg<256, 256, 2, 4> Big;
typedef FfnCfg<128, 128, 2, 2> Small;
// One workgroup per CU, four slots: where tiles are few, a stage is as long as
// its copies take to come, and three on their way hide that.  Two groups of 2 x
// 2 wavefronts with 64 x 64 each read a third less from LDS than 2 x 4 with 64 x
// 32 (1001 tokens with order and shrink, us: 2880 x 2880, rank 32, 44.7 and
// 45.6, 4096 x 4096, rank 16, 52.6 and 54.1); one such group takes 2 us more than
// 2 x 4.  2880 x 2880 (184 tiles): 24 us with inputs from the cache, 30
// from memory, of which 8.5 are launch, first trip through memory and epilogue;
// adapters' stages 4 more.
typedef SliceCfg<128, 128, 2, 2, 2> Deep;
// Decode batches: small tiles of few wavefronts, several workgroups to a CU, so
// that nearly all of its LDS is weights on their way (up to 32 tokens three or
// four slots of 12 KB in three workgroups, beyond it three of 24 KB in two).
typedef FfnCfg<64, 128, 2, 4> Few64;
typedef FfnCfg<32, 64, 1, 2> Few32;

template <bool BACK, class C, int RING, bool SPLIT, bool BOTH = false>
int launch_cfg(TileArgs a, hipStream_t st) {
  static std::atomic<uint64_t> attr_done;
  a.ncol_w = (a.out_cols + C::BN - 1) / C::BN;
  const int64_t ncol = a.ncol_w + (BOTH ? (a.slots * a.p.r + C::BN - 1) / C::BN : 0), nrow = (a.p.T + C::BM - 1) / C::BM;
  const int64_t grid = ncol * nrow * a.g.splits;
  if (grid * C::NT > 0xffffffff) return MOE_LORA_EUNSUPPORTED;
  a.ncol = (int)ncol;
  a.nrow = (int)nrow;
  const void* fn = reinterpret_cast<const void*>(&proj_tile_kernel<BACK, C, RING, SPLIT, BOTH>);
  const int rc = ensure_dynamic_lds(fn, tile_lds<C, RING>(), attr_done);
  if (rc) return rc;
  proj_tile_kernel<BACK, C, RING, SPLIT, BOTH><<<(unsigned)grid, C::NT, tile_lds<C, RING>(), st>>>(a);
  if (SPLIT && !BOTH) {
    const int64_t n = (int64_t)a.p.T * (a.out_cols / 8);
    proj_join_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a);
  }
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

// Which tile, and how many K splits: the rule of ffn_gemm.hip, or, up to a
// workgroup per CU in all, Few64 or Deep (0.33 and 0.45 us a stage; a launch for
// the join and the slabs' way to memory and back as there).  520 tokens, 2880 x
// 2880, rank 64 with its order and shrink: 50 us with Few64 (207 tiles), 60 with
// Deep; 513 tokens, rank 16, 35 and 41; 1001 tokens, rank 32 (368 and 184 tiles),
// 51 with Deep, 64 without; 4096 x 4096, rank 16, 58 and 76.
struct Plan {
  enum Tile { BIG, SMALL, DEEP, FEW64, FEW32 } tile;
  int splits;
};

Plan plan_of(int T, int N, int K, bool joined_anyway) {
  const TilePlan f = tile_plan(T, N, K);
  Plan best{f.big ? Plan::BIG : Plan::SMALL, f.splits};
  double least = f.us - (joined_anyway && f.splits > 1 ? 3.5 : 0.);
  const int stages = (K + BK - 1) / BK;
  auto consider = [&](Plan::Tile tile, int bm, double stage_us) {
    const int64_t tiles = (int64_t)((T + bm - 1) / bm) * ((N + 127) / 128);
    for (int s = 1; s * tiles <= 256 && s <= 16 && s * 3 <= std::max(3, stages); ++s) {
      const double us = 0.5 + (stages + s - 1) / s * stage_us +
                        (s > 1 || joined_anyway ? s * (double)T * N * 8 * 0.16e-6 + (joined_anyway ? 0. : 3.5) : 0.);
      if (us < least) {
        least = us;
        best = Plan{tile, s};
      }
    }
  };
  consider(Plan::DEEP, Deep::BM, 0.45);
  consider(Plan::FEW64, Few64::BM, 0.33);
  return best;
}

// (two shares a tile: what a tile of several requests has)
Plan plan_of(const ProjArgs& p, bool back) {
  return plan_of(p.T, back ? p.K : p.N, (back ? p.N : p.K) + 2 * kParts * p.r, false);
}

// x [W; A]^T.  Decode batches: Few32 up to 32 tokens, Few64 up to 256 and 256
// tiles (201 tokens, 2880 x 2880: 18.5 us, 24 with Deep; 4096 x 11008, 352
// tiles: 59 and 52), with as many K splits as pay (0.2 us a stage; a split costs
// its start and its slab), up to a workgroup per CU: with a few more, some CUs
// have two and the rest wait for them.  Forward, us, weights from memory, 8
// adapters of rank 16, up to 256 and up to 288: one token, 4096 x 4096, 13.6
// (195 workgroups) and 15.0 (260); 2048 x 4096, 10.5 and 11.3; 8192 x 4096, 19.4
// and 24.6; 32 tokens, 5120 x 4096, 15.8 and 20.0; up to as many as are resident
// (three to a CU) 15.0, 16.8 for 32 tokens, 4096 x 4096 (14.7).  Few64, where two
// to a CU are resident, up to 256 and up to 512: 100 tokens, 2880 x 5120, 19.9
// and 21.7; 201, 29.0 and 29.1; 256, 4096 x 4096, 38.6 and 35.9.
Plan plan_both(const ProjArgs& p) {
  const int cols = p.N + proj_slots(p.T, p.L) * p.r, stages = (p.K + BK - 1) / BK;
  const bool few32 = p.T <= 32;
  const int64_t tiles = few32 ? (cols + 63) / 64 : (int64_t)((p.T + 63) / 64) * ((cols + 127) / 128);
  if (!few32 && (p.T > 256 || tiles > 256)) {
    const Plan f = plan_of(p.T, cols, p.K, true);
    return Plan{f.tile == Plan::BIG ? Plan::SMALL : f.tile, f.splits};
  }
  Plan best{few32 ? Plan::FEW32 : Plan::FEW64, 1};
  double least = 1e9;
  for (int s = 1; s == 1 || (s * tiles <= 256 && s <= 16 && 2 * s <= stages); ++s) {
    const double us = (stages + s - 1) / s * 0.2 + s * (0.35 + 1.5e-6 * p.T * cols);
    if (us < least) {
      least = us;
      best.splits = s;
    }
  }
  return best;
}

template <bool BACK>
int launch(TileArgs a, hipStream_t st) {
  const Plan f = plan_of(a.p, BACK);
  a.g.splits = f.splits;
  const bool split = f.splits > 1;
  switch (f.tile) {
    case Plan::DEEP:
      return split ? launch_cfg<BACK, Deep, 4, true>(a, st) : launch_cfg<BACK, Deep, 4, false>(a, st);
    case Plan::FEW64:
      return split ? launch_cfg<BACK, Few64, 3, true>(a, st) : launch_cfg<BACK, Few64, 3, false>(a, st);
    case Plan::BIG: return launch_cfg<BACK, Big, 2, false>(a, st);
    default:
      return split ? launch_cfg<BACK, Small, 2, true>(a, st) : launch_cfg<BACK, Small, 2, false>(a, st);
  }
}

}  // namespace

int proj_gemm_plan(int T, int K, int N, int r, bool back) {
  ProjArgs p = {};
  p.T = T, p.K = K, p.N = N, p.r = r;
  const Plan f = plan_of(p, back);
  return f.tile * 32 + f.splits;
}

int proj_both_plan(int T, int K, int N, int L, int r) {
  ProjArgs p = {};
  p.T = T, p.K = K, p.N = N, p.L = L, p.r = r;
  const Plan f = plan_both(p);
  return f.tile * 32 + f.splits;
}

size_t proj_gemm_slab_bytes(const ProjArgs& p, bool back) {
  const int s = plan_of(p, back).splits;
  return s > 1 ? (size_t)s * p.T * (back ? p.K : p.N) * sizeof(float) : 0;
}

int launch_proj_gemm(const ProjArgs& p, bool back, ProjGemm g, hipStream_t st) {
  const TileArgs a{p, g, back ? p.N : p.K, back ? p.K : p.N, 0, 0, 0, 0};
  return back ? launch<true>(a, st) : launch<false>(a, st);
}

int proj_slots(int T, int L) { return T <= 64 && T < L ? T : L; }

int proj_both_splits(const ProjArgs& p) { return plan_both(p).splits; }

int launch_proj_both(const ProjArgs& p, const uint16_t* x, const uint16_t* W, const uint16_t* A, float* slabs,
                     int32_t* place, hipStream_t st) {
  const Plan f = plan_both(p);
  const ProjGemm g{x, W, nullptr, A, nullptr, slabs, f.splits, place};
  const TileArgs a{p, g, p.K, p.N, 0, 0, 0, proj_slots(p.T, p.L)};
  switch (f.tile) {
    case Plan::FEW32: return launch_cfg<false, Few32, 4, true, true>(a, st);
    case Plan::FEW64: return launch_cfg<false, Few64, 3, true, true>(a, st);
    case Plan::DEEP: return launch_cfg<false, Deep, 4, true, true>(a, st);
    default: return launch_cfg<false, Small, 2, true, true>(a, st);
  }
}

}  // namespace moelora
