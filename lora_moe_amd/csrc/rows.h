// Products of a few rows with a large weight matrix: the weight stream.
//
//   out[m][n] = sum_k x[m][k] w(n, k),   or the gated pair
//   out[m][n] = act(sum x w_gate) * sum x w_up
//
// Every weight is read once and meets all rows at once (MFMA 16 x 16 x 32,
// rows on one side, a tile of 16 weight rows on the other).  What bounds such
// a kernel is the rate at which a CU has lines fetched to it, about 30 GB/s,
// and the bytes in flight that sustain it; the rows' fragments come on top of
// the weights, so the two kernels differ in how they get those:
//
//   rows_direct_kernel, up to 8 rows: a workgroup owns one tile (gated: a
//     gate tile and its up tile), its wavefronts split K, each taking every
//     KS-th chunk of 128 k and fetching the rows' pieces itself.
//   rows_shared_kernel: up to 8 wavefronts of a workgroup own different tiles
//     and walk K together, the rows' chunk comes once for all of them,
//     through LDS.  Where that leaves too few workgroups K is split over
//     the grid into fp32 slabs, which rows_join_kernel adds up.
//
// Measured, bf16: one row, 4096 x 11008 (gate and up 180 MB, down 90): 35 and
// 20 us, 5.1 and 4.6 TB/s; 32 rows, 5120 x 25600 (524 and 262 MB): 118 and 59
// us, 4.4 TB/s; a large copy moves 4.9.
//
// Loads are buffer loads, so that rows, k and chunks past the end are zeros
// without traffic or branches: the loops are straight-line code in which each
// wait names the loads it needs.
//
// The weights' format is a policy W (ffn_rows.hip, w4.hip): Tile, where a
// tile lies; Buf, a chunk of it in registers; load(); operand(), the 32-deep
// step j of a chunk as bf16; Acc, the sums.  W::DEPTH chunks are in flight;
// a workgroup has up to W::MAX_FRAGMENTS fragments of 16 rows.
#pragma once

#include <algorithm>
#include <type_traits>

#include "device_util.h"
#include "gate_act.h"
#include "moe_lora.h"

namespace moelora {

constexpr int kRowsJoinMax = 16;  // slabs at most

struct RowsArgs {
  const uint16_t* x;     // [M][K]
  const uint16_t* x_lo;  // PAIR: the rows' remainders, the product takes x + x_lo
  uint16_t* out;         // [M][N]
  uint16_t* out_lo;      // gated: the remainder of out's rounding, or NULL
  float* gu;             // gated: [M][2N], both sums kept, or NULL
  int M, N, K;
  int act;
  float* slabs;          // K split over the grid: [split][M][N] (gated: [split][2][M][N]), or NULL
  int splits;
  int groups;            // shared form: workgroups along the columns
};

__device__ __forceinline__ void rows_store(const RowsArgs& p, bool gated, int m, int n, float a, float u) {
  const float r = gated ? gate_act<false>(p.act, a, nullptr) * u : a;
  const int64_t at = (int64_t)m * p.N + n;
  if (gated && p.gu) {
    p.gu[(int64_t)m * 2 * p.N + n] = a;
    p.gu[(int64_t)m * 2 * p.N + p.N + n] = u;
  }
  if (gated && p.out_lo) f32_to_bf16_pair(r, p.out + at, p.out_lo + at);
  else p.out[at] = f32_to_bf16(r);
}

__device__ __forceinline__ u32x4_t rows_load(const void* base, uint32_t bytes, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(u32x4_t,
                            __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(base, bytes), (int)voff, (int)soff, 0));
}

// n chunks through a ring of D register buffers that hold the first D of them:
// mul(u) takes buffer u, load(u, i) brings chunk i into it.  Whole rounds,
// then the rest without loads: one way through the loop, so that its waits
// count the loads in flight exactly.
template <int D, int U = 0, class M>
__device__ __forceinline__ void rows_rest(int left, M&& mul) {
  if constexpr (U < D) {
    if (left > U) {
      mul(std::integral_constant<int, U>());
      rows_rest<D, U + 1>(left, static_cast<M&&>(mul));
    }
  }
}
template <int U, int D, class M, class F>
__device__ __forceinline__ void rows_round(int i, M&& mul, F&& load) {
  if constexpr (U < D) {
    mul(std::integral_constant<int, U>());
    load(std::integral_constant<int, U>(), i + U + D);
    rows_round<U + 1, D>(i, static_cast<M&&>(mul), static_cast<F&&>(load));
  }
}
template <int D, class M, class F>
__device__ __forceinline__ void rows_ring(int n, M&& mul, F&& load) {
  int i = 0;
  for (; i + D <= n; i += D) rows_round<0, D>(i, mul, load);
  rows_rest<D>(n - i, mul);
}

// Up to R = 4 or 8 rows.
template <class W, int R, bool GATE, bool PAIR>
__global__ __launch_bounds__(512, 2) void rows_direct_kernel(RowsArgs p, typename W::Args wa) {
  constexpr int CT = GATE ? 2 : 1, NX = PAIR ? 2 : 1, D = W::DEPTH * 2 / CT;
  // a chunk of the rows (PAIR: then one of their remainders, which meet the
  // weights as further rows), 16 bytes of padding per row against bank conflicts
  constexpr int XROW = 256 + 16, XBYTES = R * XROW, XPL = R / 4;
  extern __shared__ __attribute__((aligned(16))) char rows_smem[];
  const int lane = threadIdx.x & 63, ks = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, kq = lane >> 4;
  const int tile0 = blockIdx.x;

  const W w(wa, p.N, p.K, lane);
  typename W::Tile tiles[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) tiles[t] = w.tile(tile0, t);
  // lane l brings piece l % 16 of rows l / 16 and l / 16 + 4 (rows past M:
  // zeros) and reads the fragment of row l % R (PAIR: l % 2R), further rows
  // repeat them and their sums are dropped
  const uint32_t xbytes = (uint32_t)p.M * (uint32_t)p.K * 2u;
  const uint32_t xoff = ((uint32_t)kq * (uint32_t)p.K + (uint32_t)l16 * 8u) * 2u;
  char* xl = rows_smem + wave * (NX * XBYTES);

  typename W::Buf q[D][CT];
  u32x4_t x[D][NX][XPL];
  const int chunks = (p.K + 127) >> 7;
  // workgroups start at different chunks: in step they would all ask for the
  // same memory channels (rows lie a fixed distance apart)
  const int rot = (int)((blockIdx.x * 5u) % (unsigned)chunks);
  auto load = [&](int u, int i) __attribute__((always_inline)) {
    const bool real = i < chunks;
    const int c = i + rot < chunks ? i + rot : i + rot - chunks;
    const uint32_t o = l16 * 8 < (real ? p.K - c * 128 : 0) ? xoff : kBufNone;
#pragma unroll
    for (int h = 0; h < XPL; ++h) {
      const uint32_t oh = o == kBufNone ? o : o + h * 8u * (uint32_t)p.K;  // 4 rows on
      x[u][0][h] = rows_load(p.x, xbytes, oh, (uint32_t)c * 256u);
      if (PAIR) x[u][NX - 1][h] = rows_load(p.x_lo, xbytes, oh, (uint32_t)c * 256u);
    }
#pragma unroll
    for (int t = 0; t < CT; ++t) w.load(q[u][t], tiles[t], c, real);
    // loads return in order: kept in the order of their use
    __builtin_amdgcn_sched_barrier(0);
  };
  typename W::template Acc<1, CT> acc;
  acc.clear();
  const int n = wave < chunks ? (chunks - wave + ks - 1) / ks : 0;
#pragma unroll
  for (int u = 0; u < D; ++u) load(u, wave + u * ks);
  auto mul = [&](auto u_c) __attribute__((always_inline)) {
    constexpr int u = decltype(u_c)::value;
    // (a wavefront's LDS accesses run in order)
#pragma unroll
    for (int v = 0; v < NX; ++v)
#pragma unroll
      for (int h = 0; h < XPL; ++h)
        *reinterpret_cast<u32x4_t*>(xl + v * XBYTES + (kq + 4 * h) * XROW + l16 * 16) = x[u][v][h];
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4_t a =
          *reinterpret_cast<const u32x4_t*>(xl + (l16 & (R * NX - 1)) * XROW + j * 64 + kq * 16);
      acc.begin(w, q[u], j);
      acc.rows(0, a);
#pragma unroll
      for (int t = 0; t < CT; ++t) acc.mul(0, t, a, w.operand(q[u][t], j));
      acc.end(w, q[u], j);
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  rows_ring<D>(n, mul, [&](auto u_c, int i) __attribute__((always_inline)) {
    load(decltype(u_c)::value, wave + i * ks);
  });

  __syncthreads();  // the rows' parts of the LDS become the sums'
  // the wavefronts' sums, added in their order
  f32x4_t* part = reinterpret_cast<f32x4_t*>(rows_smem);
#pragma unroll
  for (int t = 0; t < CT; ++t) part[(wave * CT + t) * 64 + lane] = acc.sum(0, t);
  __syncthreads();
  if (wave) return;
  f32x4_t s[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    s[t] = part[t * 64 + lane];
    for (int v = 1; v < ks; ++v) s[t] += part[(v * CT + t) * 64 + lane];
    if (PAIR) {  // row m's remainder is row R + m, 4 R lanes on
#pragma unroll
      for (int v = 0; v < 4; ++v) s[t][v] += __shfl_down(s[t][v], 4 * R, 64);
    }
  }
  const int no = tile0 * 16 + l16;
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (kq * 4 + v < p.M && no < p.N) rows_store(p, GATE, kq * 4 + v, no, s[0][v], s[CT - 1][v]);
}

// RF: fragments of 16 rows.  Grid: groups of up to 8 tiles (an even share
// each), row tiles, K splits.
template <class W, int RF, bool GATE, bool PAIR>
__global__ __launch_bounds__(512, 2) void rows_shared_kernel(RowsArgs p, typename W::Args wa) {
  constexpr int CT = GATE ? 2 : 1, NX = PAIR ? 2 : 1, D = RF <= 2 ? W::DEPTH * 2 / CT : std::min(W::DEPTH * 2 / CT, 4);
  constexpr int PIECES = RF * 256 * NX;           // 16-byte pieces of a chunk of rows
  constexpr int XPT = (PIECES + 511) / 512;       // per thread
  __shared__ __attribute__((aligned(16))) u32x4_t xl[2][PIECES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, kq = lane >> 4;
  const int m0 = blockIdx.y * (16 * RF), rows = min(16 * RF, p.M - m0);
  // wavefronts past the group's tiles only bring rows
  const int all = (p.N + 15) >> 4;
  const int first = (int)((int64_t)all * blockIdx.x / p.groups), last = (int)((int64_t)all * (blockIdx.x + 1) / p.groups);
  const int tile0 = first + wave;
  const bool active = tile0 < last;

  const W w(wa, p.N, p.K, lane);
  typename W::Tile tiles[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) tiles[t] = w.tile(active ? tile0 : first, t);

  // this workgroup's chunks
  const int chunks = (p.K + 127) >> 7, z = blockIdx.z;
  const int c0 = (int)((int64_t)chunks * z / p.splits), c1 = (int)((int64_t)chunks * (z + 1) / p.splits);

  // pieces: thread t brings piece t % 16 of rows t / 16, t / 16 + 32, ..
  // (whole lines), into the order in which a fragment reads them
  const uint32_t xbytes = (uint32_t)rows * (uint32_t)p.K * 2u;
  const uint16_t* xbase[NX];
  xbase[0] = p.x + (int64_t)m0 * p.K;
  if (PAIR) xbase[NX - 1] = p.x_lo + (int64_t)m0 * p.K;
  const int piece = tid & 15;
  // workgroups start at different chunks, as above
  const int n = c1 - c0, rot = n > 0 ? (int)((blockIdx.x * 5u) % (unsigned)n) : 0;
  auto chunk = [&](int i) { return c0 + (i + rot < n ? i + rot : i + rot - n); };
  u32x4_t xr[D][XPT];
  auto load_x = [&](int u, int i) __attribute__((always_inline)) {
    const int c = chunk(i);
    const bool ok = i < n && c * 128 + piece * 8 < p.K;
#pragma unroll
    for (int e = 0; e < XPT; ++e) {
      const int r = (tid >> 4) + e * 32;  // row of the NX * 16 RF stacked ones
      const int rr = r & (16 * RF - 1);
      const uint32_t o = ok && rr < rows && r < NX * 16 * RF
                             ? ((uint32_t)rr * (uint32_t)p.K + (uint32_t)piece * 8u) * 2u
                             : kBufNone;
      // a wavefront's 4 rows are all of one half of the pair
      xr[u][e] = rows_load(PAIR && __builtin_amdgcn_readfirstlane(r) >= 16 * RF ? xbase[NX - 1] : xbase[0], xbytes, o,
                        (uint32_t)c * 256u);
    }
  };
  auto put_x = [&](int b, int u) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < XPT; ++i) {
      const int r = (tid >> 4) + i * 32;
      if (PIECES >= 512 || r < NX * 16 * RF)
        // rows swizzled by the piece, so that a wavefront's write (4 rows, 16
        // pieces) meets all banks alike
        xl[b][((r >> 4) * 4 + (piece >> 2)) * 64 + (piece & 3) * 16 + ((r & 15) ^ ((piece & 3) << 2))] = xr[u][i];
    }
  };
  typename W::Buf q[D][CT];
  auto load_w = [&](int u, int i) __attribute__((always_inline)) {
    const int c = chunk(i);
#pragma unroll
    for (int t = 0; t < CT; ++t) w.load(q[u][t], tiles[t], c, i < n);
  };
  typename W::template Acc<RF, CT> acc;
  acc.clear();
  auto mul = [&](auto u_c, auto act_c) __attribute__((always_inline)) {
    constexpr int u = decltype(u_c)::value;
    // the buffer written here was last read two chunks ago, before the
    // previous barrier
    put_x(u & 1, u);
    lds_barrier();
    if constexpr (!decltype(act_c)::value) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4_t a[NX][RF];
#pragma unroll
      for (int v = 0; v < NX; ++v)
#pragma unroll
        for (int f = 0; f < RF; ++f) a[v][f] = xl[u & 1][((v * RF + f) * 4 + j) * 64 + (lane ^ (kq << 2))];
      acc.begin(w, q[u], j);
#pragma unroll
      for (int v = 0; v < NX; ++v)
#pragma unroll
        for (int f = 0; f < RF; ++f) acc.rows(f, a[v][f]);
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        const u32x4_t bw = w.operand(q[u][t], j);
#pragma unroll
        for (int v = 0; v < NX; ++v)
#pragma unroll
          for (int f = 0; f < RF; ++f) acc.mul(f, t, a[v][f], bw);
      }
      acc.end(w, q[u], j);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto run = [&](auto act_c) __attribute__((always_inline)) {
    constexpr bool ACT = decltype(act_c)::value;
#pragma unroll
    for (int u = 0; u < D; ++u) {
      load_x(u, u);
      if (ACT) load_w(u, u);
      __builtin_amdgcn_sched_barrier(0);  // loads return in order: kept in the order of their use
    }
    rows_ring<D>(n, [&](auto u_c) __attribute__((always_inline)) { mul(u_c, act_c); },
                 [&](auto u_c, int i) __attribute__((always_inline)) {
                   load_x(decltype(u_c)::value, i);
                   if (ACT) load_w(decltype(u_c)::value, i);
                   __builtin_amdgcn_sched_barrier(0);
                 });
  };
  if (!active) {
    run(std::false_type());
    return;
  }
  run(std::true_type());
  const int no = tile0 * 16 + l16;
  if (no >= p.N) return;
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int m = m0 + f * 16 + kq * 4 + v;
      if (m >= p.M) continue;
      if (p.splits == 1) {
        rows_store(p, GATE, m, no, acc.sum(f, 0)[v], acc.sum(f, CT - 1)[v]);
      } else {
#pragma unroll
        for (int t = 0; t < CT; ++t)
          p.slabs[((int64_t)(z * CT + t) * p.M + m) * p.N + no] = acc.sum(f, t)[v];
      }
    }
}

// Adds the slabs in their order.
template <bool GATE>
__global__ __launch_bounds__(256) void rows_join_kernel(RowsArgs p) {
  constexpr int CT = GATE ? 2 : 1;
  const int64_t size = (int64_t)p.M * p.N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= size) return;
  float s[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) s[t] = p.slabs[t * size + i];
  for (int z = 1; z < p.splits; ++z)
#pragma unroll
    for (int t = 0; t < CT; ++t) s[t] += p.slabs[(z * CT + t) * size + i];
  rows_store(p, GATE, (int)(i / p.N), (int)(i % p.N), s[0], s[CT - 1]);
}

// ---- host side: which form, with how many workgroups

inline int rows_fragments(int M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }

struct RowsPlan {
  bool direct;
  int groups, splits;  // shared form
};

// The direct form fetches the rows anew for every tile: 2 M lines of 128
// bytes per chunk beside the weights' (lines_per_chunk of them), at about 7
// TB/s over all CUs.  The shared form costs about 5 us more than its weights:
// another launch and the slabs.  (M = 5, 11008 x 2880, 4 bits: 10 us direct
// against 15; M = 32, 4096 x 11008: 30 against 14.)
inline RowsPlan rows_plan(int M, int N, int K, int lines_per_chunk) {
  RowsPlan r{false, 0, 1};
  const int64_t tiles = (N + 15) / 16, chunks = (K + 127) / 128;
  r.direct = M <= 8 && (2 * M <= lines_per_chunk / 2 || tiles * chunks * 2 * M * 128 < 5 * 7000000LL);
  if (r.direct) return r;
  // at most one workgroup per CU (256) where K is split, since a second round
  // of a few would take as long as the first; 6 chunks each, the best on the
  // mean: with fewer the slabs cost more than they spare, with more too few
  // workgroups are left in small matrices (us with 4, 6 and 8: 16 rows through
  // the bf16 block, 2880 x 2880 27.4, 24.4, 26.9; 32 rows, 29.4, 26.5, 27.8; 4
  // bits, 32 rows, 2880 x 2880 10.2, 9.7, 10.5, 4096 x 4096 12.3, 11.5, 10.8; 64
  // rows, 1024 x 2048 9.5, 9.9, 11.0; 4096 x 11008 24.4, 24.4, 24.2)
  const int64_t rt = 16 * rows_fragments(M), row_tiles = (M + rt - 1) / rt, least = (tiles + 7) / 8;
  const int64_t s = std::min<int64_t>(256 / (least * row_tiles), (chunks + 5) / 6);
  r.splits = (int)std::max<int64_t>(1, std::min<int64_t>(s, kRowsJoinMax));
  r.groups = (int)std::max<int64_t>(least, std::min<int64_t>(tiles, 256 / (r.splits * row_tiles)));
  return r;
}

// Bytes of slabs that a product needs.
inline size_t rows_slab_bytes(const RowsPlan& r, int M, int N, bool gated) {
  return r.splits > 1 ? (size_t)r.splits * (gated ? 2 : 1) * M * N * sizeof(float) : 0;
}

// The most that any product of M rows needs: with all splits the groups, of
// 128 columns (gated: pairs) and up to 16 RF rows, number at most 256.
inline size_t rows_slab_bound(int M) {
  return (size_t)256 * 128 * 16 * rows_fragments(M) * 2 * sizeof(float);
}

// Wavefronts that split K in the direct form: at most 3000 of them over the
// chip, at least two chunks each.  (4 bits, us with 1500, 3000 and 6000 at most,
// N x K, one row: 4096 x 11008 10.3, 8.0, 8.0; 5120 x 25600 20.5, 18.6, 18.4;
// 25600 x 5120 18.0, 18.2, 17.0; five rows: 11008 x 4096 9.1, 9.4, 12.6.)
inline int rows_ksplit(int64_t workgroups, int K) {
  int ks = 8;
  while (ks > 1 && (workgroups * ks > 3000 || K / 128 < 2 * ks)) ks >>= 1;
  return ks;
}

template <class W, int R, bool GATE, bool PAIR>
void launch_rows_direct(const RowsArgs& a, const typename W::Args& wa, hipStream_t st) {
  const int tiles = (a.N + 15) / 16, ks = rows_ksplit(tiles, a.K);
  constexpr int lds = std::max((GATE ? 2 : 1) * 1024, (PAIR ? 2 : 1) * R * (256 + 16));
  rows_direct_kernel<W, R, GATE, PAIR><<<tiles, 64 * ks, ks * lds, st>>>(a, wa);
}

template <class W, bool GATE, bool PAIR>
void launch_rows(RowsArgs a, const typename W::Args& wa, hipStream_t st) {
  const RowsPlan r = rows_plan(a.M, a.N, a.K, W::LINES);
  if (r.direct) {
    if (a.M <= 4) launch_rows_direct<W, 4, GATE, PAIR>(a, wa, st);
    else launch_rows_direct<W, 8, GATE, PAIR>(a, wa, st);
    return;
  }
  a.splits = r.splits;
  a.groups = r.groups;
  const int rf = rows_fragments(a.M);
  const dim3 grid(r.groups, (a.M + 16 * rf - 1) / (16 * rf), r.splits);
  if (rf == 1) rows_shared_kernel<W, 1, GATE, PAIR><<<grid, 512, 0, st>>>(a, wa);
  if constexpr (!PAIR) {
    if (rf == 2) rows_shared_kernel<W, 2, GATE, false><<<grid, 512, 0, st>>>(a, wa);
    if constexpr (W::MAX_FRAGMENTS >= 4)
      if (rf == 4) rows_shared_kernel<W, 4, GATE, false><<<grid, 512, 0, st>>>(a, wa);
  }
  if (a.splits > 1) {
    const int64_t n = (int64_t)a.M * a.N;
    rows_join_kernel<GATE><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a);
  }
}

}  // namespace moelora
