// Products of a few rows with a large weight matrix: the weight stream.
//
//   out[m][n] = sum_k x[m][k] w(n, k),  m < 16 RF,  or the gated pair
//   out[m][n] = act(sum x w_gate) * sum x w_up
//
// Every weight is read once and meets all rows at once (MFMA 16 x 16 x 32,
// rows on one side, 16 weight rows on the other), so the kernel is bound by
// how many bytes of weights are in flight.  A workgroup owns CT tiles of 16
// weight rows (gate: half of them gate rows, half the matching up rows) and
// its wavefronts split K, each taking every KS-th chunk of 128 k: the more
// wavefronts the fewer columns there are, up to 8 (the host picks KS), and
// their sums meet once, through LDS, in a fixed order.  Two chunks' loads
// are in flight per wavefront, in registers; the rows' fragments come from
// the L2 with them (rows past M repeat the last one, their sums are dropped).
//
// The weights' format is a policy W:
//   Tile  what a lane keeps of a tile between chunks
//   Buf   a chunk of a tile in registers
//   load(buf, tile, chunk, masked), and per 32-deep step j either operand
//   form, see the two policies (ffn_rows.hip, w4.hip)
#pragma once

#include "device_util.h"
#include "gate_act.h"

namespace moelora {

struct RowsArgs {
  const uint16_t* x;     // [M][K]
  const uint16_t* x_lo;  // PAIR: the rows' remainders, the product takes x + x_lo
  uint16_t* out;         // [M][N]
  uint16_t* out_lo;      // gate: the remainder of out's rounding, or NULL
  int M, N, K;
  int act;
};

template <class W, int RF, int CT, bool GATE, bool PAIR>
__global__ __launch_bounds__(512, 2) void rows_kernel(RowsArgs p, typename W::Args wa) {
  static_assert(!GATE || CT == 2, "one gate and one up tile");
  constexpr int NX = PAIR ? 2 : 1;
  extern __shared__ __attribute__((aligned(16))) char rows_smem[];
  const int lane = threadIdx.x & 63, ks = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, kq = lane >> 4;
  const int m0 = blockIdx.y * (16 * RF);
  const int tile0 = blockIdx.x * (GATE ? 1 : CT);  // first 16-column tile of the output

  W w(wa, p, lane);
  typename W::Tile tiles[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) tiles[t] = GATE ? w.tile(tile0, t) : w.tile(tile0 + t, 0);
  const uint16_t* xr[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) xr[f] = p.x + (int64_t)min(m0 + f * 16 + l16, p.M - 1) * p.K + kq * 8;
  const int64_t lo = PAIR ? p.x_lo - p.x : 0;

  struct Chunk {
    typename W::Buf q[CT];
    u32x4_t x[NX][RF][4];
  } b0, b1;
  auto load = [&](Chunk& b, int c, bool masked) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < CT; ++t) w.load(b.q[t], tiles[t], c, masked);
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = c * 128 + j * 32;
        const bool ok = !masked || k + kq * 8 < p.K;
        b.x[0][f][j] = ok ? ld16(xr[f] + k) : zero4();
        if (PAIR) b.x[NX - 1][f][j] = ok ? ld16(xr[f] + lo + k) : zero4();
      }
  };
  typename W::template Acc<RF, CT> acc;
  acc.clear();
  auto mul = [&](const Chunk& b, int c) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int v = 0; v < NX; ++v)
#pragma unroll
        for (int f = 0; f < RF; ++f) acc.rows(f, b.x[v][f][j]);
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        const u32x4_t bw = w.operand(b.q[t], j);
#pragma unroll
        for (int v = 0; v < NX; ++v)
#pragma unroll
          for (int f = 0; f < RF; ++f) acc.mul(f, t, b.x[v][f][j], bw);
      }
      acc.step(w, tiles, b.q, c, j);
    }
  };
  // this wavefront's whole chunks, two in flight; straight-line code, so that
  // each wait names the loads it needs
  const int full = p.K >> 7;
  const int n = wave < full ? (full - wave + ks - 1) / ks : 0;
  auto at = [&](int i) { return wave + i * ks; };
  if (n >= 2) {
    load(b0, at(0), false);
    load(b1, at(1), false);
    int i = 0;
    for (; i + 4 <= n; i += 2) {
      mul(b0, at(i));
      load(b0, at(i + 2), false);
      mul(b1, at(i + 1));
      load(b1, at(i + 3), false);
    }
    mul(b0, at(i));
    if (n - i == 3) {
      load(b0, at(i + 2), false);
      mul(b1, at(i + 1));
      mul(b0, at(i + 2));
    } else {
      mul(b1, at(i + 1));
    }
  } else if (n == 1) {
    load(b0, at(0), false);
    mul(b0, at(0));
  }
  if ((p.K & 127) && full % ks == wave) {  // the rest of K, lanes past its end zero
    load(b0, full, true);
    mul(b0, full);
  }

  // the wavefronts' sums, added in their order
  f32x4_t* part = reinterpret_cast<f32x4_t*>(rows_smem);
  if (ks > 1) {
#pragma unroll
    for (int t = 0; t < CT; ++t)
#pragma unroll
      for (int f = 0; f < RF; ++f) part[((wave * CT + t) * RF + f) * 64 + lane] = acc.sum(f, t);
    __syncthreads();
  }
  constexpr int OT = GATE ? 1 : CT;
  for (int o = wave; o < OT * RF; o += ks) {
    const int t = o / RF, f = o % RF;
    f32x4_t s[GATE ? 2 : 1];
    if (ks > 1) {
#pragma unroll
      for (int h = 0; h < (GATE ? 2 : 1); ++h) {
        s[h] = part[((t + h) * RF + f) * 64 + lane];
        for (int v = 1; v < ks; ++v) s[h] += part[((v * CT + t + h) * RF + f) * 64 + lane];
      }
    } else {
#pragma unroll
      for (int tt = 0; tt < CT; ++tt)
#pragma unroll
        for (int ff = 0; ff < RF; ++ff)
          if (ff == f && (GATE || tt == t)) s[GATE ? tt : 0] = acc.sum(ff, tt);
    }
    const int n_out = (tile0 + t) * 16 + l16;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int m = m0 + f * 16 + kq * 4 + v;
      if (m >= p.M || n_out >= p.N) continue;
      const float r = GATE ? gate_act<false>(p.act, s[0][v], nullptr) * s[GATE ? 1 : 0][v] : s[0][v];
      const uint16_t hi = f32_to_bf16(r);
      p.out[(int64_t)m * p.N + n_out] = hi;
      if (GATE && p.out_lo) p.out_lo[(int64_t)m * p.N + n_out] = f32_to_bf16(r - bf16_to_f32(hi));
    }
  }
}

// Wavefronts that split K: enough for about 2048 of them over the chip's 256
// CUs (8 each, which have 64 KB of weights in flight), of at least two chunks
// each.
inline int rows_ksplit(int64_t workgroups, int K) {
  int ks = 8;
  while (ks > 1 && (workgroups * ks > 3072 || K / 128 < 2 * ks)) ks >>= 1;
  return ks;
}

template <class W, int RF, int CT, bool GATE, bool PAIR>
void launch_rows_cfg(const RowsArgs& a, const typename W::Args& wa, hipStream_t st) {
  const int tiles = (a.N + 15) / 16, per = GATE ? 1 : CT;
  const dim3 grid((tiles + per - 1) / per, (a.M + 16 * RF - 1) / (16 * RF));
  const int ks = rows_ksplit((int64_t)grid.x * grid.y, a.K);
  rows_kernel<W, RF, CT, GATE, PAIR><<<grid, 64 * ks, ks > 1 ? ks * CT * RF * 1024 : 0, st>>>(a, wa);
}

}  // namespace moelora
