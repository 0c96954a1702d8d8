// The projection of a decode batch: the shared weights and the adapters' A as
// one matrix.
//
//   first launch   [y0 z'] = x [W; A]^T, fp32 (proj_gemm.hip)
//   second launch  y[t] = y0[t] + B_l (s_l z[t])
//
// A's rows lie like W's (k contiguous), so they are further columns behind
// W's.  They meet all tokens, and a token takes the columns of its own adapter:
// no order is needed, and nothing waits for z.  The second launch adds the K
// splits up and works on single outputs in fp32, so nothing of one adapter can
// reach another's tokens.
//
// What bounds it: the weights' stream from memory at 4.1 TB/s (32 tokens, 4096 x
// 11008, rank 32: 24 us for 98 MB, and 6 for the second launch; weights that are
// in the cache already take 18 and 5.5); with a single token, 4096 x 4096, 10.6
// and 3.9 us, a kernel's start and first trip each.
#include <algorithm>

#include "device_util.h"
#include "proj.h"

namespace moelora {

namespace {

struct JoinArgs {
  ProjArgs p;
  const uint16_t* B;
  const float* slabs;     // [splits][T][cols]: W's columns, then r of each adapter
  int splits, cols;
  const int32_t* places;  // [T] of the tokens' adapters, or NULL: an adapter's place is its number
  float* z;
  uint16_t* y;
};

// y and z from the first launch's sums.  Grid: 256 outputs; tokens.  G lanes
// (r / 8 of them with 8 ranks each) share an output's row of B and take G
// outputs in turn, so that a wavefront reads its 64 outputs' rows as whole
// lines, and before z is there.  32 tokens, 11008 outputs, rank 32 (11 MB of B,
// a few of sums): 6.2 us, the chain of id, place, z and barrier most of it.
template <int G>
__global__ __launch_bounds__(256) void proj_few_join_kernel(JoinArgs a) {
  __shared__ __attribute__((aligned(16))) float zs[128];
  const ProjArgs& p = a.p;
  const int t = blockIdx.y, tid = threadIdx.x, lane = tid & 63, r = p.r;
  int l = p.ids[t];
  if (l >= p.L) l = -1;
  const int place = a.places ? a.places[t] : l;
  const int n0 = (int)blockIdx.x * 256 + (tid & ~63);  // the wavefront's first output
  const int part = lane % G, of = lane / G;            // output of + u 64 / G of load u
  const int n = n0 + part * (64 / G) + of;             // what is left with this lane
  const bool mine = part * 8 < r;
  u32x4_t b[G];
  if (l >= 0) {
#pragma unroll
    for (int u = 0; u < G; ++u) {
      const int o = n0 + u * (64 / G) + of;
      b[u] = zero4();
      if (mine && o < p.N) b[u] = ld16(a.B + ((int64_t)l * p.N + o) * r + part * 8);
    }
  }
  const float* sums = a.slabs + (int64_t)t * a.cols;
  const int64_t slab = (int64_t)p.T * a.cols;
  float v = 0.f;
  if (n < p.N)
    for (int s = 0; s < a.splits; ++s) v += sums[s * slab + n];
  if (tid < r) {
    float d = 0.f;
    if (l >= 0)
      for (int s = 0; s < a.splits; ++s) d += sums[s * slab + p.N + place * r + tid];
    if (a.z && blockIdx.x == 0) a.z[(int64_t)t * r + tid] = d;
    zs[tid] = l >= 0 ? proj_scale(p, l) * d : 0.f;
  }
  __syncthreads();
  if (l >= 0) {
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = mine ? zs[part * 8 + i] : 0.f;
    float d = 0.f;
#pragma unroll
    for (int u = 0; u < G; ++u) {
      float e = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e = fmaf(z[2 * i], bf16_lo(b[u][i]), e);
        e = fmaf(z[2 * i + 1], bf16_hi(b[u][i]), e);
      }
#pragma unroll
      for (int o = 1; o < G; o <<= 1) e += __shfl_xor(e, o, 64);
      if (part == u) d = e;
    }
    v += d;
  }
  if (n < p.N) a.y[(int64_t)t * p.N + n] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Products of tokens, outputs and rank in the second launch, at most, and tokens
// (those beyond take 16 KB of B's rows and more for a tile's worth of outputs).
// Measured, us, so and sorted, inputs from memory: 400 tokens, 2048 x 4096, rank
// 64 (105 M) 35 and 42; 256, 4096 x 11008, 32 (90 M) 61 and 73; 400, 4096 x 11008,
// 32 (141 M) 87 and 94, from the cache 84 and 80; 1001, 4096 x 4096, 16 (66 M) 76
// and 58; 100, 2880 x 2880, 16 (5 M) 14 and 30.
constexpr int64_t kProjFew = 96 << 20;
constexpr int kProjFewTokens = 512;

constexpr size_t kPlaces = 64 * sizeof(int32_t);

}  // namespace

bool proj_few(int T, int N, int L, int r) {
  return T <= 64 || (T <= kProjFewTokens && (int64_t)T * N * r <= kProjFew && 2 * (int64_t)L * r <= N);
}

size_t proj_few_slab_bytes(const ProjArgs& p) {
  return kPlaces + (size_t)proj_both_splits(p) * p.T * (p.N + proj_slots(p.T, p.L) * p.r) * sizeof(float);
}

int launch_proj_few(const ProjArgs& p, const uint16_t* x, const uint16_t* W, const uint16_t* A, const uint16_t* B,
                    float* z, float* scratch, uint16_t* y, hipStream_t st) {
  int32_t* places = (int32_t*)scratch;
  float* slabs = (float*)((char*)scratch + kPlaces);
  const int slots = proj_slots(p.T, p.L);
  const int rc = launch_proj_both(p, x, W, A, slabs, places, st);
  if (rc) return rc;
  const JoinArgs j{p, B, slabs, proj_both_splits(p), p.N + slots * p.r, slots < p.L ? places : nullptr, z, y};
  const dim3 grid((p.N + 255) / 256, p.T);
  if (p.r <= 8) proj_few_join_kernel<1><<<grid, 256, 0, st>>>(j);
  else if (p.r <= 16) proj_few_join_kernel<2><<<grid, 256, 0, st>>>(j);
  else if (p.r <= 32) proj_few_join_kernel<4><<<grid, 256, 0, st>>>(j);
  else if (p.r <= 64) proj_few_join_kernel<8><<<grid, 256, 0, st>>>(j);
  else proj_few_join_kernel<16><<<grid, 256, 0, st>>>(j);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // namespace moelora
