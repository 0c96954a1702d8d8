// The projection of a decode batch: the shared weights and the adapters' A as
// one matrix.
//
//   first launch   [y0 z'] = x [W; A]^T, fp32
//   second launch  y[t] = y0[t] + B_l (s_l z[t])
//
// A's rows lie like W's (k contiguous), so they are further columns behind
// W's.  They meet all tokens, and a token takes the columns of its own adapter.
// Up to 32 tokens this is the weight stream of rows.h: the adapters that the
// batch meets are further tiles of 16 weight rows, read once however many
// tokens have them (their tiles are numbered by the first token that has one),
// and meeting all tokens costs nothing beside reading them.  Beyond it is a
// tiled product (proj_gemm.hip) with all adapters' A.  The second launch works
// on single outputs in fp32, so nothing of one adapter can reach another's
// tokens.
#include "proj.h"
#include "rows_bf16.h"

namespace moelora {

namespace {

// products of tokens, outputs and rank in the second launch (see proj_few)
constexpr int64_t kProjFew = 1 << 25;

// The batch's adapters, a lane a token: id of the lane's token (-1: none), and
// a bit for the first token of each adapter.
struct Met {
  int id;
  uint64_t first;
  __device__ __forceinline__ Met(const int32_t* ids, int T, int L, int lane) {
    id = lane < T ? ids[lane] : -1;
    if (id >= L) id = -1;
    bool is_first = id >= 0;
    for (int j = 0; j + 1 < T; ++j)
      if (j < lane && __builtin_amdgcn_readlane(id, j) == id) is_first = false;
    first = __ballot(is_first);
  }
};

struct ProjWeights : Bf16Stream {
  struct Args {
    const uint16_t* w;  // [N][K]
    const uint16_t* a;  // [L][r][K]
    const int32_t* ids;
    int T, N, L, r;
    int base, per;      // tiles of W, tiles of an adapter
  };
  static constexpr bool RAW = true;
  const Args& a;
  int lane;
  __device__ __forceinline__ ProjWeights(const Args& a_, int, int K_, int lane_)
      : Bf16Stream(K_, lane_), a(a_), lane(lane_) {}
  // rows past N or r lie past the tile's bytes, and so does all of a tile
  // behind the last adapter met
  __device__ __forceinline__ Tile tile(int t, int) const {
    if (t < a.base) {
      const int rows = max(min(16, a.N - t * 16), 0);
      return Tile{a.w + (int64_t)t * 16 * K, (uint32_t)rows * (uint32_t)K * 2u};
    }
    const int n = (t - a.base) / a.per, part = (t - a.base) - n * a.per;
    const Met met(a.ids, a.T, a.L, lane);
    uint64_t left = met.first;
    for (int i = 0; i < n; ++i) left &= left - 1;
    if (!left) return Tile{a.a, 0u};
    const int l = __builtin_amdgcn_readlane(met.id, __builtin_ctzll(left));
    const int rows = min(16, a.r - part * 16);
    return Tile{a.a + ((int64_t)l * a.r + part * 16) * K, (uint32_t)rows * (uint32_t)K * 2u};
  }
};

struct JoinArgs {
  ProjArgs p;
  const uint16_t* B;
  const float* slabs;  // [splits][T][cols]: W's columns, then adapters'
  int splits, cols, first, per;  // first: of the adapters' columns, per: of one adapter
  float* z;
  uint16_t* y;
};

// y and z from the first launch's sums.  Grid: 256 outputs; tokens.  G lanes
// (r / 8 of them with 8 ranks each) share an output's row of B and take G
// outputs in turn, so that a wavefront reads its 64 outputs' rows as whole
// lines, before z is there (32 tokens, 11008 outputs, rank 32: XX us so, 9.4
// with a lane an output, whose lines drop out of the L1 cache between their
// pieces).  MET: the adapters' columns are those met by at most 64 tokens, else
// all adapters'.
template <int G, bool MET>
__global__ __launch_bounds__(256) void proj_rows_join_kernel(JoinArgs a) {
  __shared__ __attribute__((aligned(16))) float zs[128];
  const ProjArgs& p = a.p;
  const int t = blockIdx.y, tid = threadIdx.x, lane = tid & 63, r = p.r;
  int l, place;
  if constexpr (MET) {
    // an adapter's place among those met is that of the first token that has it
    const Met met(p.ids, p.T, p.L, lane);
    l = __builtin_amdgcn_readlane(met.id, t);
    const int owner = __builtin_ctzll(__ballot(met.id == l));
    place = __popcll(met.first & ((1ull << owner) - 1));
  } else {
    l = p.ids[t];
    if (l >= p.L) l = -1;
    place = l;
  }
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
      for (int s = 0; s < a.splits; ++s) d += sums[s * slab + a.first + place * a.per + tid];
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

template <bool MET>
void launch_join(const JoinArgs& j, hipStream_t st) {
  const int r = j.p.r;
  const dim3 grid((j.p.N + 255) / 256, j.p.T);
  if (r <= 8) proj_rows_join_kernel<1, MET><<<grid, 256, 0, st>>>(j);
  else if (r <= 16) proj_rows_join_kernel<2, MET><<<grid, 256, 0, st>>>(j);
  else if (r <= 32) proj_rows_join_kernel<4, MET><<<grid, 256, 0, st>>>(j);
  else if (r <= 64) proj_rows_join_kernel<8, MET><<<grid, 256, 0, st>>>(j);
  else proj_rows_join_kernel<16, MET><<<grid, 256, 0, st>>>(j);
}

struct Columns {
  int base, per, all;  // tiles of W, of an adapter, of everything
  Columns(int T, int N, int L, int r) : base((N + 15) / 16), per((r + 15) / 16), all(base + std::min(T, L) * per) {}
};

}  // namespace

bool proj_few(int T, int N, int L, int r) {
  return T <= kProjRows || (T <= 4096 && (int64_t)T * N * r <= kProjFew && 2 * (int64_t)L * r <= N);
}

size_t proj_rows_slab_bytes(const ProjArgs& p) {
  if (p.T > kProjRows) return (size_t)proj_both_splits(p) * p.T * (p.N + p.L * p.r) * sizeof(float);
  const Columns c(p.T, p.N, p.L, p.r);
  const RowsPlan f = rows_plan(p.T, c.all * 16, p.K, Bf16Stream::LINES);
  return (size_t)f.splits * p.T * c.all * 16 * sizeof(float);
}

int launch_proj_rows(const ProjArgs& p, const uint16_t* x, const uint16_t* W, const uint16_t* A, const uint16_t* B,
                     float* z, float* slabs, uint16_t* y, hipStream_t st) {
  if (p.T > kProjRows) {
    const int rc = launch_proj_both(p, x, W, A, slabs, st);
    if (rc) return rc;
    launch_join<false>(JoinArgs{p, B, slabs, proj_both_splits(p), p.N + p.L * p.r, p.N, p.r, z, y}, st);
    return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
  }
  const Columns c(p.T, p.N, p.L, p.r);
  const RowsPlan f = rows_plan(p.T, c.all * 16, p.K, Bf16Stream::LINES);
  RowsArgs a = {};
  a.x = x, a.M = p.T, a.N = c.all * 16, a.K = p.K, a.slabs = slabs, a.splits = f.splits, a.groups = f.groups;
  const ProjWeights::Args w{W, A, p.ids, p.T, p.N, p.L, p.r, c.base, c.per};
  if (f.direct) {
    if (p.T <= 4) launch_rows_direct<ProjWeights, 4, false, false>(a, w, st);
    else launch_rows_direct<ProjWeights, 8, false, false>(a, w, st);
  } else {
    const dim3 grid(f.groups, 1, f.splits);
    if (p.T <= 16) rows_shared_kernel<ProjWeights, 1, false, false><<<grid, 512, 0, st>>>(a, w);
    else rows_shared_kernel<ProjWeights, 2, false, false><<<grid, 512, 0, st>>>(a, w);
  }
  launch_join<true>(JoinArgs{p, B, slabs, f.splits, c.all * 16, c.base * 16, c.per * 16, z, y}, st);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // namespace moelora
