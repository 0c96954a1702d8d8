// The projection of a few tokens (decode): the weight stream of rows.h over
// the shared weights and the adapters' A as one matrix.
//
//   first launch   [y0 z'] = x [W; A_l of every adapter met]^T, fp32
//   second launch  y[t] = y0[t] + B_l (s_l z[t])
//
// A's rows lie like W's (k contiguous), so the adapters that the batch meets
// are further tiles of 16 weight rows behind W's.  They meet all tokens, which
// costs nothing beside reading them, and a token takes the columns of its own
// adapter.  An adapter is read once, however many tokens have it: its tiles
// are numbered by the first token that has it.  The second launch is one
// output per lane and token, in fp32, so nothing of one adapter can reach
// another's tokens.
#include "proj.h"
#include "rows_bf16.h"

namespace moelora {

namespace {

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
  const float* slabs;  // [splits][T][cols]: W's columns, then each met adapter's
  int splits, cols, first, per;  // first: of the adapters' columns, per: of one adapter
  float* z;
  uint16_t* y;
};

// Grid: 512 outputs, two a thread; tokens.
__global__ __launch_bounds__(256) void proj_rows_join_kernel(JoinArgs a) {
  __shared__ float zs[128];
  const ProjArgs& p = a.p;
  const int t = blockIdx.y, tid = threadIdx.x, r = p.r;
  const Met met(p.ids, p.T, p.L, tid & 63);
  const int l = __builtin_amdgcn_readlane(met.id, t);
  const float* mine = a.slabs + (int64_t)t * a.cols;
  const int64_t slab = (int64_t)p.T * a.cols;
  // this token's z: its adapter's place among those met is that of the first
  // token that has it
  const int owner = __builtin_ctzll(__ballot(met.id == l));
  const int place = __popcll(met.first & ((1ull << owner) - 1));
  if (tid < r) {
    float v = 0.f;
    if (l >= 0)
      for (int s = 0; s < a.splits; ++s) v += mine[s * slab + a.first + place * a.per + tid];
    if (a.z && blockIdx.x == 0) a.z[(int64_t)t * r + tid] = v;
    if (l >= 0) zs[tid] = proj_scale(p, l) * v;
  }
  __syncthreads();
  const int n = ((int)blockIdx.x * 256 + tid) * 2;
  if (n >= p.N) return;
  float v[2] = {0.f, 0.f};
  for (int s = 0; s < a.splits; ++s) {
    const float2 q = *reinterpret_cast<const float2*>(mine + s * slab + n);
    v[0] += q.x;
    v[1] += q.y;
  }
  if (l >= 0) {
    const uint16_t* b = a.B + ((int64_t)l * p.N + n) * r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float d = 0.f;
      for (int j = 0; j < r; j += 8) {
        const u32x4_t q = ld16(b + h * r + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d = fmaf(zs[j + 2 * i], bf16_lo(q[i]), d);
          d = fmaf(zs[j + 2 * i + 1], bf16_hi(q[i]), d);
        }
      }
      v[h] += d;
    }
  }
  *reinterpret_cast<uint32_t*>(a.y + (int64_t)t * p.N + n) = f32x2_to_bf16(v[0], v[1]);
}

struct Columns {
  int base, per, all;  // tiles of W, of an adapter, of everything
  Columns(int T, int N, int L, int r) : base((N + 15) / 16), per((r + 15) / 16), all(base + std::min(T, L) * per) {}
};

}  // namespace

size_t proj_rows_slab_bytes(int T, int K, int N, int L, int r) {
  const Columns c(T, N, L, r);
  const RowsPlan f = rows_plan(T, c.all * 16, K, Bf16Stream::LINES);
  return (size_t)f.splits * T * c.all * 16 * sizeof(float);
}

int launch_proj_rows(const ProjArgs& p, const uint16_t* x, const uint16_t* W, const uint16_t* A, const uint16_t* B,
                     float* z, float* slabs, uint16_t* y, hipStream_t st) {
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
  const JoinArgs j{p, B, slabs, f.splits, c.all * 16, c.base * 16, c.per * 16, z, y};
  proj_rows_join_kernel<<<dim3((p.N + 511) / 512, p.T), 256, 0, st>>>(j);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // namespace moelora
