// Internal declarations of the shared projection with the adapters of many
// requests (proj.hip: ABI; proj_few.hip: decode batches; proj_order.hip,
// proj_shrink.hip, proj_gemm.hip, proj_grads.hip: the rest).  Not part of the
// public ABI.
//
// Beyond a few tokens everything works on rows, the tokens sorted by adapter:
// row m is token perm[m], the tokens of one adapter are one run, those without
// an adapter come last.  Only indices are sorted; x, dy, y and dx stay where
// they are and the kernels gather and scatter their rows.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_lora.h"

namespace moelora {

// Rows [row, row + n) of one adapter; slab: where a piece of a longer run puts
// its sums (-1: the run's only piece).
struct ProjItem {
  int adapter, row, n, slab;
};

// What proj_order.hip writes for the other kernels.
struct ProjOrder {
  int32_t* perm;       // [T] token of a row
  int32_t* run;        // [T] which run the row is in (runs with tokens, counted from 0)
  int32_t* adapter;    // [L + 1] adapter of a run; L: the tokens without
  int32_t* count;      // [4] shrink items, gradient items, runs with an adapter
  ProjItem* shrink;    // pieces of at most shrink_rows rows of the runs with an adapter
  ProjItem* grad;      // pieces of at most grad_rows rows, one at least of every adapter
  int32_t* slabs;      // [L][2] first slab of an adapter and how many (0: one piece)
};

struct ProjArgs {
  int T, K, N, L, r;
  float scale;
  const int32_t* ids;
  const float* scales;  // [L] or NULL
  ProjOrder o;
  int shrink_rows, grad_rows;
};

// Rows of a shrink's piece.
inline int proj_shrink_rows(int T, int r) { return T <= 4096 || r > 64 ? 16 : 32; }
// Pieces at most: whole ones, and a short one for each run.
inline int64_t proj_items(int T, int L, int rows) { return T / rows + (T < L ? T : L); }

// s_l
__device__ __forceinline__ float proj_scale(const ProjArgs& p, int l) {
  return p.scales ? p.scale * p.scales[l] : p.scale;
}

// Parts: [T rows][3r] bf16, a row's r values rounded, behind them what is left
// of each, rounded too, and behind those what is left then.  All three meet the
// same weights, and their sum is the fp32 value: sums down to the rank keep all
// of their bits on the way into the next product.  (The first two alone, 16
// bits, show in the gradients: 1.1e-4 of their norm from sums in fp32, where the
// order of sums makes 5e-5.  The third takes 2 us of 28 of a tile kernel with
// 1001 tokens, 2880 x 2880, rank 32, 5 of 228 with 8192, 4096 x 4096, rank 16.)
constexpr int kParts = 3;

// z (NULL: not wanted): zeros for the tokens without an adapter are written
// here; zs (backward; NULL else): parts of s_l z.
int launch_proj_order(const ProjArgs& p, float* z, const float* kept, uint16_t* zs, hipStream_t st);

// parts[m] = s_l * (weights of row m's adapter) in[perm[m]] and, on request,
// the product without s_l by token (z).  back: in = dy, weights = B [L][N][r];
// else in = x, weights = A [L][r][K].
int launch_proj_shrink(const ProjArgs& p, bool back, const uint16_t* in, const uint16_t* weights, uint16_t* parts,
                       float* z, hipStream_t st);

// out[perm[m]] = in[perm[m]] W^T + parts[m] weights^T; back: the same with W
// and the adapters' weights by their columns.
struct ProjGemm {
  const uint16_t* in;
  const uint16_t* W;
  const uint16_t* parts;
  const uint16_t* weights;
  uint16_t* out;
  float* slabs;
  int splits;
  int32_t* place;  // [64] of a token's adapter among those met (launch_proj_both)
};
size_t proj_gemm_slab_bytes(const ProjArgs& p, bool back);
// Its tile (0 to 4: 256 x 256, 128 x 128, the same in two groups, 64 x 128, 32 x
// 64) times 32 plus its K splits, for tests that have to meet all of them; and
// those of launch_proj_both.
int proj_gemm_plan(int T, int K, int N, int r, bool back);
int proj_both_plan(int T, int K, int N, int L, int r);
int launch_proj_gemm(const ProjArgs& p, bool back, ProjGemm g, hipStream_t st);

// dA and dB (either may be NULL)
struct ProjGrads {
  const uint16_t* x;
  const uint16_t* dy;
  const uint16_t* us;  // parts of u
  const uint16_t* zs;  // parts of s_l z
  uint16_t* dA;
  uint16_t* dB;
  float* slabs;
};
int proj_grad_rows(int T, int K, int N, int L, int r);
inline int64_t proj_grad_items(const ProjArgs& p) { return p.T / p.grad_rows + p.L; }
size_t proj_grad_slab_bytes(const ProjArgs& p);
int launch_proj_grads(const ProjArgs& p, const ProjGrads& g, hipStream_t st);

// x [W; A]^T, fp32, into slabs [proj_both_splits][T][N + proj_slots r]: of at most
// 64 tokens and more adapters those that are met (place: [64], which of them a
// token's is), else of all adapters, met or not: their A are L r columns beside N,
// no more than the tokens have at most.
int proj_slots(int T, int L);
int proj_both_splits(const ProjArgs& p);
int launch_proj_both(const ProjArgs& p, const uint16_t* x, const uint16_t* W, const uint16_t* A, float* slabs,
                     int32_t* place, hipStream_t st);

// Whether a forward takes the two launches of proj_few.hip, which need no order:
// decode batches, and more tokens where the adapters' A are few columns beside
// W's and the tokens' shares of B are little to read one by one.
bool proj_few(int T, int N, int L, int r);
size_t proj_few_slab_bytes(const ProjArgs& p);
int launch_proj_few(const ProjArgs& p, const uint16_t* x, const uint16_t* W, const uint16_t* A, const uint16_t* B,
                    float* z, float* scratch, uint16_t* y, hipStream_t st);

}  // namespace moelora
