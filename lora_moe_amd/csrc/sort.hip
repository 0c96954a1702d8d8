// Tokens sorted by expert and back, with the gradients of both, and the
// gradient of the router's logits.  Contracts: include/moe_lora.h.
//
//   sort       row(t, j) = off[e] + #{pairs before (t, j) with expert e},  rows[row(t, j)] = x[t]
//   its grad   dx[t] = sum_j drows[row(t, j)]
//   unsort     y[t] = sum_j w[t][j] rows[row(t, j)]
//   its grad   drows[row(t, j)] = w[t][j] dy[t],  dw[t][j] = <dy[t], rows[row(t, j)]>
//   router     dlogits[t][e_j] = w_j (dw_j - sum_i w_i dw_i), 0 elsewhere
//
// All of it is bound by the rows' way through memory.  The sort reads a
// token's row once and writes it topk times, so that what is left is the order
// of the pairs: a stable counting sort whose counts are integers (LDS atomics,
// the same whatever their order).  8192 tokens of 7168 bf16 values, top-8: sort
// 228 us at 4.7 TB/s and 13 for the order, back 177 at 6.0; 4096 tokens of 2048
// fp32 values: 64 (4.9 TB/s) and 10, 54 (5.5), gradient 126 (4.8).  A large copy
// reaches 4.4 to 4.9.  1001 tokens of 2880 fp16 values, top-4: 11, 7 and 13
// us, a third of them a kernel's start and first trip.
#include <algorithm>

#include "abi_util.h"
#include "element.h"
#include "sort_util.h"

namespace moelora {

namespace {

constexpr int kThreads = 256;
constexpr int32_t kMaxTokens = 1 << 25, kMaxWidth = 1 << 20, kMaxTopk = 64;
// Up to this many pairs every workgroup counts all of them for itself, in one
// launch; beyond it a first launch counts chunks and a second adds them up.
constexpr int64_t kRecount = 8192;
constexpr int kRecountGroups = 512;  // workgroups at most, two to a CU
constexpr int kChunks = 2048;        // chunks at most

struct SortArgs {
  const int32_t* ids;  // [T][k]
  int T, k, E;
  int tokens;          // of a workgroup (a chunk)
  int chunks;
  int32_t* table;      // [E][chunks] counts, then exclusive prefixes
  int32_t* totals;     // [E]
  const u32x4_t* x;    // [T][pieces] 16-byte pieces, or NULL (the order only)
  u32x4_t* rows;       // [T k][pieces]
  int pieces;
  int32_t* off;         // [E + 1]
  int32_t* row_of_pair; // [T][k]
  int32_t* pair_of_row; // [T k] or NULL
};

__device__ __forceinline__ int expert_of(const SortArgs& p, int64_t pair) {
  const int e = p.ids[pair];
  return e >= 0 && e < p.E ? e : -1;
}

// counts of one chunk
__global__ __launch_bounds__(kThreads) void sort_count_kernel(SortArgs p) {
  extern __shared__ int hist[];  // [E]
  for (int e = threadIdx.x; e < p.E; e += kThreads) hist[e] = 0;
  lds_barrier();
  const int64_t p0 = (int64_t)blockIdx.x * p.tokens * p.k;
  const int64_t p1 = min(p0 + (int64_t)p.tokens * p.k, (int64_t)p.T * p.k);
  for (int64_t i = p0 + threadIdx.x; i < p1; i += kThreads) {
    const int e = expert_of(p, i);
    if (e >= 0) atomicAdd(&hist[e], 1);
  }
  lds_barrier();
  for (int e = threadIdx.x; e < p.E; e += kThreads) p.table[(int64_t)e * p.chunks + blockIdx.x] = hist[e];
}

// one workgroup per expert: its counts to exclusive prefixes, and their total
// (at most kChunks of them, kChunks / kThreads neighbouring ones a thread)
__global__ __launch_bounds__(kThreads) void sort_scan_kernel(SortArgs p) {
  constexpr int PER = kChunks / kThreads;
  __shared__ int scan[16];
  const int e = blockIdx.x, c0 = threadIdx.x * PER;
  int32_t* row = p.table + (int64_t)e * p.chunks;
  int v[PER], mine = 0, all;
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = c0 + i < p.chunks ? row[c0 + i] : 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) mine += v[i];
  int at = block_exclusive_scan<true>(mine, scan, &all);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (c0 + i < p.chunks) row[c0 + i] = at;
    at += v[i];
  }
  if (threadIdx.x == 0) p.totals[e] = all;
}

// The rows of a workgroup's tokens: pieces are loaded once, kAhead of them per
// thread in flight, and stored to the token's k rows (row < 0: a pair without an
// expert).
constexpr int kAhead = 4;
__device__ __forceinline__ void load_pieces(u32x4_t* q, const u32x4_t* src, int i0, int n) {
#pragma unroll
  for (int a = 0; a < kAhead; ++a)
    q[a] = __builtin_nontemporal_load(src + min(i0 + a * kThreads, n - 1));  // (past the last: that one again)
}
// q: the first ones, loaded already
__device__ __forceinline__ void copy_rows(const SortArgs& p, const u32x4_t* src, int n, const int* row, u32x4_t* q) {
  for (int i0 = threadIdx.x; i0 < n; i0 += kAhead * kThreads) {
    if (i0 >= kAhead * kThreads) load_pieces(q, src, i0, n);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + a * kThreads;
      if (i >= n) break;
      const int t = i / p.pieces, c = i - t * p.pieces;
      for (int j = 0; j < p.k; ++j) {
        const int r = row[t * p.k + j];
        if (r >= 0) __builtin_nontemporal_store(q[a], p.rows + (int64_t)r * p.pieces + c);
      }
    }
  }
}

// Places a workgroup's pairs and copies its tokens' rows.  LARGE: the counts
// come from the table, else they are counted here.
template <bool LARGE>
__global__ __launch_bounds__(kThreads) void sort_place_kernel(SortArgs p) {
  extern __shared__ __attribute__((aligned(16))) int lds[];
  int* wkeys = lds;                // [kThreads]
  int* rows = wkeys + kThreads;    // [kThreads]
  int* scan = rows + kThreads;     // [16]
  int* run = scan + 16;            // [E] next row of each expert
  int* total = run + p.E;          // [E]
  const int tid = threadIdx.x;
  const int first = blockIdx.x * p.tokens, last = min(first + p.tokens, p.T);
  const int step = kThreads / p.k;  // tokens at a time
  // the first rows are on their way while the pairs are counted
  u32x4_t q[kAhead];
  const int ahead = p.x ? max(0, min(step, last - first)) * p.pieces : 0;
  if (ahead) load_pieces(q, p.x + (int64_t)first * p.pieces, threadIdx.x, ahead);
  if (LARGE) {
    for (int e = tid; e < p.E; e += kThreads) {
      run[e] = p.table[(int64_t)e * p.chunks + blockIdx.x];
      total[e] = p.totals[e];
    }
  } else {
    for (int e = tid; e < p.E; e += kThreads) run[e] = total[e] = 0;
    lds_barrier();
    const int before = first * p.k, all = p.T * p.k;
    constexpr int AHEAD = 8;  // ids of a thread in flight
    for (int i0 = tid; i0 < all; i0 += AHEAD * kThreads) {
      int e[AHEAD];
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) e[q] = i0 + q * kThreads < all ? p.ids[i0 + q * kThreads] : -1;
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        if (e[q] < 0 || e[q] >= p.E) continue;
        atomicAdd(&total[e[q]], 1);
        if (i0 + q * kThreads < before) atomicAdd(&run[e[q]], 1);
      }
    }
  }
  lds_barrier();
  add_run_starts(run, total, p.E, scan, blockIdx.x == 0 ? p.off : nullptr);

  for (int t0 = first; t0 < last; t0 += step) {
    const int n = min(step, last - t0), pairs = n * p.k;
    const u32x4_t* src = p.x + (int64_t)t0 * p.pieces;
    if (t0 > first && p.x) load_pieces(q, src, tid, n * p.pieces);
    const int64_t pair = (int64_t)t0 * p.k + tid;
    const int e = tid < pairs ? expert_of(p, pair) : -1;
    const int r = ordered_rank(e, run, (pairs + 63) >> 6, wkeys);
    rows[tid] = e >= 0 ? r : -1;
    if (tid < pairs) p.row_of_pair[pair] = e >= 0 ? r : -1;
    if (e >= 0 && p.pair_of_row) p.pair_of_row[r] = (int32_t)pair;
    lds_barrier();
    if (p.x) copy_rows(p, src, n * p.pieces, rows, q);
    lds_barrier();
  }
}

// ---- back

struct BackArgs {
  const u32x4_t* rows;   // [T k][pieces]
  const u32x4_t* dy;     // backward: [T][pieces]
  const int32_t* row;    // [T][k]
  const float* w;        // [T][k], or NULL: ones
  u32x4_t* out;          // y [T][pieces]; backward: drows or NULL
  float* dw;             // backward: [T][k] or NULL
  int T, k, pieces;
};

// row of a pair, -1 where the caller's table holds none
__device__ __forceinline__ int row_of(const BackArgs& p, int64_t pair) {
  const int r = p.row[pair];
  return r >= 0 && r < p.T * p.k ? r : -1;
}

// One thread sums 16 bytes of a token over its pairs, in their order.  K: the
// pairs of a token, all their loads in flight together; 0: any number, four at
// a time.
template <int DT, int K>
__global__ __launch_bounds__(kThreads) void unsort_kernel(BackArgs p) {
  typedef Elements<DT> X;
  constexpr int STEP = K ? K : 4;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (int64_t)p.T * p.pieces) return;
  const int t = (int)(i / p.pieces), c = (int)(i - (int64_t)t * p.pieces);
  const int k = K ? K : p.k;
  float s[X::N];
#pragma unroll
  for (int n = 0; n < X::N; ++n) s[n] = 0.f;
  for (int j0 = 0; j0 < k; j0 += STEP) {
    u32x4_t q[STEP];
    int r[STEP];
    float w[STEP];
#pragma unroll
    for (int j = 0; j < STEP; ++j) {
      const bool has = j0 + j < k;
      r[j] = has ? row_of(p, (int64_t)t * k + j0 + j) : -1;
      w[j] = r[j] >= 0 && p.w ? p.w[(int64_t)t * k + j0 + j] : 1.f;
    }
    // a dropped pair loads row 0 and adds zeros: without branches the loads go
    // out together (and in 32 bits 8 pairs take 46 registers, not 238)
#pragma unroll
    for (int j = 0; j < STEP; ++j) q[j] = __builtin_nontemporal_load(p.rows + (int64_t)max(r[j], 0) * p.pieces + c);
#pragma unroll
    for (int j = 0; j < STEP; ++j) {
      float v[X::N];
      X::load(q[j], v);
#pragma unroll
      for (int n = 0; n < X::N; ++n) s[n] = fmaf(w[j], r[j] >= 0 ? v[n] : 0.f, s[n]);
    }
  }
  p.out[i] = X::store(s);
}

// A token's pairs on WAVES wavefronts of a workgroup: dy's pieces are loaded
// once for all pairs, STEP pairs at a time.
template <int DT, int WAVES>
__global__ __launch_bounds__(kThreads) void unsort_backward_kernel(BackArgs p) {
  typedef Elements<DT> X;
  constexpr int STEP = 4, TOKENS = kThreads / 64 / WAVES;
  __shared__ float part[kThreads / 64][STEP];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * TOKENS + wave / WAVES;
  const bool real = t < p.T;
  const int at = wave % WAVES * 64 + lane;
  for (int j0 = 0; j0 < p.k; j0 += STEP) {
    int r[STEP];
    float w[STEP], dot[STEP];
#pragma unroll
    for (int j = 0; j < STEP; ++j) {
      const bool has = real && j0 + j < p.k;
      r[j] = has ? row_of(p, (int64_t)t * p.k + j0 + j) : -1;
      w[j] = has && p.w ? p.w[(int64_t)t * p.k + j0 + j] : 1.f;
      dot[j] = 0.f;
    }
    if (real) {
      for (int c = at; c < p.pieces; c += 64 * WAVES) {
        const u32x4_t qy = p.dy[(int64_t)t * p.pieces + c];
        u32x4_t q[STEP];
        if (p.dw) {
#pragma unroll
          for (int j = 0; j < STEP; ++j)
            q[j] = __builtin_nontemporal_load(p.rows + (int64_t)max(r[j], 0) * p.pieces + c);
        }
        float y[X::N], v[X::N];
        X::load(qy, y);
#pragma unroll
        for (int j = 0; j < STEP; ++j) {
          if (r[j] < 0) continue;
          if (p.out) {
#pragma unroll
            for (int n = 0; n < X::N; ++n) v[n] = w[j] * y[n];
            __builtin_nontemporal_store(X::store(v), p.out + (int64_t)r[j] * p.pieces + c);
          }
          if (p.dw) {
            // a piece's products in pairs, so that few sums follow one another
            X::load(q[j], v);
#pragma unroll
            for (int n = 0; n < X::N; n += 2) v[n] = fmaf(y[n + 1], v[n + 1], y[n] * v[n]);
#pragma unroll
            for (int h = 2; h < X::N; h *= 2)
#pragma unroll
              for (int n = 0; n < X::N; n += 2 * h) v[n] += v[n + h];
            dot[j] += v[0];
          }
        }
      }
    }
    if (!p.dw) continue;
#pragma unroll
    for (int j = 0; j < STEP; ++j) {
#pragma unroll
      for (int o = 32; o; o >>= 1) dot[j] += __shfl_xor(dot[j], o, 64);
    }
    if (WAVES > 1) {
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < STEP; ++j) part[wave][j] = dot[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < STEP; ++j) {
        dot[j] = part[wave - wave % WAVES][j];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) dot[j] += part[wave - wave % WAVES + v][j];
      }
      __syncthreads();
    }
    if (real && at == 0) {
#pragma unroll
      for (int j = 0; j < STEP; ++j)
        if (j0 + j < p.k) p.dw[(int64_t)t * p.k + j0 + j] = r[j] >= 0 ? dot[j] : 0.f;
    }
  }
}

// ---- router

// P lanes write P V logits' gradients of one token: lane j brings pair j, so that
// a wavefront reads each of the three arrays once, and hands it to the others (8192
// tokens, 256 experts, top-8: 5.8 us, 8.5 where every lane reads all pairs; the
// 8.4 MB of logits would take 2, launch and first trip the rest).  A slot without
// an expert takes no part.
template <int V>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ w,
                                                                  const float* __restrict__ dw, int T, int E, int k,
                                                                  int P, int chunks, float* __restrict__ dlogits) {
  const int64_t group = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / P;
  const int lane = threadIdx.x & (P - 1);
  const int64_t t = chunks == 1 ? group : group / chunks;
  const int e0 = ((int)(group - t * chunks) * P + lane) * V;  // (below E + 64 V)
  int e = -1;
  float mine = 0.f, g = 0.f;
  if (t < T && lane < k) {  // (on their way together, an expert or not)
    e = ids[t * k + lane];
    mine = w[t * k + lane];
    g = dw[t * k + lane];
  }
  const bool has = e >= 0 && e < E;
  float sum = has ? mine * g : 0.f;
  for (int o = 1; o < P; o <<= 1) sum += __shfl_xor(sum, o, 64);
  g = has ? mine * (g - sum) : 0.f;
  if (!has) e = -1;
  float v[V];
#pragma unroll
  for (int q = 0; q < V; ++q) v[q] = 0.f;
  for (int j = 0; j < k; ++j) {
    const int at = __shfl(e, j, P) - e0;
    const float of = __shfl(g, j, P);
#pragma unroll
    for (int q = 0; q < V; ++q)
      if (at == q) v[q] += of;
  }
  if (t >= T || e0 >= E) return;
  float* out = dlogits + t * E + e0;
  if constexpr (V == 4) *reinterpret_cast<f32x4_t*>(out) = f32x4_t{v[0], v[1], v[2], v[3]};
  else out[0] = v[0];
}

template <int V>
int launch_route_backward(const int32_t* ids, const float* w, const float* dw, int T, int E, int k, float* dlogits,
                          hipStream_t st) {
  int P = 1;
  while (P < 64 && (P < k || P * V < E)) P *= 2;
  const int chunks = (E + P * V - 1) / (P * V);
  const int64_t blocks = ((int64_t)T * chunks * P + kThreads - 1) / kThreads;
  if (blocks * kThreads > 0xffffffff) return MOE_LORA_EUNSUPPORTED;
  route_backward_kernel<V><<<(unsigned)blocks, kThreads, 0, st>>>(ids, w, dw, T, E, k, P, chunks, dlogits);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

// ---- host side

int check_shape(const moe_lora_sort_shape* s) {
  if (!s || s->T < 0 || s->H <= 0 || s->E <= 0 || s->topk <= 0 || s->topk > s->E || !is_element(s->dtype))
    return MOE_LORA_EINVAL;
  if (s->H % 8) return MOE_LORA_EALIGN;
  if (s->T > kMaxTokens || s->H > kMaxWidth || s->E > kSortKeys || s->topk > kMaxTopk ||
      (int64_t)s->T * s->topk >= (1LL << 31) - kThreads)
    return MOE_LORA_EUNSUPPORTED;
  return MOE_LORA_OK;
}

struct Sizes {  // bytes
  size_t pairs, x, rows;
  int pieces;
  explicit Sizes(const moe_lora_sort_shape& s) {
    const size_t row = (size_t)s.H * element_size(s.dtype);
    pairs = (size_t)s.T * s.topk * 4;
    x = row * s.T;
    rows = x * s.topk;
    pieces = (int)(row / 16);
  }
};

struct Plan {
  bool large;
  int tokens, chunks;
};

Plan plan(const moe_lora_sort_shape& s) {
  Plan r;
  const int64_t pairs = (int64_t)s.T * s.topk;
  r.large = pairs > kRecount;
  const int most = r.large ? kChunks : kRecountGroups;
  r.tokens = std::max(1, (s.T + most - 1) / most);
  r.chunks = std::max(1, (s.T + r.tokens - 1) / r.tokens);
  return r;
}

size_t table_bytes(const moe_lora_sort_shape& s) {
  const Plan r = plan(s);
  return r.large ? round256((size_t)s.E * r.chunks * 4) + round256((size_t)s.E * 4) : 256;
}

bool launched() { return hipGetLastError() == hipSuccess; }

unsigned blocks_of(int64_t n) { return (unsigned)((n + kThreads - 1) / kThreads); }

template <int DT>
void launch_unsort(const BackArgs& a, hipStream_t st) {
  const unsigned grid = blocks_of((int64_t)a.T * a.pieces);
  switch (a.k) {
    case 1: unsort_kernel<DT, 1><<<grid, kThreads, 0, st>>>(a); break;
    case 2: unsort_kernel<DT, 2><<<grid, kThreads, 0, st>>>(a); break;
    case 4: unsort_kernel<DT, 4><<<grid, kThreads, 0, st>>>(a); break;
    case 6: unsort_kernel<DT, 6><<<grid, kThreads, 0, st>>>(a); break;
    case 8: unsort_kernel<DT, 8><<<grid, kThreads, 0, st>>>(a); break;
    default: unsort_kernel<DT, 0><<<grid, kThreads, 0, st>>>(a);
  }
}

template <int DT>
void launch_unsort_backward(const BackArgs& a, hipStream_t st) {
  if (a.T <= 1024) unsort_backward_kernel<DT, 4><<<a.T, kThreads, 0, st>>>(a);
  else unsort_backward_kernel<DT, 1><<<(a.T + 3) / 4, kThreads, 0, st>>>(a);
}

int unsort(const moe_lora_sort_shape* s, const void* rows, const int32_t* row_of_pair, const float* w, void* y,
           void* stream) {
  const int rc = check_shape(s);
  if (rc) return rc;
  if (s->T == 0) return MOE_LORA_OK;
  if (!rows || !row_of_pair || !y) return MOE_LORA_EINVAL;
  if (!aligned16(rows) || !aligned16(row_of_pair) || !aligned16(w) || !aligned16(y)) return MOE_LORA_EALIGN;
  const Sizes z(*s);
  const Range in[] = {{rows, z.rows}, {row_of_pair, z.pairs}, {w, w ? z.pairs : 0}};
  const Range out[] = {{y, z.x}};
  if (any_overlap(in, 3, out, 1)) return MOE_LORA_EINVAL;
  if ((int64_t)s->T * z.pieces > (int64_t)kThreads * 0x7fffff) return MOE_LORA_EUNSUPPORTED;
  const BackArgs a{(const u32x4_t*)rows, nullptr, row_of_pair, w, (u32x4_t*)y, nullptr, s->T, s->topk, z.pieces};
  hipStream_t st = (hipStream_t)stream;
  if (s->dtype == MOE_LORA_F32) launch_unsort<MOE_LORA_F32>(a, st);
  else if (s->dtype == MOE_LORA_BF16) launch_unsort<MOE_LORA_BF16>(a, st);
  else launch_unsort<MOE_LORA_F16>(a, st);
  return launched() ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // namespace
}  // namespace moelora

using namespace moelora;

extern "C" {

size_t moe_lora_sort_workspace_bytes(const moe_lora_sort_shape* shape) {
  return check_shape(shape) ? 0 : table_bytes(*shape);
}

int moe_lora_sort(const moe_lora_sort_shape* shape, const int32_t* topk_ids, const void* x, void* workspace,
                  size_t ws_bytes, void* rows, int32_t* expert_off, int32_t* row_of_pair, int32_t* pair_of_row,
                  void* stream) {
  const int rc = check_shape(shape);
  if (rc) return rc;
  const size_t need = table_bytes(*shape);
  const Sizes z(*shape);
  if (!expert_off || (shape->T && (!topk_ids || !row_of_pair || !x != !rows))) return MOE_LORA_EINVAL;
  if (!workspace || ws_bytes < need) return MOE_LORA_EWORKSPACE;
  const void* ptrs[] = {topk_ids, x, workspace, rows, expert_off, row_of_pair, pair_of_row};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_LORA_EALIGN;
  const Range in[] = {{topk_ids, z.pairs}, {x, x ? z.x : 0}};
  const Range out[] = {{rows, rows ? z.rows : 0},
                       {expert_off, ((size_t)shape->E + 1) * 4},
                       {row_of_pair, z.pairs},
                       {pair_of_row, pair_of_row ? z.pairs : 0},
                       {workspace, need}};
  if (any_overlap(in, 2, out, 5)) return MOE_LORA_EINVAL;
  const Plan r = plan(*shape);
  SortArgs a = {};
  a.ids = topk_ids, a.T = shape->T, a.k = shape->topk, a.E = shape->E, a.tokens = r.tokens, a.chunks = r.chunks;
  a.table = (int32_t*)workspace;
  a.totals = (int32_t*)((char*)workspace + round256((size_t)shape->E * r.chunks * 4));
  a.x = (const u32x4_t*)x, a.rows = (u32x4_t*)rows, a.pieces = z.pieces;
  a.off = expert_off, a.row_of_pair = row_of_pair, a.pair_of_row = pair_of_row;
  hipStream_t st = (hipStream_t)stream;
  const int lds = (2 * kThreads + 16 + 2 * a.E) * 4;  // at most 35 KB
  if (!r.large) {
    sort_place_kernel<false><<<r.chunks, kThreads, lds, st>>>(a);
    return launched() ? MOE_LORA_OK : MOE_LORA_EHIP;
  }
  sort_count_kernel<<<r.chunks, kThreads, a.E * 4, st>>>(a);
  sort_scan_kernel<<<a.E, kThreads, 0, st>>>(a);
  sort_place_kernel<true><<<r.chunks, kThreads, lds, st>>>(a);
  return launched() ? MOE_LORA_OK : MOE_LORA_EHIP;
}

int moe_lora_sort_backward(const moe_lora_sort_shape* shape, const void* drows, const int32_t* row_of_pair, void* dx,
                           void* stream) {
  return unsort(shape, drows, row_of_pair, nullptr, dx, stream);
}

int moe_lora_unsort(const moe_lora_sort_shape* shape, const void* rows, const int32_t* row_of_pair,
                    const float* weights, void* y, void* stream) {
  return unsort(shape, rows, row_of_pair, weights, y, stream);
}

int moe_lora_unsort_backward(const moe_lora_sort_shape* shape, const void* dy, const void* rows,
                             const int32_t* row_of_pair, const float* weights, void* drows, float* dweights,
                             void* stream) {
  const int rc = check_shape(shape);
  if (rc) return rc;
  if (shape->T == 0) return MOE_LORA_OK;
  if (!dy || !row_of_pair || (!drows && !dweights) || (dweights && !rows)) return MOE_LORA_EINVAL;
  const void* ptrs[] = {dy, rows, row_of_pair, weights, drows, dweights};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_LORA_EALIGN;
  const Sizes z(*shape);
  const Range in[] = {{dy, z.x}, {rows, rows ? z.rows : 0}, {row_of_pair, z.pairs}, {weights, weights ? z.pairs : 0}};
  const Range out[] = {{drows, drows ? z.rows : 0}, {dweights, dweights ? z.pairs : 0}};
  if (any_overlap(in, 4, out, 2)) return MOE_LORA_EINVAL;
  const BackArgs a{(const u32x4_t*)rows, (const u32x4_t*)dy, row_of_pair, weights, (u32x4_t*)drows, dweights,
                   shape->T, shape->topk, z.pieces};
  hipStream_t st = (hipStream_t)stream;
  if (shape->dtype == MOE_LORA_F32) launch_unsort_backward<MOE_LORA_F32>(a, st);
  else if (shape->dtype == MOE_LORA_BF16) launch_unsort_backward<MOE_LORA_BF16>(a, st);
  else launch_unsort_backward<MOE_LORA_F16>(a, st);
  return launched() ? MOE_LORA_OK : MOE_LORA_EHIP;
}

int moe_lora_route_backward(const moe_lora_shape* shape, const int32_t* topk_ids, const float* topk_weights,
                            const float* dweights, float* dlogits, void* stream) {
  // (of the layer's sizes a router has these three)
  if (!shape || shape->T < 0 || shape->E <= 0 || shape->topk <= 0 || shape->topk > shape->E) return MOE_LORA_EINVAL;
  const int E = shape->E, k = shape->topk;
  const int64_t logits = (int64_t)shape->T * E;
  if (k > kMaxTopk || logits > (int64_t)kThreads * 0x7fffff) return MOE_LORA_EUNSUPPORTED;
  if (shape->T == 0) return MOE_LORA_OK;
  if (!topk_ids || !topk_weights || !dweights || !dlogits) return MOE_LORA_EINVAL;
  const void* ptrs[] = {topk_ids, topk_weights, dweights, dlogits};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_LORA_EALIGN;
  const size_t pairs = (size_t)shape->T * k * 4;
  const Range in[] = {{topk_ids, pairs}, {topk_weights, pairs}, {dweights, pairs}};
  const Range out[] = {{dlogits, (size_t)logits * 4}};
  if (any_overlap(in, 3, out, 1)) return MOE_LORA_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  const auto launch = E % 4 ? launch_route_backward<1> : launch_route_backward<4>;
  return launch(topk_ids, topk_weights, dweights, shape->T, E, k, dlogits, st);
}

}  // extern "C"
