// The order of a batch's tokens by adapter, and the pieces of its runs.
//
// One launch: every workgroup counts all tokens' adapters for itself (the ids
// are a few KB in the L2 cache, and integer counts do not depend on the order
// of the LDS atomics), then places its own 256 tokens.  The first workgroup
// writes the runs' tables as well.  What bounds it is the chain of its steps
// (ids, counts, scans, ranks, tables), one after another: 7 to 8 us with 130 to
// 1001 tokens, 10 with 8192 of 32 workgroups, at a few hundred KB in and out.
#include "proj.h"
#include "sort_util.h"

namespace moelora {

namespace {

constexpr int kThreads = 1024, kTokens = 256;  // of a workgroup; the tokens that it places

// ids outside [0, L) have no adapter
__device__ __forceinline__ int key_of(int l, int L) { return l >= 0 && l < L ? l : L; }

// Counts the lanes' keys (< 0: none) into total, those with `early` into next
// too.  A run of tokens has one adapter: lanes with the same key as the first
// that is left are counted together, a few times, and only the rest one by
// one (atomics on one address follow each other).
__device__ __forceinline__ void count_keys(int key, bool early, int* total, int* next) {
  const int lane = threadIdx.x & 63;
  uint64_t left = __ballot(key >= 0);
  const uint64_t before = __ballot(early);
#pragma unroll 1
  for (int i = 0; i < 4 && left; ++i) {
    const int first = __builtin_ctzll(left), k = __builtin_amdgcn_readlane(key, first);
    const uint64_t same = __ballot(key == k);
    if (lane == first) {
      atomicAdd(&total[k], __popcll(same));
      if (same & before) atomicAdd(&next[k], __popcll(same & before));
    }
    left &= ~same;
  }
  if (left >> lane & 1) {
    atomicAdd(&total[key], 1);
    if (early) atomicAdd(&next[key], 1);
  }
}

// Exclusive scan over the keys of f(key), to g(key, sum before), by one
// wavefront; returns the whole sum.
template <class F, class G>
__device__ __forceinline__ int scan_keys(int n, F&& f, G&& g) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < n; e0 += 64) {
    const int e = e0 + lane, v = e < n ? f(e) : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(x, o, 64);
      if (lane >= o) x += y;
    }
    if (e < n) g(e, before + x - v);
    before += __shfl(x, 63, 64);
  }
  return before;
}

__device__ __forceinline__ int pieces(int n, int rows) { return (n + rows - 1) / rows; }

__global__ __launch_bounds__(kThreads) void proj_order_kernel(ProjArgs p, float* z, const float* kept, uint16_t* zs) {
  extern __shared__ __attribute__((aligned(16))) int lds[];
  const int S = p.L + 1;
  int* wkeys = lds;               // [kThreads]
  int* place = wkeys + kThreads;  // [kTokens]
  int* keys = place + kTokens;    // [kTokens]
  int* next = keys + kTokens;     // [S] next row of each key
  int* total = next + S;          // [S]
  int* first = total + S;         // [S] first row, and how many runs, pieces and slabs lie before the key's
  int* runs = first + S;          // [S]
  int* shrink = runs + S;         // [S]
  int* grad = shrink + S;         // [S]
  int* slab = grad + S;           // [S]
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * kTokens, mine = min(kTokens, p.T - t0);
  for (int e = tid; e < S; e += kThreads) next[e] = total[e] = 0;
  lds_barrier();
  constexpr int AHEAD = 8;  // ids of a thread in flight
  for (int base = 0; base < p.T; base += AHEAD * kThreads) {
    int id[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int t = base + i * kThreads + tid;
      id[i] = t < p.T ? p.ids[t] : 0;
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int t = base + i * kThreads + tid;
      if (t - (tid & 63) < p.T) count_keys(t < p.T ? key_of(id[i], p.L) : -1, t < t0, total, next);
    }
  }
  lds_barrier();
  // The tables, a wavefront each; the first workgroup writes what belongs to
  // no token.
  const int wave = tid >> 6;
  const bool writes = blockIdx.x == 0, counts = writes && (tid & 63) == 0;
  const ProjOrder& o = p.o;
  if (wave == 0) {
    scan_keys(S, [&](int e) { return total[e]; }, [&](int e, int at) {
      first[e] = at;
      next[e] += at;
    });
  } else if (wave == 1) {
    const int n = scan_keys(S, [&](int e) { return (int)(total[e] > 0); }, [&](int e, int at) {
      runs[e] = at;
      if (writes && total[e]) o.adapter[at] = e;
    });
    if (counts) o.count[2] = n - (total[p.L] > 0);
  } else if (wave == 2) {
    const int n = scan_keys(p.L, [&](int e) { return pieces(total[e], p.shrink_rows); },
                            [&](int e, int at) { shrink[e] = at; });
    if (counts) o.count[0] = n;
  } else if (wave == 3 && p.grad_rows) {
    // an adapter without tokens has an empty piece, whose gradients are zeros
    const int n = scan_keys(p.L, [&](int e) { return max(1, pieces(total[e], p.grad_rows)); }, [&](int e, int at) {
      grad[e] = at;
      if (writes && !total[e]) o.grad[at] = ProjItem{e, 0, 0, -1};
    });
    if (counts) o.count[1] = n;
  } else if (wave == 4 && p.grad_rows) {
    auto slabs_of = [&](int e) { return total[e] > p.grad_rows ? pieces(total[e], p.grad_rows) : 0; };
    scan_keys(p.L, slabs_of, [&](int e, int at) {
      slab[e] = at;
      if (!writes) return;
      o.slabs[2 * e] = at;
      o.slabs[2 * e + 1] = slabs_of(e);
    });
  }
  lds_barrier();
  const int key = tid < mine ? key_of(p.ids[t0 + tid], p.L) : -1;
  const int row = ordered_rank(key, next, (mine + 63) >> 6, wkeys);
  if (key >= 0) {
    place[tid] = row;
    keys[tid] = key;
    o.perm[row] = t0 + tid;
    o.run[row] = runs[key];
    if (key < p.L) {  // a piece is written by its first row's token
      const int at = row - first[key], left = total[key] - at;
      if (at % p.shrink_rows == 0)
        o.shrink[shrink[key] + at / p.shrink_rows] = ProjItem{key, row, min(p.shrink_rows, left), -1};
      if (p.grad_rows && at % p.grad_rows == 0) {
        const int i = at / p.grad_rows;
        o.grad[grad[key] + i] =
            ProjItem{key, row, min(p.grad_rows, left), total[key] > p.grad_rows ? slab[key] + i : -1};
      }
    }
  }
  if (!z && !zs) return;
  lds_barrier();
  const int per = p.r / 8;  // 8 values at a time
  for (int i = tid; i < mine * per; i += kThreads) {
    const int t = i / per, j = (i - t * per) * 8, l = keys[t];
    if (l == p.L) {
      if (z) {
        f32x4_t* to = reinterpret_cast<f32x4_t*>(z + (int64_t)(t0 + t) * p.r + j);
        to[0] = to[1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    } else if (zs) {
      const f32x4_t* from = reinterpret_cast<const f32x4_t*>(kept + (int64_t)(t0 + t) * p.r + j);
      const f32x4_t a = from[0], b = from[1];
      const float s = proj_scale(p, l);
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = s * (q < 4 ? a[q & 3] : b[q & 3]);
      store8_three(zs + (int64_t)place[t] * kParts * p.r + j, p.r, v);
    }
  }
}

}  // namespace

int launch_proj_order(const ProjArgs& p, float* z, const float* kept, uint16_t* zs, hipStream_t st) {
  const int lds = (kThreads + 2 * kTokens + 7 * (p.L + 1)) * 4;  // at most 62 KB
  proj_order_kernel<<<(p.T + kTokens - 1) / kTokens, kThreads, lds, st>>>(p, z, kept, zs);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // namespace moelora
