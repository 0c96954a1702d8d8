// The order of a batch's tokens by adapter, and the pieces of its runs.
//
// One launch: every workgroup counts all tokens' adapters for itself (the ids
// are a few KB in the L2 cache, and integer counts do not depend on the order
// of the LDS atomics), then places its own tokens.  The first workgroup writes
// the runs' tables as well.  8192 tokens, 8 adapters: 8 us.
#include "proj.h"
#include "sort_util.h"

namespace moelora {

namespace {

constexpr int kThreads = 256;

// ids outside [0, L) have no adapter
__device__ __forceinline__ int key_of(const ProjArgs& p, int t) {
  const int l = p.ids[t];
  return l >= 0 && l < p.L ? l : p.L;
}

// Exclusive scan over the keys of f(key), to g(key, sum before); returns the
// whole sum.  scan: 16 ints of LDS.
template <class F, class G>
__device__ __forceinline__ int scan_keys(int n, int* scan, F&& f, G&& g) {
  const int per = (n + kThreads - 1) / kThreads, e0 = min(n, (int)threadIdx.x * per), e1 = min(n, e0 + per);
  int mine = 0, all;
  for (int e = e0; e < e1; ++e) mine += f(e);
  int at = block_exclusive_scan<true>(mine, scan, &all);
  for (int e = e0; e < e1; ++e) {
    g(e, at);
    at += f(e);
  }
  return all;
}

__device__ __forceinline__ int pieces(int n, int rows) { return (n + rows - 1) / rows; }

__global__ __launch_bounds__(kThreads) void proj_order_kernel(ProjArgs p, float* z, const float* kept, uint16_t* zs) {
  extern __shared__ __attribute__((aligned(16))) int lds[];
  const int S = p.L + 1;
  int* wkeys = lds;               // [kThreads]
  int* place = wkeys + kThreads;  // [kThreads]
  int* keys = place + kThreads;   // [kThreads]
  int* scan = keys + kThreads;    // [16]
  int* next = scan + 16;          // [S] next row of each key
  int* total = next + S;          // [S]
  int* runs = total + S;          // [S] runs before the key's
  int* slab = runs + S;           // [S] slabs before the key's
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * kThreads, mine = min(kThreads, p.T - t0);
  for (int e = tid; e < S; e += kThreads) next[e] = total[e] = 0;
  lds_barrier();
  for (int t = tid; t < p.T; t += kThreads) {
    const int e = key_of(p, t);
    atomicAdd(&total[e], 1);
    if (t < t0) atomicAdd(&next[e], 1);
  }
  lds_barrier();
  scan_keys(S, scan, [&](int e) { return (int)(total[e] > 0); }, [&](int e, int at) { runs[e] = at; });
  scan_keys(S, scan, [&](int e) { return total[e]; }, [&](int e, int at) { next[e] += at; });
  lds_barrier();
  if (blockIdx.x == 0) {
    // (nothing lies before this workgroup's tokens: next is a run's first row)
    const ProjOrder& o = p.o;
    for (int e = tid; e < S; e += kThreads)
      if (total[e]) o.adapter[runs[e]] = e;
    const int ns = scan_keys(p.L, scan, [&](int e) { return pieces(total[e], p.shrink_rows); },
                             [&](int e, int at) {
                               for (int i = 0; i < total[e]; i += p.shrink_rows)
                                 o.shrink[at++] = ProjItem{e, next[e] + i, min(p.shrink_rows, total[e] - i), -1};
                             });
    int ng = 0;
    if (p.grad_rows) {
      auto slabs_of = [&](int e) { return total[e] > p.grad_rows ? pieces(total[e], p.grad_rows) : 0; };
      scan_keys(p.L, scan, slabs_of, [&](int e, int at) {
        slab[e] = at;
        o.slabs[2 * e] = at;
        o.slabs[2 * e + 1] = total[e] ? slabs_of(e) : -1;
      });
      // (a thread meets the same keys in every scan)
      ng = scan_keys(p.L, scan, [&](int e) { return pieces(total[e], p.grad_rows); },
                     [&](int e, int at) {
                       const bool split = total[e] > p.grad_rows;
                       for (int i = 0, s = slab[e]; i < total[e]; i += p.grad_rows, ++s)
                         o.grad[at++] = ProjItem{e, next[e] + i, min(p.grad_rows, total[e] - i), split ? s : -1};
                     });
    }
    if (tid == 0) {
      o.count[0] = ns;
      o.count[1] = ng;
      o.count[2] = runs[p.L];
    }
    lds_barrier();  // before the tokens below move next
  }
  const int key = tid < mine ? key_of(p, t0 + tid) : -1;
  const int row = ordered_rank(key, next, (mine + 63) >> 6, wkeys);
  place[tid] = row;
  keys[tid] = key;
  if (key >= 0) {
    p.o.perm[row] = t0 + tid;
    p.o.run[row] = runs[key];
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
      uint16_t* to = zs + (int64_t)place[t] * 2 * p.r + j;
      store8_pair(to, to + p.r, v);
    }
  }
}

}  // namespace

int launch_proj_order(const ProjArgs& p, float* z, const float* kept, uint16_t* zs, hipStream_t st) {
  const int lds = (3 * kThreads + 16 + 4 * (p.L + 1)) * 4;  // at most 36 KB
  proj_order_kernel<<<(p.T + kThreads - 1) / kThreads, kThreads, lds, st>>>(p, z, kept, zs);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // namespace moelora
