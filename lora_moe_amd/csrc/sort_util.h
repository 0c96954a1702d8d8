// A stable counting sort inside a workgroup: ranks of equal keys in order, and
// the starts of their runs.  Barriers order LDS only; no thread reads global
// data that another of its workgroup wrote.
#pragma once

#include "device_util.h"

namespace moelora {

constexpr int kSortKeys = 4096;  // keys at most: their tables lie in LDS

// The place of each thread's key (>= 0) in its run: run[key] (LDS) is the next
// free place and moves on.  The wavefronts take turns, and inside one the
// lanes of a key follow each other, so places are in thread order.  wkeys:
// blockDim.x ints of LDS, 16-byte aligned; waves: wavefronts that hold keys.
// All threads call it; it ends with a barrier.
__device__ __forceinline__ int ordered_rank(int key, int* run, int waves, int* wkeys) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int* mine = wkeys + wave * 64;
  mine[lane] = key;  // a wavefront's LDS operations run in order
  int before = 0, all = 0;
#pragma unroll
  for (int j = 0; j < 64; j += 4) {
    const int4 q = *reinterpret_cast<const int4*>(mine + j);
    const int m[4] = {q.x == key, q.y == key, q.z == key, q.w == key};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      all += m[i];
      before += m[i] & (j + i < lane);
    }
  }
  int place = 0;
  for (int w = 0; w < waves; ++w) {
    if (wave == w && key >= 0) {
      const int at = run[key];  // every lane reads before the first of a key writes
      place = at + before;
      if (before == 0) run[key] = at + all;
    }
    lds_barrier();
  }
  return place;
}

// run[e] += sum of total[0..e), e < n, and the sums to off[0..n] (a workgroup
// that has one).  scan: 16 ints of LDS.  Starts and ends behind a barrier.
__device__ __forceinline__ void add_run_starts(int* run, const int* total, int n, int* scan, int32_t* off) {
  const int per = (n + (int)blockDim.x - 1) / (int)blockDim.x;
  const int e0 = min(n, (int)threadIdx.x * per), e1 = min(n, e0 + per);
  int mine = 0, all;
  for (int e = e0; e < e1; ++e) mine += total[e];
  int at = block_exclusive_scan<true>(mine, scan, &all);
  for (int e = e0; e < e1; ++e) {
    run[e] += at;
    if (off) off[e] = at;
    at += total[e];
  }
  if (off && threadIdx.x == 0) off[n] = all;
  lds_barrier();
}

}  // namespace moelora
