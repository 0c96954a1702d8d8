// Global gradient norm over many tensors, and clipping.  Contract:
// include/moe_lora.h.
//
//   norm = sqrt(sum over all tensors of sum g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = c * g
//
// Two passes, since no gradient can be scaled before the norm is known: the
// first writes one partial sum per workgroup, the second adds them up in
// every workgroup (in the same order, so c is the same everywhere and from
// run to run) and scales.  Both are bound by memory; the second goes through
// the chunks backwards, so that what the first read last is still in the 256
// MB cache beside the HBM.  Squares and sums are fp64: squares cannot overflow
// or vanish, and the order of addition does not show in fp32.
//
// Measured: 541 M bf16 gradients (1.08 GB) 181 us for the norm, 6.0 TB/s, and
// 420 for the second pass, 5.1 TB/s (1.08 GB read, as much written); 224
// tensors of 52 MB in all 13 and 20 us, half of it the launch, the table's
// search and the partial sums.
//
// The tensors' table travels in the kernel arguments, kTensors at a time, so
// nothing is kept between calls and a captured call holds its own copy.
#include <math.h>

#include <algorithm>
#include <new>

#include "abi_util.h"
#include "device_util.h"
#include "moe_lora.h"

namespace moelora {

namespace {

constexpr int kTensors = 256;      // per launch: 7.4 KB of kernel arguments
// elements one workgroup takes at a time: enough chunks to go round in a small
// call, whole batches of loads in a large one (540 M gradients: 577 us with
// 16384, 608 with 8192)
constexpr int kChunkMin = 2048, kChunkMax = 16384;
constexpr int kMaxParts = 2048;    // partial sums of one call, beyond one per launch
constexpr float kEps = 1e-6f;

struct Table {
  const void* g[kTensors];
  void* out[kTensors];
  int64_t numel[kTensors];
  int first[kTensors + 1];  // first chunk of each tensor
  uint8_t dtype[kTensors];
  int n, chunk;
};

__device__ __forceinline__ float f16_to_f32(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
__device__ __forceinline__ uint16_t f32_to_f16(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if (DT == MOE_LORA_F32) return static_cast<const float*>(p)[i];
  const uint16_t v = static_cast<const uint16_t*>(p)[i];
  return DT == MOE_LORA_BF16 ? bf16_to_f32(v) : f16_to_f32(v);
}

template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if (DT == MOE_LORA_F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = DT == MOE_LORA_BF16 ? f32_to_bf16(v) : f32_to_f16(v);
}

// 16 bytes of gradients as fp32
template <int DT>
struct Piece {
  static constexpr int N = DT == MOE_LORA_F32 ? 4 : 8;
  float v[N];
  __device__ __forceinline__ explicit Piece(u32x4_t q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == MOE_LORA_F32) {
        v[i] = __uint_as_float(q[i]);
      } else {
        v[2 * i % N] = DT == MOE_LORA_BF16 ? bf16_lo(q[i]) : f16_to_f32((uint16_t)q[i]);
        v[(2 * i + 1) % N] = DT == MOE_LORA_BF16 ? bf16_hi(q[i]) : f16_to_f32((uint16_t)(q[i] >> 16));
      }
    }
  }
  __device__ __forceinline__ double squares() const {
    double d = 0.;
#pragma unroll
    for (int i = 0; i < N; ++i) d = fma((double)v[i], (double)v[i], d);
    return d;
  }
  __device__ __forceinline__ u32x4_t scaled(float c) const {
    u32x4_t q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == MOE_LORA_F32) {
        q[i] = __float_as_uint(v[i] * c);
      } else {
        const float a = v[2 * i % N] * c, b = v[(2 * i + 1) % N] * c;
        q[i] = DT == MOE_LORA_BF16 ? f32x2_to_bf16(a, b)
                                   : f32_to_f16(a) | (uint32_t)f32_to_f16(b) << 16;
      }
    }
    return q;
  }
};

// the tensor that holds chunk c: the last whose first chunk is <= c (empty
// tensors share their first chunk with the next one)
__device__ __forceinline__ int tensor_of(const Table& t, int c) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return lds[0] + lds[1] + lds[2] + lds[3];
}

constexpr int kAhead = 8;  // 16-byte loads in flight per thread

template <int DT>
__device__ __forceinline__ double chunk_squares(const void* g, int64_t i0, int64_t i1) {
  typedef Piece<DT> P;
  double s = 0.;
  int64_t done = i0;
  if (((uintptr_t)g & 15u) == 0) {
    const u32x4_t* p = static_cast<const u32x4_t*>(g) + i0 / P::N;
    const int pieces = (int)((i1 - i0) / P::N);
    for (int i = threadIdx.x; i < pieces; i += kAhead * 256) {
      u32x4_t q[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j * 256 < pieces) q[j] = p[i + j * 256];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j * 256 < pieces) s += P(q[j]).squares();
    }
    done = i0 + (int64_t)pieces * P::N;
  }
  for (int64_t i = done + threadIdx.x; i < i1; i += 256) {
    const double v = (double)load1<DT>(g, i);
    s += v * v;
  }
  return s;
}

__global__ __launch_bounds__(256) void norm_kernel(Table t, double* __restrict__ parts) {
  __shared__ double lds[4];
  double s = 0.;
  for (int c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    const int k = tensor_of(t, c), dt = t.dtype[k];
    const void* g = t.g[k];
    const int64_t i0 = (int64_t)(c - t.first[k]) * t.chunk, i1 = min(i0 + t.chunk, t.numel[k]);
    if (dt == MOE_LORA_F32) s += chunk_squares<MOE_LORA_F32>(g, i0, i1);
    else if (dt == MOE_LORA_BF16) s += chunk_squares<MOE_LORA_BF16>(g, i0, i1);
    else s += chunk_squares<MOE_LORA_F16>(g, i0, i1);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

template <int DT>
__device__ __forceinline__ void chunk_scale(const void* g, void* o, int64_t i0, int64_t i1, float c) {
  typedef Piece<DT> P;
  int64_t done = i0;
  if ((((uintptr_t)g | (uintptr_t)o) & 15u) == 0) {
    const u32x4_t* p = static_cast<const u32x4_t*>(g) + i0 / P::N;
    u32x4_t* d = static_cast<u32x4_t*>(o) + i0 / P::N;
    const int pieces = (int)((i1 - i0) / P::N);
    for (int i = threadIdx.x; i < pieces; i += kAhead * 256) {
      u32x4_t q[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j * 256 < pieces) q[j] = __builtin_nontemporal_load(p + i + j * 256);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j * 256 < pieces) __builtin_nontemporal_store(P(q[j]).scaled(c), d + i + j * 256);
    }
    done = i0 + (int64_t)pieces * P::N;
  }
  for (int64_t i = done + threadIdx.x; i < i1; i += 256) store1<DT>(o, i, load1<DT>(g, i) * c);
}

__global__ __launch_bounds__(256) void scale_kernel(Table t, const double* __restrict__ parts, int nparts,
                                                    float max_norm, float* __restrict__ norm) {
  __shared__ double lds[4];
  double s = 0.;
  for (int i = threadIdx.x; i < nparts; i += 256) s += parts[i];
  s = sqrt(block_sum(s, lds));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)s;
  const double cd = (double)max_norm / (s + (double)kEps);
  // NaN stays NaN; without a bound (infinity) the norm does not matter
  const float c = cd > 1. || max_norm == INFINITY ? 1.f : (float)cd;
  for (int k0 = t.first[t.n] - 1 - (int)blockIdx.x; k0 >= 0; k0 -= gridDim.x) {
    const int k = tensor_of(t, k0), dt = t.dtype[k];
    const void* g = t.g[k];
    void* o = t.out[k];
    if (c == 1.f && g == o) continue;  // in place and nothing to scale
    const int64_t i0 = (int64_t)(k0 - t.first[k]) * t.chunk, i1 = min(i0 + t.chunk, t.numel[k]);
    if (dt == MOE_LORA_F32) chunk_scale<MOE_LORA_F32>(g, o, i0, i1, c);
    else if (dt == MOE_LORA_BF16) chunk_scale<MOE_LORA_BF16>(g, o, i0, i1, c);
    else chunk_scale<MOE_LORA_F16>(g, o, i0, i1, c);
  }
}

size_t dtype_size(int32_t d) { return d == MOE_LORA_F32 ? 4 : 2; }

int64_t chunks_of(int64_t numel, int chunk) { return (numel + chunk - 1) / chunk; }

int chunk_for(int64_t elements) {
  int c = kChunkMin;
  while (c < kChunkMax && elements > (int64_t)c * kMaxParts) c *= 2;
  return c;
}

}  // namespace

}  // namespace moelora

using namespace moelora;

extern "C" {

size_t moe_lora_clip_workspace_bytes(int32_t n) {
  if (n < 0) return 0;
  return sizeof(double) * (size_t)(kMaxParts + 1 + n / kTensors);
}

int moe_lora_clip_grads(const moe_lora_grad* grads, int32_t n, float max_norm, float* norm, void* workspace,
                        size_t ws_bytes, void* stream) {
  if (n < 0 || (n && !grads) || !norm || !(max_norm >= 0.f)) return MOE_LORA_EINVAL;
  if (!workspace || ws_bytes < moe_lora_clip_workspace_bytes(n)) return MOE_LORA_EWORKSPACE;
  if ((uintptr_t)workspace % 8 || (uintptr_t)norm % 4) return MOE_LORA_EALIGN;
  int64_t elements = 0;
  for (int32_t i = 0; i < n; ++i) {
    const moe_lora_grad& t = grads[i];
    if (t.numel < 0 || (t.dtype != MOE_LORA_F32 && t.dtype != MOE_LORA_BF16 && t.dtype != MOE_LORA_F16))
      return MOE_LORA_EINVAL;
    if (t.numel && (!t.g || !t.out)) return MOE_LORA_EINVAL;
    if ((uintptr_t)t.g % dtype_size(t.dtype) || (uintptr_t)t.out % dtype_size(t.dtype)) return MOE_LORA_EALIGN;
    if (t.numel > (1LL << 40) || elements > (1LL << 50)) return MOE_LORA_EUNSUPPORTED;
    elements += t.numel;
  }
  const int chunk = chunk_for(elements);
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) total += chunks_of(grads[i].numel, chunk);
  if (total > (1LL << 30)) return MOE_LORA_EUNSUPPORTED;
  // every byte written has one owner, and only a gradient's own output may
  // lie on it: the same tensor twice would be scaled twice
  struct Span {
    uintptr_t a, b;
    int32_t tensor;
    bool out;
  };
  Span* sp = new (std::nothrow) Span[2 * (size_t)n + 2];
  if (!sp) return MOE_LORA_EHIP;
  size_t ns = 0;
  for (int32_t i = 0; i < n; ++i) {
    const size_t bytes = (size_t)grads[i].numel * dtype_size(grads[i].dtype);
    if (!bytes) continue;
    sp[ns++] = Span{(uintptr_t)grads[i].out, (uintptr_t)grads[i].out + bytes, i, true};
    if (grads[i].g != grads[i].out) sp[ns++] = Span{(uintptr_t)grads[i].g, (uintptr_t)grads[i].g + bytes, i, false};
  }
  sp[ns++] = Span{(uintptr_t)norm, (uintptr_t)norm + 4, -1, true};
  sp[ns++] = Span{(uintptr_t)workspace, (uintptr_t)workspace + moe_lora_clip_workspace_bytes(n), -2, true};
  std::sort(sp, sp + ns, [](const Span& x, const Span& y) { return x.a < y.a; });
  uintptr_t end_any = 0, end_out = 0;
  bool bad = false;
  for (size_t i = 0; i < ns; ++i) {
    if (sp[i].a < (sp[i].out ? end_any : end_out)) bad = true;
    end_any = std::max(end_any, sp[i].b);
    if (sp[i].out) end_out = std::max(end_out, sp[i].b);
  }
  delete[] sp;
  if (bad) return MOE_LORA_EINVAL;

  hipStream_t st = (hipStream_t)stream;
  double* parts = (double*)workspace;
  int nparts = 0;
  const int32_t launches = std::max<int32_t>(1, (n + kTensors - 1) / kTensors);
  for (int pass = 0; pass < 2; ++pass) {
    for (int32_t l = 0; l < launches; ++l) {
      // backwards in the second pass
      const int32_t i0 = (pass ? launches - 1 - l : l) * kTensors;
      Table t = {};
      t.chunk = chunk;
      int64_t c = 0;
      while (t.n < kTensors && i0 + t.n < n) {
        const moe_lora_grad& e = grads[i0 + t.n];
        t.g[t.n] = e.g;
        t.out[t.n] = e.out;
        t.numel[t.n] = e.numel;
        t.dtype[t.n] = (uint8_t)e.dtype;
        t.first[t.n++] = (int)c;
        c += chunks_of(e.numel, chunk);
      }
      t.first[t.n] = (int)c;
      if (pass == 0) {
        // this launch's share of the partial sums, one at least
        const int blocks = (int)std::max<int64_t>(1, std::min(c, kMaxParts * c / std::max<int64_t>(1, total)));
        norm_kernel<<<blocks, 256, 0, st>>>(t, parts + nparts);
        nparts += blocks;
      } else {
        const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(c, kMaxParts));
        scale_kernel<<<blocks, 256, 0, st>>>(t, parts, nparts, max_norm, i0 == 0 ? norm : nullptr);
      }
      if (hipGetLastError() != hipSuccess) return MOE_LORA_EHIP;
    }
  }
  return MOE_LORA_OK;
}

}  // extern "C"
