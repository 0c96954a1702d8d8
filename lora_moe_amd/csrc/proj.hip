// C ABI of the shared projection with the adapters of many requests: argument
// checks, workspace layout and the order of its kernels.  Contracts:
// include/moe_lora.h.
#include <algorithm>

#include "abi_util.h"
#include "device_util.h"
#include "proj.h"

using namespace moelora;

namespace moelora {
namespace {

constexpr int32_t kMaxTokens = 1 << 17, kMaxWidth = 1 << 20, kMaxAdapters = 2047, kMaxRank = 128;
// what a 32-bit offset reaches, a stage's padding aside
constexpr int64_t kMaxBytes = (1LL << 31) - 256;

int check_shape(const moe_lora_proj_shape* s) {
  if (!s || s->T < 0 || s->K <= 0 || s->N <= 0 || s->L <= 0 || s->r <= 0) return MOE_LORA_EINVAL;
  if (s->K % 8 || s->N % 8) return MOE_LORA_EALIGN;
  if (s->r % 8 || s->r > kMaxRank || s->L > kMaxAdapters || s->T > kMaxTokens || s->K > kMaxWidth ||
      s->N > kMaxWidth)
    return MOE_LORA_EUNSUPPORTED;
  const int64_t wide = std::max(s->K, s->N);
  if (s->T * wide * 2 > kMaxBytes || (int64_t)s->L * s->r * wide * 2 > kMaxBytes) return MOE_LORA_EUNSUPPORTED;
  return MOE_LORA_OK;
}

struct Sizes {  // bytes
  size_t x, y, ids, W, A, B, scales, z;
  explicit Sizes(const moe_lora_proj_shape& s) {
    const size_t T = s.T, K = s.K, N = s.N, L = s.L, r = s.r;
    x = T * K * 2;
    y = T * N * 2;
    ids = T * 4;
    W = N * K * 2;
    A = L * r * K * 2;
    B = L * r * N * 2;
    scales = L * 4;
    z = T * r * 4;
  }
};

ProjArgs args_of(const moe_lora_proj_shape& s, const int32_t* ids, const float* scales, bool grads) {
  ProjArgs p = {};
  p.T = s.T, p.K = s.K, p.N = s.N, p.L = s.L, p.r = s.r, p.scale = s.lora_scale;
  p.ids = ids, p.scales = scales;
  p.shrink_rows = proj_shrink_rows(s.T, s.r);
  p.grad_rows = grads ? proj_grad_rows(s.T, s.K, s.N, s.L, s.r) : 0;
  return p;
}

// A workspace's parts, in the order that they are taken.
struct Parts {
  char* at;
  size_t used = 0;
  explicit Parts(void* ws) : at((char*)ws) {}
  template <class E>
  E* take(size_t n) {
    E* p = (E*)(at + used);
    used += round256(n * sizeof(E));
    return p;
  }
};

void take_order(ProjArgs& p, Parts& w) {
  p.o.perm = w.take<int32_t>(p.T);
  p.o.run = w.take<int32_t>(p.T);
  p.o.adapter = w.take<int32_t>(p.L + 1);
  p.o.count = w.take<int32_t>(4);
  p.o.shrink = w.take<ProjItem>(proj_items(p.T, p.L, p.shrink_rows));
  if (!p.grad_rows) return;
  p.o.grad = w.take<ProjItem>(proj_grad_items(p));
  p.o.slabs = w.take<int32_t>(2 * p.L);
}

struct Forward {
  uint16_t* parts;
  float* slabs;
  size_t bytes;
  Forward(ProjArgs& p, void* ws) {
    Parts w(ws);
    if (proj_few(p.T, p.N, p.L, p.r)) {
      slabs = w.take<float>(proj_few_slab_bytes(p) / 4);
    } else {
      take_order(p, w);
      parts = w.take<uint16_t>((size_t)p.T * kParts * p.r);
      slabs = w.take<float>(proj_gemm_slab_bytes(p, false) / 4);
    }
    bytes = w.used;
  }
};

struct Backward {
  uint16_t *us, *zs;
  float* slabs;  // of dx, then of the gradients
  size_t bytes;
  Backward(ProjArgs& p, void* ws) {
    Parts w(ws);
    take_order(p, w);
    us = w.take<uint16_t>((size_t)p.T * kParts * p.r);
    zs = w.take<uint16_t>((size_t)p.T * kParts * p.r);
    slabs = w.take<float>(std::max(proj_gemm_slab_bytes(p, true), proj_grad_slab_bytes(p)) / 4);
    bytes = w.used;
  }
};

size_t ws_bytes_of(const moe_lora_proj_shape& s, bool backward) {
  ProjArgs p = args_of(s, nullptr, nullptr, false);
  const size_t forward = Forward(p, nullptr).bytes;
  if (!backward) return forward;
  ProjArgs q = args_of(s, nullptr, nullptr, true);
  return std::max(forward, Backward(q, nullptr).bytes);
}

__global__ __launch_bounds__(256) void proj_zero_kernel(u32x4_t* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = zero4();
}

int zero(void* p, size_t bytes, hipStream_t st) {
  const int64_t n = (int64_t)(bytes / 16);
  proj_zero_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>((u32x4_t*)p, n);
  return hipGetLastError() == hipSuccess ? MOE_LORA_OK : MOE_LORA_EHIP;
}

}  // namespace
}  // namespace moelora

extern "C" {

size_t moe_lora_proj_workspace_bytes(const moe_lora_proj_shape* shape, int backward) {
  if (check_shape(shape)) return 0;
  // T = 0 too: 0 says the shape is invalid
  return shape->T ? ws_bytes_of(*shape, backward != 0) : 256;
}

int moe_lora_proj_forward(const moe_lora_proj_shape* shape, const uint16_t* x, const int32_t* lora_ids,
                          const uint16_t* W, const uint16_t* A, const uint16_t* B, const float* scales, float* z,
                          void* workspace, size_t ws_bytes, uint16_t* y, void* stream) {
  const int rc = check_shape(shape);
  if (rc) return rc;
  if (shape->T == 0) return MOE_LORA_OK;
  if (!x || !lora_ids || !W || !A || !B || !y) return MOE_LORA_EINVAL;
  const size_t need = ws_bytes_of(*shape, false);
  if (!workspace || ws_bytes < need) return MOE_LORA_EWORKSPACE;
  const void* ptrs[] = {x, lora_ids, W, A, B, scales, z, workspace, y};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_LORA_EALIGN;
  const Sizes n(*shape);
  const Range in[] = {{x, n.x}, {lora_ids, n.ids}, {W, n.W}, {A, n.A}, {B, n.B}, {scales, scales ? n.scales : 0}};
  const Range out[] = {{y, n.y}, {z, z ? n.z : 0}, {workspace, need}};
  if (any_overlap(in, 6, out, 3)) return MOE_LORA_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  ProjArgs p = args_of(*shape, lora_ids, scales, false);
  const Forward f(p, workspace);
  if (proj_few(p.T, p.N, p.L, p.r)) return launch_proj_few(p, x, W, A, B, z, f.slabs, y, st);
  int r = launch_proj_order(p, z, nullptr, nullptr, st);
  if (!r) r = launch_proj_shrink(p, false, x, A, f.parts, z, st);
  return r ? r : launch_proj_gemm(p, false, ProjGemm{x, W, f.parts, B, y, f.slabs, 1}, st);
}

int moe_lora_proj_backward(const moe_lora_proj_shape* shape, const uint16_t* dy, const uint16_t* x,
                           const int32_t* lora_ids, const float* z, const uint16_t* W, const uint16_t* A,
                           const uint16_t* B, const float* scales, void* workspace, size_t ws_bytes, uint16_t* dx,
                           uint16_t* dA, uint16_t* dB, void* stream) {
  const int rc = check_shape(shape);
  if (rc) return rc;
  const Sizes n(*shape);
  hipStream_t st = (hipStream_t)stream;
  // without tokens dx is empty, whatever its address, and only the adapters'
  // gradients are left to write
  if (shape->T == 0) dx = nullptr;
  else if (!dx && !dA && !dB) return MOE_LORA_EINVAL;
  const size_t need = shape->T > 0 ? ws_bytes_of(*shape, true) : 0;
  if (shape->T > 0) {
    if (!dy || !x || !lora_ids || !z || !W || !A || !B) return MOE_LORA_EINVAL;
    if (!workspace || ws_bytes < need) return MOE_LORA_EWORKSPACE;
  }
  const void* ptrs[] = {dy, x, lora_ids, z, W, A, B, scales, workspace, dx, dA, dB};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_LORA_EALIGN;
  const Range in[] = {{dy, n.y}, {x, n.x}, {lora_ids, n.ids}, {z, n.z},
                      {W, n.W},  {A, n.A}, {B, n.B},          {scales, scales ? n.scales : 0}};
  const Range out[] = {{dx, dx ? n.x : 0}, {dA, dA ? n.A : 0}, {dB, dB ? n.B : 0}, {workspace, need}};
  if (any_overlap(in, 8, out, 4)) return MOE_LORA_EINVAL;
  int r = MOE_LORA_OK;
  if (shape->T == 0) {
    if (dA) r = zero(dA, n.A, st);
    if (dB && !r) r = zero(dB, n.B, st);
    return r;
  }
  ProjArgs p = args_of(*shape, lora_ids, scales, true);
  const Backward b(p, workspace);
  r = launch_proj_order(p, nullptr, z, dB ? b.zs : nullptr, st);
  if (!r && (dx || dA)) r = launch_proj_shrink(p, true, dy, B, b.us, nullptr, st);
  if (!r && dx) r = launch_proj_gemm(p, true, ProjGemm{dy, W, b.us, A, dx, b.slabs, 1}, st);
  if (!r && (dA || dB)) r = launch_proj_grads(p, ProjGrads{x, dy, b.us, b.zs, dA, dB, b.slabs}, st);
  return r;
}

}  // extern "C"
