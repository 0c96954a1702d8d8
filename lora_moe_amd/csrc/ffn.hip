// C ABI of the gated feed-forward block: argument checks, workspace layout
// and the order of its products.  Contracts: include/moe_lora.h.
#include "ffn.h"

#include <algorithm>

#include "abi_util.h"

using namespace moelora;

namespace moelora {
namespace {

// Row-major offsets inside a tile are 32-bit: a panel of 256 rows of 2I or H
// bf16 stays under 2^31 bytes up to 2^21 columns.
constexpr int32_t kMaxWidth = 1 << 20, kMaxTokens = 1 << 26;

int check_shape(const moe_lora_ffn_shape* s) {
  if (!s || s->T < 0 || s->H <= 0 || s->I <= 0) return MOE_LORA_EINVAL;
  if (s->act != MOE_LORA_ACT_SILU && s->act != MOE_LORA_ACT_GELU) return MOE_LORA_EINVAL;
  if (s->H % 8 || s->I % 8) return MOE_LORA_EALIGN;
  if (s->H > kMaxWidth || s->I > kMaxWidth || s->T > kMaxTokens) return MOE_LORA_EUNSUPPORTED;
  return MOE_LORA_OK;
}

struct Sizes {  // bytes
  size_t x, w_gu, w_down, gu, h, dgu;
  explicit Sizes(const moe_lora_ffn_shape& s) {
    const size_t T = s.T, H = s.H, I = s.I;
    x = T * H * 2;
    w_gu = 2 * I * H * 2;
    w_down = H * I * 2;
    gu = T * 2 * I * 4;
    h = T * I * 2;
    dgu = T * 2 * I * 2;
  }
};

// forward: h, slabs; backward: h, dgu, slabs; up to kRowsPair tokens h and
// dgu with their remainders, of as many rows, right behind them
size_t h_bytes(const moe_lora_ffn_shape& s) { return round256(Sizes(s).h * (s.T <= kRowsPair ? 2 : 1)); }
size_t backward_fixed(const moe_lora_ffn_shape& s) {
  return h_bytes(s) + round256(Sizes(s).dgu * (s.T <= kRowsPair ? 2 : 1));
}

size_t ws_bytes_of(const moe_lora_ffn_shape& s, bool backward) {
  const int T = s.T, H = s.H, I = s.I;
  const size_t slabs = T <= kRowsMax ? ffn_rows_slab_bytes(T, H, I)
                                     : std::max(ffn_gemm_slab_bytes(T, I, H, FFN_GATE_UP),
                                                ffn_gemm_slab_bytes(T, H, I, FFN_DOWN));
  const size_t forward = h_bytes(s) + round256(slabs);
  if (!backward) return forward;
  const bool pair = T <= kRowsPair;
  const int k = pair ? 2 * T : T;
  const size_t back = std::max({ffn_grads_slab_bytes(T, H, I), ffn_gemm_slab_bytes(T, I, H, FFN_DH), ffn_gemm_slab_bytes(T, H, 2 * I, FFN_DX, pair),
                                ffn_gemm_slab_bytes(2 * I, H, k, FFN_DW), ffn_gemm_slab_bytes(H, I, k, FFN_DW)});
  return std::max(forward, backward_fixed(s) + round256(back));
}

}  // namespace
}  // namespace moelora

extern "C" {

size_t moe_lora_ffn_workspace_bytes(const moe_lora_ffn_shape* shape, int backward) {
  if (check_shape(shape)) return 0;
  // T = 0 too: 0 says the shape is invalid
  return shape->T ? ws_bytes_of(*shape, backward != 0) : 256;
}

int moe_lora_ffn_forward(const moe_lora_ffn_shape* shape, const uint16_t* x, const uint16_t* W_gu,
                         const uint16_t* W_down, float* gu, void* workspace, size_t ws_bytes, uint16_t* y,
                         void* stream) {
  const int rc = check_shape(shape);
  if (rc) return rc;
  if (shape->T == 0) return MOE_LORA_OK;
  const Sizes z(*shape);
  const size_t need = ws_bytes_of(*shape, false);
  if (!x || !W_gu || !W_down || !y) return MOE_LORA_EINVAL;
  if (!workspace || ws_bytes < need) return MOE_LORA_EWORKSPACE;
  if (!aligned16(x) || !aligned16(W_gu) || !aligned16(W_down) || !aligned16(gu) || !aligned16(y) ||
      !aligned16(workspace))
    return MOE_LORA_EALIGN;
  const Range in[] = {{x, z.x}, {W_gu, z.w_gu}, {W_down, z.w_down}};
  const Range out[] = {{y, z.x}, {gu, gu ? z.gu : 0}, {workspace, need}};
  if (any_overlap(in, 3, out, 3)) return MOE_LORA_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  const int T = shape->T, H = shape->H, I = shape->I;
  uint16_t* h = (uint16_t*)workspace;
  FfnGemm g = {};
  g.act = shape->act;
  g.A = x, g.lda = H, g.B = W_gu, g.ldb = H, g.M = T, g.N = I, g.K = H, g.out = h, g.gu = gu;
  g.slabs = (float*)((char*)workspace + h_bytes(*shape));
  if (T <= kRowsMax) {
    uint16_t* h_lo = T <= kRowsPair ? h + (size_t)T * I : nullptr;
    const int r = launch_ffn_rows(g, FFN_GATE_UP, nullptr, h_lo, st);
    if (r) return r;
    g.A = h, g.lda = I, g.B = W_down, g.ldb = I, g.N = H, g.K = I, g.out = y, g.gu = nullptr;
    return launch_ffn_rows(g, FFN_DOWN, h_lo, nullptr, st);
  }
  const int r1 = launch_ffn_gemm(g, FFN_GATE_UP, st);
  if (r1) return r1;
  g.A = h, g.lda = I, g.B = W_down, g.ldb = I, g.N = H, g.K = I, g.out = y, g.gu = nullptr;
  return launch_ffn_gemm(g, FFN_DOWN, st);
}

int moe_lora_ffn_backward(const moe_lora_ffn_shape* shape, const uint16_t* dy, const uint16_t* x, const float* gu,
                          const uint16_t* W_gu, const uint16_t* W_down, void* workspace, size_t ws_bytes,
                          uint16_t* dx, uint16_t* dW_gu, uint16_t* dW_down, void* stream) {
  const int rc = check_shape(shape);
  if (rc) return rc;
  // without tokens dx is empty, whatever its address, and only the weights'
  // gradients are left to write
  if (shape->T == 0) dx = nullptr;
  else if (!dx && !dW_gu && !dW_down) return MOE_LORA_EINVAL;
  const int T = shape->T, H = shape->H, I = shape->I;
  const Sizes z(*shape);
  const size_t need = T > 0 ? ws_bytes_of(*shape, true) : 0;
  if (T > 0) {
    if (!dy || !x || !gu || !W_gu || !W_down) return MOE_LORA_EINVAL;
    if (!workspace || ws_bytes < need) return MOE_LORA_EWORKSPACE;
  }
  const void* ptrs[] = {dy, x, gu, W_gu, W_down, workspace, dx, dW_gu, dW_down};
  for (const void* p : ptrs)
    if (!aligned16(p)) return MOE_LORA_EALIGN;
  const Range in[] = {{dy, z.x}, {x, z.x}, {gu, z.gu}, {W_gu, z.w_gu}, {W_down, z.w_down}};
  const Range out[] = {{dx, dx ? z.x : 0},
                       {dW_gu, dW_gu ? z.w_gu : 0},
                       {dW_down, dW_down ? z.w_down : 0},
                       {workspace, need}};
  if (any_overlap(in, 5, out, 4)) return MOE_LORA_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  uint16_t* h = (uint16_t*)workspace;
  uint16_t* dgu = (uint16_t*)((char*)workspace + h_bytes(*shape));
  FfnGemm g = {};
  g.act = shape->act;
  g.slabs = (float*)((char*)workspace + backward_fixed(*shape));
  g.A = dy, g.lda = H, g.B = W_down, g.ldb = I, g.M = T, g.N = I, g.K = H;
  g.out = dgu, g.out2 = h, g.gu = const_cast<float*>(gu), g.pair = T <= kRowsPair;
  int r = launch_ffn_gemm(g, FFN_DH, st);
  if (r) return r;
  g.gu = nullptr, g.out2 = nullptr;
  FfnGemm gx = g, gw = g, gd = g;
  gx.A = dgu, gx.lda = 2 * (int64_t)I, gx.B = W_gu, gx.ldb = H, gx.M = T, gx.N = H, gx.K = 2 * I, gx.out = dx;
  // the pair's remainders are further tokens of the sums, with the same x or dy
  const int K = g.pair ? 2 * T : T;
  gw.A = dgu, gw.lda = 2 * (int64_t)I, gw.B = x, gw.ldb = H, gw.M = 2 * I, gw.N = H, gw.K = K, gw.out = dW_gu;
  gw.wrap_a = 0, gw.wrap_b = g.pair ? T : 0;
  gd.A = dy, gd.lda = H, gd.B = h, gd.ldb = I, gd.M = H, gd.N = I, gd.K = K, gd.out = dW_down;
  gd.wrap_a = g.pair ? T : 0, gd.wrap_b = 0;
  if (dx && dW_gu && dW_down) return launch_ffn_grads(gx, gw, gd, st);
  if (dx && (r = launch_ffn_gemm(gx, FFN_DX, st))) return r;
  if (dW_gu && (r = launch_ffn_gemm(gw, FFN_DW, st))) return r;
  if (dW_down && (r = launch_ffn_gemm(gd, FFN_DW, st))) return r;
  return MOE_LORA_OK;
}

}  // extern "C"
