// Internal declarations of the gated feed-forward block (ffn.hip,
// ffn_gemm.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_lora.h"

namespace moelora {

// The products of the block.  Each is C[m][n] = sum_k A(m, k) B(n, k) with
// bf16 operands that lie either with k contiguous (A[m*lda + k]) or with the
// output index contiguous (A[k*lda + m]), and an epilogue on the fp32 sums.
enum FfnProduct {
  FFN_GATE_UP,   // A = x, B = W_gu (gate and up rows interleaved): h = act(g) * u, gu kept on request
  FFN_DOWN,      // A = h, B = W_down: y
  FFN_DH,        // A = dy, B = W_down by its columns: dg, du and h from dh and the kept gu
  FFN_DX,        // A = dgu, B = W_gu by its columns: dx
  FFN_DW,        // A = dgu or dy, B = x or h, both by their columns (k = token): dW
};

struct FfnGemm {
  const uint16_t* A;
  const uint16_t* B;
  int64_t lda, ldb;  // elements
  int M, N, K;       // FFN_GATE_UP: N = I
  uint16_t* out;     // bf16: h (GATE_UP), y, dgu (DH: [M][2N]), dx, dW
  uint16_t* out2;    // DH: h
  float* gu;         // GATE_UP: kept pre-activations [M][2N] or NULL; DH: read
  int act;
  int pair;          // DH: dgu and h get their remainders as rows M..2M-1; DX: A is such a pair (rows M..2M-1,
                     // added to rows 0..M-1 of the product); DW: A or B is one (K = 2 tokens, see wrap)
  int wrap_a, wrap_b;  // DW of a pair: k from here on meets the side's rows from 0 again (0: no pair); K <= 64
  float* slabs;      // scratch of ffn_gemm_slab_bytes
  int splits;        // K splits, set by the launch
};

// Up to this many tokens a forward streams the weights (ffn_rows.hip), beyond
// it takes tiles.  One limit for all sizes, between what small and what wide
// blocks would rather have.  Measured, us, streamed and tiled, at 24, 33 and 64
// tokens: H 1024, I 2816, 18 and 23, 21 and 23, 23 and 25; 2880, 2880, 26 and
// 32, 28 and 33, 32 and 35; 4096, 11008, 70 and 78, 75 and 79, 83 and 86; 5120,
// 25600, 179 and 157, 187 and 162, 197 and 177 (there tiles are better from 17
// tokens on, 174 and 167).
constexpr int kRowsMax = 32;
// Up to this many, h, dg and du go from one product to the next as bf16 pairs
// hi + lo: with so few tokens a few large values carry a result, so that one
// rounding more than its own can show by more than its share (in 64-bit
// emulations of 1 to 3 tokens up to 1.68 times a single rounding's error).  It
// costs nothing beside the weights: the remainders lie in the same fragment of
// 16 rows, or in a second one.  From 17 tokens on they are rounded once, as by
// a layer that writes bf16 between its products: y and the gradients are then
// off by 1.41 times their own rounding (relative L2 2.35e-3 against 1.66e-3),
// at most 1.48 in the emulations, while pairs would double the operations of
// the down, dx and weight-gradient products, which these bound in training.
constexpr int kRowsPair = 16;

// FFN_GATE_UP or FFN_DOWN of at most kRowsMax rows.  a_lo: the remainder of A
// (at most kRowsPair rows), or NULL; out_lo: that of h, or NULL; g.slabs:
// ffn_rows_slab_bytes of scratch.
int launch_ffn_rows(const FfnGemm& g, FfnProduct product, const uint16_t* a_lo, uint16_t* out_lo, hipStream_t st);
size_t ffn_rows_slab_bytes(int T, int H, int I);

// Bytes of scratch that a product of these sizes needs (0 where K is not split
// and A is no pair).
size_t ffn_gemm_slab_bytes(int M, int N, int K, FfnProduct product, bool pair = false);

int launch_ffn_gemm(const FfnGemm& g, FfnProduct product, hipStream_t st);

// The FFN_DX and the two FFN_DW of a backward that wants all three; dx.slabs:
// the larger of ffn_grads_slab_bytes and the products' own.
size_t ffn_grads_slab_bytes(int T, int H, int I);
int launch_ffn_grads(const FfnGemm& dx, const FfnGemm& dw_gu, const FfnGemm& dw_down, hipStream_t st);

}  // namespace moelora
