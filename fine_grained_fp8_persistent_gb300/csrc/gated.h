// gated.h -- declarations shared by the gated feed-forward and 4-bit matrix-vector
// translation units (not part of the public ABI).
#pragma once
#include "fgf8_internal.h"

namespace fgf8 {

constexpr int kGemvMaxRows = 16;   // rows of X the matrix-vector kernels take
// Largest M, N and K of these operators: the kernels round sizes up to tiles, at most 512
// rows or columns past the end, in 32-bit integers.
constexpr int kMaxSize = 0x7FFFFFFF - 1023;

// One gated_f16 / gated_f16_backward call: M tokens, N inner columns, K hidden size.
struct GatedArgs {
  int M, N, K;
  int bf16;   // operand type: 1 bf16, 0 fp16
  int act;    // fgf8_act
};

// One matrix-vector call: M rows of X, N weight rows (of each matrix when gated), K.
struct GemvArgs {
  const void* X;
  const void* W[2];    // quantize_fp4 codes (gate, up when gated)
  const void* SF[2];   // their scale tables
  void* out;
  int M, N, K;
  int fmt;             // fgf8_fp4_fmt
  int bf16;            // type of X and out: 1 bf16, 0 fp16
  int act;             // fgf8_act, or -1: not gated
};

int launch_gated_forward(const GatedArgs& a, const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                         cudaStream_t stream);
int launch_gated_backward(const GatedArgs& a, const void* dH, const void* X, const void* Wg, const void* Wu,
                          const void* G, const void* U, void* dX, void* dWg, void* dWu, void* dG, void* dU,
                          cudaStream_t stream);
// The forward pass for a few tokens (M <= kGemvMaxRows), bound by reading the weights.
int launch_gated_gemv_f16(const GatedArgs& a, const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                          cudaStream_t stream);
int launch_gemv_fp4(const GemvArgs& a, cudaStream_t stream);

}  // namespace fgf8
