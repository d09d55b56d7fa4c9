// routed.h -- declarations shared by the translation units of the operators whose rows
// choose their own weights (not part of the public ABI).
#pragma once
#include "fgf8_internal.h"

namespace fgf8 {

constexpr int kRouteMaxGroups = 1024;             // one thread per group in the routing kernel's scan
constexpr int kRouteMaxSize = 0x7FFFFFFF - 1023;  // entries and rows: 32-bit integers, rounded up to tiles

// One routing: n = T k ids in flat order.
struct RouteArgs {
  const void* ids;      // int32 or int64
  int ids64;
  int32_t* rows;        // [n] row of each entry, -1 = none
  int32_t* src;         // [M] entry of each row, -1 = none
  int32_t* m_indices;   // [M] group of each row, -1 = none (null: masked layout)
  int32_t* counts;      // [G]
  int32_t* starts;      // [G + 1] (null: masked layout)
  int n, G, M;
  int align;            // contiguous: rows to which a segment is padded
  int slots;            // masked: rows of a group, 0 = contiguous layout
  uint32_t* status;
};

// Rows of T tokens of which entry (t, j) owns row rows[t][j].
struct RowsArgs {
  const int32_t* rows;  // [T][k]
  const int32_t* src;   // [M], null where rows without an entry stay as they are
  int T, k, M;
  int H;                // elements of a row
  int slots;            // masked layout: rows of a group, 0 = contiguous layout
  uint32_t* status;
};

int launch_route(const RouteArgs& a, cudaStream_t stream);
int launch_dispatch_f16(const RowsArgs& a, const void* X, void* Xs, cudaStream_t stream);
int launch_dispatch_fp8(const RowsArgs& a, const void* X, void* Xq, void* SFA, int fmt, cudaStream_t stream);
// W null: weights of one.
int launch_combine_f16(const RowsArgs& a, const void* Ys, const float* W, void* Y, int bf16, cudaStream_t stream);
int launch_combine_f16_backward(const RowsArgs& a, const void* dY, const void* Ys, const float* W, void* dYs, float* dW,
                                int bf16, cudaStream_t stream);

// One lora_f16 call: rows of the contiguous layout, one entry per token.
struct LoraArgs {
  const void* X;            // [T][K], rows ldx apart
  const void* A;            // [G][r][K]
  const void* B;            // [G][N][r]
  const float* scale;       // [G], null: 1
  const void* base;         // [T][N], rows ldb apart, null: 0
  void* out;                // [T][N], rows ldo apart
  const int32_t* rows;      // [T]
  const int32_t* src;       // [M]
  const int32_t* m_indices; // [M]
  long long ldx, ldb, ldo;
  int T, K, N, r, G, M;
  int align;                // rows with one adapter, a multiple of 16 that divides M
  uint32_t* status;
};
int launch_lora_f16(const LoraArgs& a, int bf16, cudaStream_t stream);

}  // namespace fgf8
