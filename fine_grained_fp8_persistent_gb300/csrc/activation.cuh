// activation.cuh -- the activations of the gated operators and their slopes, in FP32.
//
// Both are g * s with a logistic s = 1 / (1 + exp(-y)), c = s (1 - s):
//   SiLU       y = g
//   GELU-tanh  y = 2 z, z = sqrt(2/pi) (g + 0.044715 g^3), as (1 + tanh z) / 2 = sigma(2 z)
// (this form has no cancellation for negative g, where 1 + tanh z would lose all
// its digits), so a'(g) = s + g c y'(g).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace fgf8 {
namespace act {

constexpr int kSilu = 0;
constexpr int kGeluTanh = 1;
constexpr float kGeluA = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

template <int ACT>
__device__ __forceinline__ float inner(float g) {
  return ACT == kSilu ? g : 2.0f * kGeluA * g * fmaf(kGeluB * g, g, 1.0f);
}
template <int ACT>
__device__ __forceinline__ float inner_slope(float g) {
  return ACT == kSilu ? 1.0f : 2.0f * kGeluA * fmaf(3.0f * kGeluB * g, g, 1.0f);
}
// s and s (1 - s) from t = exp(-|y|) <= 1: nothing overflows, 1 - s does not cancel, and t
// goes down into the FP32 subnormals (y = -103), where g s times a large U is still a plain
// value.  The fast exponential is off by about |y| 2^-23 of itself (2^-16 where t is
// smallest), the reciprocal of [1, 2] by one unit: far below the 16-bit rounding.
template <int ACT>
__device__ __forceinline__ float logistic(float g, float& c) {
  const float y = inner<ACT>(g);
  const float t = __expf(-fabsf(y));
  float r;                                            // 1 / (1 + t): no operand out of [1, 2] but NaN
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
  const float tr = t * r;
  c = tr * r;
  return y < 0.0f ? tr : r;
}
template <int ACT>
__device__ __forceinline__ float value(float g) {
  float c;
  return g * logistic<ACT>(g, c);
}

// a(g) and a'(g).  Where s is 0 or 1 the second term of the slope is 0, also for
// |g| so large that y'(g) overflows.
template <int ACT>
__device__ __forceinline__ void value_slope(float g, float& v, float& d) {
  float c;
  const float s = logistic<ACT>(g, c);
  v = g * s;
  d = s + (c == 0.0f ? 0.0f : g * c * inner_slope<ACT>(g));
}

__device__ __forceinline__ float to_float(uint32_t bits16, bool bf16) {
  return bf16 ? __uint_as_float(bits16 << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(bits16)));
}
__device__ __forceinline__ uint16_t from_float(float v, bool bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

}  // namespace act
}  // namespace fgf8
