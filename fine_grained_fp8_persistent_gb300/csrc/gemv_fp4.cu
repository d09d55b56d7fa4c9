// gemv_fp4.cu -- products of a few rows of X with 4-bit weights (the layouts of
// quantize_fp4), plain or gated.
//
//   Y[m][n] = sum_k X[m][k] * E2M1(code[n][k]) * scale[n][k / SV]
//
// SV = 32 with E8M0 scales (MXFP4) or 16 with E4M3 scales (NVFP4).
#include "activation.cuh"
#include "gated.h"
#include "ptx.cuh"

namespace fgf8 {
namespace {

constexpr int kMaxRows = 16;

// The value of an E2M1 code (bit 3 sign, bits 2-1 exponent, bit 0 mantissa).
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float v = e == 0 ? 0.5f * m : (1.0f + 0.5f * m) * static_cast<float>(1u << (e - 1));
  return (c & 8u) ? -v : v;
}

// The value of a scale byte: 2^(b - 127), or E4M3.
__device__ __forceinline__ float scale_value(uint32_t b, int fmt) {
  if (fmt != 0) return ptx::e4m3_value(b);
  return b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

// One warp per output column n; lane l takes the 8-code words l, l + 32, ... of the row.
__global__ void __launch_bounds__(128) gemv_kernel(GemvArgs a) {
  const int n = blockIdx.x * 4 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (n >= a.N) return;
  const int sv = a.fmt == 0 ? 32 : 16, ld = (a.N + 3) / 4 * 4, mats = a.act >= 0 ? 2 : 1;
  const uint16_t* X = static_cast<const uint16_t*>(a.X);
  for (int m = 0; m < a.M; ++m) {
    float sum[2] = {0.0f, 0.0f};
    for (int j = 0; j < mats; ++j) {
      const uint32_t* w = static_cast<const uint32_t*>(a.W[j]) + static_cast<size_t>(n) * (a.K / 8);
      const uint8_t* sf = static_cast<const uint8_t*>(a.SF[j]);
      for (int i = lane; i < a.K / 8; i += 32) {
        const uint32_t codes = w[i];
        const int group = i * 8 / sv;
        const float s = scale_value(sf[(static_cast<size_t>(group / 4) * ld + n) * 4 + group % 4], a.fmt);
        float part = 0.0f;
        for (int c = 0; c < 8; ++c)
          part = fmaf(act::to_float(X[static_cast<size_t>(m) * a.K + 8 * i + c], a.bf16 != 0), e2m1_value(codes >> (4 * c) & 15u), part);
        sum[j] = fmaf(part, s, sum[j]);
      }
      for (int off = 16; off > 0; off >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], off);
    }
    if (lane == 0) {
      float v = sum[0];
      if (a.act >= 0) v = (a.act == act::kSilu ? act::value<act::kSilu>(v) : act::value<act::kGeluTanh>(v)) * sum[1];
      static_cast<uint16_t*>(a.out)[static_cast<size_t>(m) * a.N + n] = act::from_float(v, a.bf16 != 0);
    }
  }
}

}  // namespace

int launch_gemv_fp4(const GemvArgs& a, cudaStream_t stream) {
  gemv_kernel<<<(a.N + 3) / 4, 128, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? 0 : set_error(4, "gemv_fp4 launch: %s", cudaGetErrorString(e));
}

}  // namespace fgf8
