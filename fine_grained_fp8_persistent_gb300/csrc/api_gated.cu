// api_gated.cu -- the C ABI of the gated feed-forward and 4-bit matrix-vector
// operators (include/fgf8.h): host-side validation and dispatch.
#include "../../include/fgf8.h"
#include "check.h"
#include "gated.h"

namespace {

using fgf8::check_pointers;

int check_sizes(const char* who, int M, int N, int K) {
  if (M < 0 || N <= 0 || K <= 0) return fgf8::set_error(FGF8_ERR_INVALID_ARG, "%s: M=%d N=%d K=%d", who, M, N, K);
  if (M > fgf8::kMaxSize || N > fgf8::kMaxSize || K > fgf8::kMaxSize)
    return fgf8::set_error(FGF8_ERR_UNSUPPORTED, "%s: M=%d N=%d K=%d: sizes above %d", who, M, N, K, fgf8::kMaxSize);
  return FGF8_OK;
}

int check_gated(const char* who, int M, int N, int K, int dtype, int act) {
  if (int r = check_sizes(who, M, N, K)) return r;
  if (dtype != FGF8_F16 && dtype != FGF8_BF16) return fgf8::set_error(FGF8_ERR_INVALID_ARG, "%s: bad dtype %d", who, dtype);
  if (act != FGF8_ACT_SILU && act != FGF8_ACT_GELU_TANH)
    return fgf8::set_error(FGF8_ERR_INVALID_ARG, "%s: bad activation %d", who, act);
  if (K % 8 != 0 || N % 8 != 0)
    return fgf8::set_error(FGF8_ERR_UNSUPPORTED, "%s: K=%d and N=%d must be multiples of 8", who, K, N);
  return FGF8_OK;
}

int check_gemv(const char* who, int M, int N, int K, int fmt, int dtype) {
  if (int r = check_sizes(who, M, N, K)) return r;
  if (fmt != FGF8_FP4_MX && fmt != FGF8_FP4_NV) return fgf8::set_error(FGF8_ERR_INVALID_ARG, "%s: bad format %d", who, fmt);
  if (dtype != FGF8_F16 && dtype != FGF8_BF16) return fgf8::set_error(FGF8_ERR_INVALID_ARG, "%s: bad dtype %d", who, dtype);
  if (K % 64 != 0) return fgf8::set_error(FGF8_ERR_UNSUPPORTED, "%s: K=%d not a multiple of 64", who, K);
  if (M > fgf8::kGemvMaxRows)
    return fgf8::set_error(FGF8_ERR_UNSUPPORTED, "%s: M=%d above %d rows", who, M, fgf8::kGemvMaxRows);
  return FGF8_OK;
}

}  // namespace

extern "C" {

int gated_f16(const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U, int M, int N, int K,
              int dtype, int act, void* stream) {
  if (int r = check_gated("gated_f16", M, N, K, dtype, act)) return r;
  if (M == 0) return FGF8_OK;
  if ((G == nullptr) != (U == nullptr))
    return fgf8::set_error(FGF8_ERR_INVALID_ARG, "gated_f16: G and U must be given together");
  if (int r = check_pointers("gated_f16", {X, Wg, Wu, H})) return r;
  if (G != nullptr)
    if (int r = check_pointers("gated_f16", {G, U})) return r;
  const fgf8::GatedArgs a{M, N, K, dtype == FGF8_BF16, act};
  return fgf8::launch_gated_forward(a, X, Wg, Wu, H, G, U, static_cast<cudaStream_t>(stream));
}

// dG and dU back to back, each padded to 16 bytes (N is a multiple of 8)
long long fgf8_gated_backward_ws_bytes(int M, int N) {
  if (M < 0 || N <= 0 || N % 8 != 0) return -1;
  return 4LL * M * N;
}

int gated_f16_backward(const void* dH, const void* X, const void* Wg, const void* Wu, const void* G, const void* U,
                       void* dX, void* dWg, void* dWu, void* workspace, int M, int N, int K, int dtype, int act,
                       void* stream) {
  if (int r = check_gated("gated_f16_backward", M, N, K, dtype, act)) return r;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (int r = check_pointers("gated_f16_backward", {Wg, Wu, dWg, dWu})) return r;
  if (M == 0) {
    const size_t bytes = static_cast<size_t>(N) * K * 2;
    cudaError_t e = cudaMemsetAsync(dWg, 0, bytes, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dWu, 0, bytes, s);
    if (e != cudaSuccess) return fgf8::set_error(FGF8_ERR_CUDA, "gated_f16_backward: %s", cudaGetErrorString(e));
    return FGF8_OK;
  }
  if (int r = check_pointers("gated_f16_backward", {dH, X, G, U, dX, workspace})) return r;
  const fgf8::GatedArgs a{M, N, K, dtype == FGF8_BF16, act};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return fgf8::launch_gated_backward(a, dH, X, Wg, Wu, G, U, dX, dWg, dWu, ws, ws + 2LL * M * N, s);
}

int gemv_fp4(const void* X, const void* Wq, const void* SF, void* Y, int M, int N, int K, int fmt, int dtype,
             void* stream) {
  if (int r = check_gemv("gemv_fp4", M, N, K, fmt, dtype)) return r;
  if (M == 0) return FGF8_OK;
  if (int r = check_pointers("gemv_fp4", {X, Wq, SF, Y})) return r;
  const fgf8::GemvArgs a{X, {Wq, nullptr}, {SF, nullptr}, Y, M, N, K, fmt, dtype == FGF8_BF16, -1};
  return fgf8::launch_gemv_fp4(a, static_cast<cudaStream_t>(stream));
}

int gated_gemv_fp4(const void* X, const void* WgQ, const void* SFg, const void* WuQ, const void* SFu, void* H, int M,
                   int N, int K, int fmt, int dtype, int act, void* stream) {
  if (int r = check_gemv("gated_gemv_fp4", M, N, K, fmt, dtype)) return r;
  if (act != FGF8_ACT_SILU && act != FGF8_ACT_GELU_TANH)
    return fgf8::set_error(FGF8_ERR_INVALID_ARG, "gated_gemv_fp4: bad activation %d", act);
  if (M == 0) return FGF8_OK;
  if (int r = check_pointers("gated_gemv_fp4", {X, WgQ, SFg, WuQ, SFu, H})) return r;
  const fgf8::GemvArgs a{X, {WgQ, WuQ}, {SFg, SFu}, H, M, N, K, fmt, dtype == FGF8_BF16, act};
  return fgf8::launch_gemv_fp4(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
