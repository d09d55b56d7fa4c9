// api_routed.cu -- the C ABI of the operators whose rows choose their own weights
// (include/fgf8.h): host-side validation and dispatch.
#include "../../include/fgf8.h"
#include "check.h"
#include "routed.h"

namespace {

using fgf8::check_pointers;
using fgf8::kRouteMaxSize;
using fgf8::set_error;

int check_entries(const char* who, int T, int k) {
  if (T < 0 || k < 1) return set_error(FGF8_ERR_INVALID_ARG, "%s: T=%d k=%d", who, T, k);
  if (static_cast<long long>(T) * k > kRouteMaxSize)
    return set_error(FGF8_ERR_UNSUPPORTED, "%s: T=%d k=%d: entries above %d", who, T, k, kRouteMaxSize);
  return FGF8_OK;
}

int check_groups(const char* who, int G) {
  if (G < 1) return set_error(FGF8_ERR_INVALID_ARG, "%s: G=%d", who, G);
  if (G > fgf8::kRouteMaxGroups)
    return set_error(FGF8_ERR_UNSUPPORTED, "%s: G=%d above %d", who, G, fgf8::kRouteMaxGroups);
  return FGF8_OK;
}

// T tokens with k entries each in a layout of M rows of H elements, H a multiple of `unit`.
int check_rows(const char* who, int T, int k, int H, int M, int unit) {
  if (int r = check_entries(who, T, k)) return r;
  if (H < 1 || M < 0) return set_error(FGF8_ERR_INVALID_ARG, "%s: row size %d, M=%d", who, H, M);
  if (H > kRouteMaxSize || M > kRouteMaxSize)
    return set_error(FGF8_ERR_UNSUPPORTED, "%s: row size %d, M=%d: sizes above %d", who, H, M, kRouteMaxSize);
  if (H % unit != 0) return set_error(FGF8_ERR_UNSUPPORTED, "%s: row size %d not a multiple of %d", who, H, unit);
  return FGF8_OK;
}

int check_dtype(const char* who, int dtype) {
  if (dtype != FGF8_F16 && dtype != FGF8_BF16) return set_error(FGF8_ERR_INVALID_ARG, "%s: bad dtype %d", who, dtype);
  return FGF8_OK;
}

int status_word(const char* who, uint32_t** word) {
  *word = fgf8::device_status_ptr();
  return *word != nullptr ? FGF8_OK : set_error(FGF8_ERR_CUDA, "%s: no device", who);
}

// p where it is looked at, else `other`, which is checked anyway: all pointers of a call are
// checked together, null pointers and alignment first.
const void* when(bool used, const void* p, const void* other) { return used ? p : other; }

int combine(const char* who, const void* Ys, const float* W, const int32_t* rows, void* Y, int T, int k, int N, int M,
            int dtype, void* stream) {
  if (int r = check_rows(who, T, k, N, M, 8)) return r;
  if (int r = check_dtype(who, dtype)) return r;
  if (T == 0) return FGF8_OK;
  if (int r = check_pointers(who, {when(M > 0, Ys, Y), when(W != nullptr, W, Y), rows, Y})) return r;
  fgf8::RowsArgs a{rows, nullptr, T, k, M, N, 0, nullptr};
  if (int r = status_word(who, &a.status)) return r;
  return fgf8::launch_combine_f16(a, Ys, W, Y, dtype == FGF8_BF16, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

// every group that has entries wastes at most align - 1 rows
long long fgf8_route_rows(int T, int k, int G, int align) {
  if (T < 0 || k < 1 || G < 1 || align < 1) return -1;
  const long long n = static_cast<long long>(T) * k, used = n < G ? n : G;
  return (n + used * (align - 1)) / align * align;
}

int route_contiguous(const void* ids, int32_t* rows, int32_t* src, int32_t* m_indices, int32_t* counts, int32_t* starts,
                     int T, int k, int G, int align, int M, int ids64, void* stream) {
  const char* who = "route_contiguous";
  if (int r = check_entries(who, T, k)) return r;
  if (int r = check_groups(who, G)) return r;
  if (align < 1 || M < 0 || M % align != 0) return set_error(FGF8_ERR_INVALID_ARG, "%s: M=%d rows in segments of %d", who, M, align);
  const long long need = fgf8_route_rows(T, k, G, align);
  if (need > M) return set_error(FGF8_ERR_INVALID_ARG, "%s: M=%d rows, %lld can be needed", who, M, need);
  if (M > kRouteMaxSize) return set_error(FGF8_ERR_UNSUPPORTED, "%s: M=%d above %d", who, M, kRouteMaxSize);
  if (int r = check_pointers(who, {when(T > 0, ids, counts), when(T > 0, rows, counts), when(M > 0, src, counts),
                                   when(M > 0, m_indices, counts), counts, starts}))
    return r;
  fgf8::RouteArgs a{ids, ids64 != 0, rows, src, m_indices, counts, starts, T * k, G, M, align, 0, nullptr};
  if (int r = status_word(who, &a.status)) return r;
  return fgf8::launch_route(a, static_cast<cudaStream_t>(stream));
}

int route_masked(const void* ids, int32_t* rows, int32_t* src, int32_t* masked_m, int T, int k, int G, int Mmax, int ids64,
                 void* stream) {
  const char* who = "route_masked";
  if (int r = check_entries(who, T, k)) return r;
  if (int r = check_groups(who, G)) return r;
  if (Mmax < 1) return set_error(FGF8_ERR_INVALID_ARG, "%s: Mmax=%d", who, Mmax);
  if (static_cast<long long>(G) * Mmax > kRouteMaxSize)
    return set_error(FGF8_ERR_UNSUPPORTED, "%s: G=%d Mmax=%d: rows above %d", who, G, Mmax, kRouteMaxSize);
  if (int r = check_pointers(who, {when(T > 0, ids, src), when(T > 0, rows, src), src, masked_m})) return r;
  fgf8::RouteArgs a{ids, ids64 != 0, rows, src, nullptr, masked_m, nullptr, T * k, G, G * Mmax, 1, Mmax, nullptr};
  if (int r = status_word(who, &a.status)) return r;
  return fgf8::launch_route(a, static_cast<cudaStream_t>(stream));
}

int dispatch_f16(const void* X, const int32_t* rows, const int32_t* src, void* Xs, int T, int k, int K, int M, void* stream) {
  const char* who = "dispatch_f16";
  if (int r = check_rows(who, T, k, K, M, 8)) return r;
  if (M == 0 || (T == 0 && src == nullptr)) return FGF8_OK;
  if (int r = check_pointers(who, {when(T > 0, X, Xs), when(T > 0, rows, Xs), when(src != nullptr, src, Xs), Xs})) return r;
  fgf8::RowsArgs a{rows, src, T, k, M, K, 0, nullptr};
  if (int r = status_word(who, &a.status)) return r;
  return fgf8::launch_dispatch_f16(a, X, Xs, static_cast<cudaStream_t>(stream));
}

int dispatch_fp8(const void* X, const int32_t* rows, void* Xq, void* SFA, int T, int k, int K, int M, int Mmax, int fmt,
                 void* stream) {
  const char* who = "dispatch_fp8";
  if (int r = check_rows(who, T, k, K, M, 128)) return r;
  if (fmt != FGF8_SCALE_F32 && fmt != FGF8_SCALE_UE8M0) return set_error(FGF8_ERR_INVALID_ARG, "%s: bad scale format %d", who, fmt);
  if (Mmax < 0 || (Mmax > 0 && M % Mmax != 0)) return set_error(FGF8_ERR_INVALID_ARG, "%s: M=%d rows in slots of %d", who, M, Mmax);
  if (T == 0 || M == 0) return FGF8_OK;
  if (int r = check_pointers(who, {X, rows, Xq, SFA})) return r;
  fgf8::RowsArgs a{rows, nullptr, T, k, M, K, Mmax, nullptr};
  if (int r = status_word(who, &a.status)) return r;
  return fgf8::launch_dispatch_fp8(a, X, Xq, SFA, fmt, static_cast<cudaStream_t>(stream));
}

int combine_f16(const void* Ys, const float* W, const int32_t* rows, void* Y, int T, int k, int N, int M, int dtype, void* stream) {
  return combine("combine_f16", Ys, W, rows, Y, T, k, N, M, dtype, stream);
}

int dispatch_f16_backward(const void* dXs, const int32_t* rows, void* dX, int T, int k, int K, int M, int dtype, void* stream) {
  return combine("dispatch_f16_backward", dXs, nullptr, rows, dX, T, k, K, M, dtype, stream);
}

int combine_f16_backward(const void* dY, const void* Ys, const float* W, const int32_t* rows, const int32_t* src, void* dYs,
                         float* dW, int T, int k, int N, int M, int dtype, void* stream) {
  const char* who = "combine_f16_backward";
  if (int r = check_rows(who, T, k, N, M, 8)) return r;
  if (int r = check_dtype(who, dtype)) return r;
  if (T == 0 && (M == 0 || src == nullptr)) return FGF8_OK;
  const void* any = T > 0 ? dY : dYs;
  if (int r = check_pointers(who, {any, when(M > 0, Ys, any), when(T > 0, W, any), when(T > 0, rows, any),
                                   when(src != nullptr && M > 0, src, any), when(M > 0, dYs, any), when(T > 0, dW, any)}))
    return r;
  fgf8::RowsArgs a{rows, M > 0 ? src : nullptr, T, k, M, N, 0, nullptr};
  if (int r = status_word(who, &a.status)) return r;
  return fgf8::launch_combine_f16_backward(a, dY, Ys, W, dYs, dW, dtype == FGF8_BF16, static_cast<cudaStream_t>(stream));
}

int lora_f16(const void* X, const void* A, const void* B, const float* scale, const void* base, const int32_t* rows,
             const int32_t* src, const int32_t* m_indices, void* out, int T, int K, int N, int r, int G, int M, int align,
             long long ldx, long long ldb, long long ldo, int dtype, void* stream) {
  const char* who = "lora_f16";
  if (int e = check_rows(who, T, 1, K, M, 8)) return e;
  if (int e = check_rows(who, T, 1, N, M, 8)) return e;
  if (int e = check_dtype(who, dtype)) return e;
  if (r < 1 || G < 1) return set_error(FGF8_ERR_INVALID_ARG, "%s: r=%d G=%d", who, r, G);
  if (r % 8 != 0 || r > 128) return set_error(FGF8_ERR_UNSUPPORTED, "%s: rank %d not a multiple of 8 up to 128", who, r);
  if (align < 16 || align % 16 != 0) return set_error(FGF8_ERR_UNSUPPORTED, "%s: align=%d not a multiple of 16", who, align);
  if (M % align != 0) return set_error(FGF8_ERR_INVALID_ARG, "%s: M=%d not a multiple of align=%d", who, M, align);
  if (ldx < K || ldo < N || (base != nullptr && ldb < N))
    return set_error(FGF8_ERR_INVALID_ARG, "%s: rows of X, base and out are %lld, %lld and %lld apart", who, ldx, ldb, ldo);
  if (ldx % 8 != 0 || ldo % 8 != 0 || (base != nullptr && ldb % 8 != 0))
    return set_error(FGF8_ERR_MISALIGNED, "%s: row distances must be multiples of 8", who);
  if (base == out && ldb != ldo) return set_error(FGF8_ERR_INVALID_ARG, "%s: base is out with another row distance", who);
  if (T == 0) return FGF8_OK;
  if (M == 0) return set_error(FGF8_ERR_INVALID_ARG, "%s: no rows for T=%d tokens", who, T);
  if (int e = check_pointers(who, {X, A, B, when(scale != nullptr, scale, X), when(base != nullptr, base, X), rows, src,
                                   m_indices, out}))
    return e;
  fgf8::LoraArgs a{X, A, B, scale, base, out, rows, src, m_indices, ldx, ldb, ldo, T, K, N, r, G, M, align, nullptr};
  if (int e = status_word(who, &a.status)) return e;
  return fgf8::launch_lora_f16(a, dtype == FGF8_BF16, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
