// dispatch.cu -- tokens to the rows of the grouped products and back, with their gradients.
//
//   dispatch_f16            Xs[rows[t][j]] = X[t], the other rows zero
//   dispatch_fp8            the same with 1x128 quantization to E4M3 on the way
//   combine_f16             Y[t] = sum_j W[t][j] Ys[rows[t][j]]        (dispatch_f16_backward: W = 1)
//   combine_f16_backward    dYs[rows[t][j]] = W[t][j] dY[t], dW[t][j] = <dY[t], Ys[rows[t][j]]>
//
// All four are HBM-bound streams in token order: a token's row is read (and quantized) once
// for its k copies, and the k rows that make up a token are read together, so every byte
// moves once.  In row order the same work would read X k times.
#include <cstring>

#include "activation.cuh"
#include "gemm_persistent.cuh"
#include "per_device.h"
#include "quant_common.cuh"
#include "routed.h"

namespace fgf8 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ void st_global_v4(void* p, const uint4& v) { *static_cast<uint4*>(p) = v; }

// Row of entry (t, j), -1 for none; one past the layout is reported and not used.
__device__ __forceinline__ int load_row(const RowsArgs& a, long long entry) {
  const int row = ptx::ld_global(a.rows + entry);
  if (row >= -1 && row < a.M) return row;
  atomicOr(a.status, FGF8_DEVERR_INPUT);
  return -1;
}
// Rows of up to 32 entries of token t from j0 on, one per lane (-1 past the last).
__device__ __forceinline__ int load_rows(const RowsArgs& a, int t, int j0, int lane) {
  return j0 + lane < a.k ? load_row(a, static_cast<long long>(t) * a.k + j0 + lane) : -1;
}

// Rows that no entry owns, of the 32 from r0 on, as a mask.
__device__ __forceinline__ uint32_t empty_rows(const RowsArgs& a, int r0, int lane) {
  const bool empty = r0 + lane < a.M && ptx::ld_global(a.src + r0 + lane) < 0;
  return __ballot_sync(kFull, empty);
}

// ----------------------------------------------------------------- dispatch, 16 bits
// A warp's item is 2 KB of a token (four 16-byte loads in flight per lane), written to its
// k rows; behind the tokens, 2 KB of each of 32 rows of the layout that are zeros if no
// entry owns them.
constexpr int kPart = 4;                        // 16-byte pieces per lane and item

__global__ void __launch_bounds__(kThreads) dispatch_f16_kernel(RowsArgs a, const uint4* __restrict__ X,
                                                                uint4* __restrict__ Xs) {
  ptx::griddep_wait();                          // everything may come from the previous kernel
  ptx::griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int vecs = a.H / 8, parts = (vecs + 32 * kPart - 1) / (32 * kPart);
  const long long tokens = static_cast<long long>(a.T) * parts;
  const long long items = tokens + (a.src != nullptr ? (static_cast<long long>(a.M) + 31) / 32 * parts : 0);
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += step) {
    if (it < tokens) {
      const int t = static_cast<int>(it / parts), v0 = static_cast<int>(it % parts) * 32 * kPart + lane;
      uint4 v[kPart];
#pragma unroll
      for (int u = 0; u < kPart; ++u)
        if (v0 + 32 * u < vecs) v[u] = ptx::ld_global_v4(X + static_cast<size_t>(t) * vecs + v0 + 32 * u);
      for (int j0 = 0; j0 < a.k; j0 += 32) {
        const int rows = load_rows(a, t, j0, lane);
        for (int j = 0; j < 32 && j0 + j < a.k; ++j) {
          const int row = __shfl_sync(kFull, rows, j);
          if (row < 0) continue;
          uint4* out = Xs + static_cast<size_t>(row) * vecs + v0;
#pragma unroll
          for (int u = 0; u < kPart; ++u)
            if (v0 + 32 * u < vecs) st_global_v4(out + 32 * u, v[u]);
        }
      }
    } else {
      const long long z = it - tokens;
      const int r0 = static_cast<int>(z / parts) * 32, v0 = static_cast<int>(z % parts) * 32 * kPart + lane;
      for (uint32_t left = empty_rows(a, r0, lane); left != 0; left &= left - 1) {
        uint4* out = Xs + static_cast<size_t>(r0 + __ffs(left) - 1) * vecs + v0;
#pragma unroll
        for (int u = 0; u < kPart; ++u)
          if (v0 + 32 * u < vecs) st_global_v4(out + 32 * u, make_uint4(0u, 0u, 0u, 0u));
      }
    }
  }
}

// ----------------------------------------------------------------- dispatch, E4M3
// A warp's item is 512 elements of a token, quantized as quantize_1x128 does it (lanes
// 8 i .. 8 i + 7 hold K block i, 16 elements each), codes and scales written to its k rows.
template <bool UE8M0>
__global__ void __launch_bounds__(kThreads) dispatch_fp8_kernel(RowsArgs a, const uint4* __restrict__ X,
                                                                uint4* __restrict__ Xq, uint32_t* __restrict__ SF) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int nkb = a.H / 128, kq = (nkb + 3) / 4;
  const int per = a.slots > 0 ? a.slots : a.M;             // rows of one scale table
  const size_t ld = (static_cast<size_t>(per) + 3) / 4 * 4;
  const size_t table = ld * (UE8M0 ? kq : nkb);
  const long long items = static_cast<long long>(a.T) * kq;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += step) {
    const int t = static_cast<int>(it / kq), qw = static_cast<int>(it % kq);
    const int kb = 4 * qw + (lane >> 3);
    const bool active = kb < nkb;
    float f0[8], f1[8];
    float amax = 0.0f;
    if (active) {
      const uint4* src = X + (static_cast<size_t>(t) * a.H + static_cast<size_t>(qw) * 512 + 16 * lane) / 8;
      const uint4 w0 = ptx::ld_global_v4(src), w1 = ptx::ld_global_v4(src + 1);
      quant::unpack8(w0, f0);
      quant::unpack8(w1, f1);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(f0[i]), fabsf(f1[i])));
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, off));
    float s = 1.0f, inv = 1.0f;
    uint32_t word = 0;                                     // what this lane writes to the scale table
    if (UE8M0) {
      const int e = quant::ue8m0_exponent(amax);
      inv = quant::exp2_neg(e);
      const uint32_t byte = active ? static_cast<uint32_t>(e + 127) : 0u;
      word = byte | (__shfl_sync(kFull, byte, 8) << 8) | (__shfl_sync(kFull, byte, 16) << 16) | (__shfl_sync(kFull, byte, 24) << 24);
    } else {
      if (amax != 0.0f) s = __fdiv_rn(amax, quant::kE4M3Max);
      inv = quant::scale_reciprocal(s);
      word = __float_as_uint(s);
    }
    uint4 code = make_uint4(0u, 0u, 0u, 0u);
    if (active) {
      const uint2 lo = quant::quant8<UE8M0>(f0, s, inv), hi = quant::quant8<UE8M0>(f1, s, inv);
      code = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    const bool scales = UE8M0 ? lane == 0 : (lane & 7) == 0 && active;
    const size_t at = ld * (UE8M0 ? qw : kb);
    for (int j0 = 0; j0 < a.k; j0 += 32) {
      const int rows = load_rows(a, t, j0, lane);
      for (int j = 0; j < 32 && j0 + j < a.k; ++j) {
        const int row = __shfl_sync(kFull, rows, j);
        if (row < 0) continue;
        if (active) st_global_v4(Xq + (static_cast<size_t>(row) * a.H + static_cast<size_t>(qw) * 512 + 16 * lane) / 16, code);
        if (scales) SF[static_cast<size_t>(row / per) * table + at + row % per] = word;
      }
    }
  }
}

// ----------------------------------------------------------------- combine
// Eight 16-bit values as FP32.
template <bool BF16>
__device__ __forceinline__ void unpack16(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = act::to_float(u[i] & 0xFFFFu, BF16);
    f[2 * i + 1] = act::to_float(u[i] >> 16, BF16);
  }
}
__device__ __forceinline__ uint4 pack16(const float (&f)[8], bool bf16) {
  return make_uint4(pack_2x16(f[0], f[1], bf16), pack_2x16(f[2], f[3], bf16), pack_2x16(f[4], f[5], bf16), pack_2x16(f[6], f[7], bf16));
}

// A warp's item is 512 bytes of a token: 16 bytes per lane of each of its rows, up to
// kBatch rows in flight, added in FP32 in the order of j.
constexpr int kBatch = 8;

template <bool BF16, bool WEIGHTED>
__global__ void __launch_bounds__(kThreads) combine_f16_kernel(RowsArgs a, const uint4* __restrict__ Ys,
                                                               const float* __restrict__ W, uint4* __restrict__ Y) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int vecs = a.H / 8, parts = (vecs + 31) / 32;
  const long long items = static_cast<long long>(a.T) * parts;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += step) {
    const int t = static_cast<int>(it / parts), v = static_cast<int>(it % parts) * 32 + lane;
    float sum[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += 32) {
      const int rows = load_rows(a, t, j0, lane);
      float weights = 1.0f;
      if (WEIGHTED && j0 + lane < a.k) weights = ptx::ld_global(W + static_cast<long long>(t) * a.k + j0 + lane);
      const int n = min(32, a.k - j0);
      for (int j = 0; j < n; j += kBatch) {
        uint4 y[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int row = __shfl_sync(kFull, rows, (j + u) & 31);
          if (j + u < n && row >= 0 && v < vecs) y[u] = ptx::ld_global_v4(Ys + static_cast<size_t>(row) * vecs + v);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int row = __shfl_sync(kFull, rows, (j + u) & 31);
          const float w = WEIGHTED ? __shfl_sync(kFull, weights, (j + u) & 31) : 1.0f;
          if (j + u < n && row >= 0) {
            float f[8];
            unpack16<BF16>(y[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = WEIGHTED ? fmaf(w, f[i], sum[i]) : sum[i] + f[i];
          }
        }
      }
    }
    if (v < vecs) st_global_v4(Y + static_cast<size_t>(t) * vecs + v, pack16(sum, BF16));
  }
}

// ----------------------------------------------------------------- gradients of combine
// A CTA takes a token: its threads walk the row once for every kBatch entries, so dY is read
// from HBM once; the dot products are summed over lanes and warps in a fixed order.  Behind
// the tokens, rows without an entry are zeroed.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) combine_f16_backward_kernel(RowsArgs a, const uint4* __restrict__ dY,
                                                                        const uint4* __restrict__ Ys, const float* __restrict__ W,
                                                                        uint4* __restrict__ dYs, float* __restrict__ dW) {
  __shared__ float part[2][kWarps][kBatch];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5, warps = static_cast<int>(blockDim.x) >> 5;
  const int vecs = a.H / 8;
  int turn = 0;
  for (int t = static_cast<int>(blockIdx.x); t < a.T; t += static_cast<int>(gridDim.x)) {
    for (int j0 = 0; j0 < a.k; j0 += kBatch) {
      int row[kBatch];
      float w[kBatch], dot[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const long long entry = static_cast<long long>(t) * a.k + j0 + u;
        row[u] = j0 + u < a.k ? load_row(a, entry) : -1;
        w[u] = row[u] >= 0 ? ptx::ld_global(W + entry) : 0.0f;
        dot[u] = 0.0f;
      }
      for (int v = tid; v < vecs; v += static_cast<int>(blockDim.x)) {
        float d[8];
        const uint4 dv = ptx::ld_global_v4(dY + static_cast<size_t>(t) * vecs + v);
        uint4 y[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (row[u] >= 0) y[u] = ptx::ld_global_v4(Ys + static_cast<size_t>(row[u]) * vecs + v);
        unpack16<BF16>(dv, d);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (row[u] >= 0) {
            float f[8], g[8];
            unpack16<BF16>(y[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dot[u] = fmaf(d[i], f[i], dot[u]);
              g[i] = w[u] * d[i];
            }
            st_global_v4(dYs + static_cast<size_t>(row[u]) * vecs + v, pack16(g, BF16));
          }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot[u] += __shfl_xor_sync(kFull, dot[u], off);
        if (lane == 0) part[turn][warp][u] = dot[u];
      }
      __syncthreads();
      if (tid < kBatch && j0 + tid < a.k) {
        float s = 0.0f;
        for (int i = 0; i < warps; ++i) s += part[turn][i][tid];
        dW[static_cast<long long>(t) * a.k + j0 + tid] = s;
      }
      turn ^= 1;                                            // the next sums need no second barrier
    }
  }
  if (a.src == nullptr) return;
  const int blocks = static_cast<int>((static_cast<long long>(a.M) + 31) / 32);
  for (int b = static_cast<int>(blockIdx.x); b < blocks; b += static_cast<int>(gridDim.x))
    for (uint32_t left = empty_rows(a, 32 * b, lane); left != 0; left &= left - 1) {
      uint4* out = dYs + static_cast<size_t>(32 * b + __ffs(left) - 1) * vecs;
      for (int v = tid; v < vecs; v += static_cast<int>(blockDim.x)) st_global_v4(out + v, make_uint4(0u, 0u, 0u, 0u));
    }
}

// ----------------------------------------------------------------- launches
// Resident CTAs of a kernel on the current device.
template <typename... KArgs>
int resident(void (*kernel)(KArgs...), PerDevice<int>& cache, int* ctas) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  const int* n = nullptr;
  const int r = cache.get(dev, &n, [&](int& v) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kernel, kThreads, 0);
    if (e != cudaSuccess || v <= 0) return set_error(4, "dispatch occupancy: %s", cudaGetErrorString(e));
    v *= device_sm_count();
    return 0;
  });
  if (r == 0) *ctas = *n;
  return r;
}

template <typename... KArgs, typename... Args>
int launch(void (*kernel)(KArgs...), long long ctas, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
  return e == cudaSuccess ? 0 : set_error(4, "dispatch launch: %s", cudaGetErrorString(e));
}

// One resident wave of warps at most.
template <typename... KArgs, typename... Args>
int launch_items(void (*kernel)(KArgs...), PerDevice<int>& cache, long long items, cudaStream_t stream, Args... args) {
  int most = 0;
  if (const int r = resident(kernel, cache, &most)) return r;
  const long long ctas = (items + kWarps - 1) / kWarps;
  return launch(kernel, ctas < most ? ctas : most, kThreads, stream, args...);
}

}  // namespace

int launch_dispatch_f16(const RowsArgs& a, const void* X, void* Xs, cudaStream_t stream) {
  static PerDevice<int> cache;
  const long long parts = (a.H / 8 + 32 * kPart - 1) / (32 * kPart);
  const long long rows = a.T + (a.src != nullptr ? (static_cast<long long>(a.M) + 31) / 32 : 0);
  return launch_items(dispatch_f16_kernel, cache, rows * parts, stream, a, static_cast<const uint4*>(X), static_cast<uint4*>(Xs));
}

int launch_dispatch_fp8(const RowsArgs& a, const void* X, void* Xq, void* SFA, int fmt, cudaStream_t stream) {
  static PerDevice<int> cache[2];
  const long long items = static_cast<long long>(a.T) * ((a.H / 128 + 3) / 4);
  return launch_items(fmt ? dispatch_fp8_kernel<true> : dispatch_fp8_kernel<false>, cache[fmt ? 1 : 0], items, stream, a,
                      static_cast<const uint4*>(X), static_cast<uint4*>(Xq), static_cast<uint32_t*>(SFA));
}

int launch_combine_f16(const RowsArgs& a, const void* Ys, const float* W, void* Y, int bf16, cudaStream_t stream) {
  static PerDevice<int> cache[4];
  const long long items = static_cast<long long>(a.T) * ((a.H / 8 + 31) / 32);
  auto* fn = W != nullptr ? (bf16 ? combine_f16_kernel<true, true> : combine_f16_kernel<false, true>)
                          : (bf16 ? combine_f16_kernel<true, false> : combine_f16_kernel<false, false>);
  return launch_items(fn, cache[(bf16 ? 1 : 0) + (W != nullptr ? 2 : 0)], items, stream, a, static_cast<const uint4*>(Ys), W,
                      static_cast<uint4*>(Y));
}

int launch_combine_f16_backward(const RowsArgs& a, const void* dY, const void* Ys, const float* W, void* dYs, float* dW,
                                int bf16, cudaStream_t stream) {
  static PerDevice<int> cache[2];
  auto* fn = bf16 ? combine_f16_backward_kernel<true> : combine_f16_backward_kernel<false>;
  int most = 0;
  if (const int r = resident(fn, cache[bf16 ? 1 : 0], &most)) return r;
  // as few threads as walk the row in the same number of steps
  const int vecs = a.H / 8, steps = (vecs + kThreads - 1) / kThreads;
  const int threads = ((vecs + steps - 1) / steps + 31) / 32 * 32;
  const long long work = a.src != nullptr && (a.M + 31LL) / 32 > a.T ? (a.M + 31LL) / 32 : a.T;
  return launch(fn, work < most ? work : most, threads, stream, a, static_cast<const uint4*>(dY), static_cast<const uint4*>(Ys), W,
                static_cast<uint4*>(dYs), dW);
}

}  // namespace fgf8
