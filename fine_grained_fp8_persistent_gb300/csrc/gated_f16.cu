// gated_f16.cu -- the gated feed-forward block in 16-bit types and its backward pass.
//
// Forward:   G = X Wg^T, U = X Wu^T, H = a(G) * U.
// Backward:  dG = dH * U * a'(G), dU = dH * a(G); dX = dG Wg + dU Wu,
//            dWg = dG^T X, dWu = dU^T X.
#include <cstring>

#include "activation.cuh"
#include "gated.h"

namespace fgf8 {
namespace {

// A strided view of a 16-bit matrix: element (i, k) at base[i * si + k * sk].
struct View {
  const uint16_t* p;
  long long si, sk;
  __device__ __forceinline__ float at(int i, int k, int ni, int nk, bool bf16) const {
    return i < ni && k < nk ? act::to_float(p[i * si + k * sk], bf16) : 0.0f;
  }
};

constexpr int kTile = 64, kDepth = 16;

// One 64 x 64 tile per CTA of 256 threads, 4 x 4 outputs per thread and accumulator.
// GATED: acc[0] = A B0^T, acc[1] = A B1^T, out = a(acc[0]) * acc[1]; else
// out = A0 B0^T + A1 B1^T (the second product only when nk1 > 0).
template <bool GATED>
__global__ void __launch_bounds__(256) tile_kernel(View a0, View b0, View a1, View b1, int M, int N, int K, int terms,
                                                   uint16_t* out, uint16_t* g, uint16_t* u, bool bf16, int act_code) {
  __shared__ float sa[kDepth][kTile + 1], sb[2][kDepth][kTile + 1];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  float acc[2][4][4] = {};
  for (int term = 0; term < (GATED ? 1 : terms); ++term) {
    const View a = term ? a1 : a0, b = term ? b1 : b0;
    for (int k0 = 0; k0 < K; k0 += kDepth) {
      for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
        const int r = i / kDepth, k = i % kDepth;
        sa[k][r] = a.at(m0 + r, k0 + k, M, K, bf16);
        sb[0][k][r] = b.at(n0 + r, k0 + k, N, K, bf16);
        if (GATED) sb[1][k][r] = b1.at(n0 + r, k0 + k, N, K, bf16);
      }
      __syncthreads();
      for (int k = 0; k < kDepth; ++k)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) {
            acc[0][i][j] = fmaf(sa[k][ty + 16 * i], sb[0][k][tx + 16 * j], acc[0][i][j]);
            if (GATED) acc[1][i][j] = fmaf(sa[k][ty + 16 * i], sb[1][k][tx + 16 * j], acc[1][i][j]);
          }
      __syncthreads();
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= M || n >= N) continue;
      const size_t at = static_cast<size_t>(m) * N + n;
      float v = acc[0][i][j];
      if (GATED) {
        if (g != nullptr) {
          g[at] = act::from_float(v, bf16);
          u[at] = act::from_float(acc[1][i][j], bf16);
        }
        v = (act_code == act::kSilu ? act::value<act::kSilu>(v) : act::value<act::kGeluTanh>(v)) * acc[1][i][j];
      }
      out[at] = act::from_float(v, bf16);
    }
}

// dG, dU from dH, G, U.  Eight elements (16 bytes) per thread; n8 = M * N / 8.
template <int ACT>
__global__ void __launch_bounds__(256) slope_kernel(const uint4* __restrict__ dh, const uint4* __restrict__ g,
                                                    const uint4* __restrict__ u, uint4* __restrict__ dg,
                                                    uint4* __restrict__ du, long long n8, bool bf16) {
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n8; i += gridDim.x * 256LL) {
    const uint4 a = dh[i], b = g[i], c = u[i];
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w}, cw[4] = {c.x, c.y, c.z, c.w};
    uint32_t gw[4], uw[4];
    for (int j = 0; j < 4; ++j) {
      uint32_t go = 0, uo = 0;
      for (int h = 0; h < 2; ++h) {
        const float d = act::to_float(aw[j] >> (16 * h) & 0xFFFFu, bf16);
        float v, s;
        act::value_slope<ACT>(act::to_float(bw[j] >> (16 * h) & 0xFFFFu, bf16), v, s);
        go |= static_cast<uint32_t>(act::from_float(d * act::to_float(cw[j] >> (16 * h) & 0xFFFFu, bf16) * s, bf16)) << (16 * h);
        uo |= static_cast<uint32_t>(act::from_float(d * v, bf16)) << (16 * h);
      }
      gw[j] = go;
      uw[j] = uo;
    }
    dg[i] = make_uint4(gw[0], gw[1], gw[2], gw[3]);
    du[i] = make_uint4(uw[0], uw[1], uw[2], uw[3]);
  }
}

int check_launch(const char* who) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? 0 : set_error(4, "%s launch: %s", who, cudaGetErrorString(e));
}

dim3 tiles(int M, int N) { return dim3((N + kTile - 1) / kTile, (M + kTile - 1) / kTile); }
const uint16_t* u16(const void* p) { return static_cast<const uint16_t*>(p); }

}  // namespace

int launch_gated_forward(const GatedArgs& a, const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                         cudaStream_t stream) {
  const View x{u16(X), a.K, 1}, wg{u16(Wg), a.K, 1}, wu{u16(Wu), a.K, 1};
  tile_kernel<true><<<tiles(a.M, a.N), 256, 0, stream>>>(x, wg, x, wu, a.M, a.N, a.K, 1, static_cast<uint16_t*>(H),
                                                         static_cast<uint16_t*>(G), static_cast<uint16_t*>(U), a.bf16 != 0, a.act);
  return check_launch("gated_f16");
}

int launch_gated_backward(const GatedArgs& a, const void* dH, const void* X, const void* Wg, const void* Wu,
                          const void* G, const void* U, void* dX, void* dWg, void* dWu, void* dG, void* dU,
                          cudaStream_t stream) {
  const long long n8 = static_cast<long long>(a.M) * a.N / 8;
  const long long want = (n8 + 255) / 256, cap = 8LL * device_sm_count();
  const int grid = static_cast<int>(want < cap ? want : cap);
  auto* k = a.act == act::kSilu ? slope_kernel<act::kSilu> : slope_kernel<act::kGeluTanh>;
  k<<<grid, 256, 0, stream>>>(static_cast<const uint4*>(dH), static_cast<const uint4*>(G), static_cast<const uint4*>(U),
                              static_cast<uint4*>(dG), static_cast<uint4*>(dU), n8, a.bf16 != 0);
  if (int r = check_launch("gated_f16_backward")) return r;
  // dX[m][k] = sum_n dG[m][n] Wg[n][k] + dU[m][n] Wu[n][k]
  const View dg{u16(dG), a.N, 1}, du{u16(dU), a.N, 1}, wgt{u16(Wg), 1, a.K}, wut{u16(Wu), 1, a.K};
  tile_kernel<false><<<tiles(a.M, a.K), 256, 0, stream>>>(dg, wgt, du, wut, a.M, a.K, a.N, 2, static_cast<uint16_t*>(dX),
                                                          nullptr, nullptr, a.bf16 != 0, a.act);
  // dW[n][k] = sum_m dG[m][n] X[m][k]
  const View xt{u16(X), 1, a.K}, dgt{u16(dG), 1, a.N}, dut{u16(dU), 1, a.N};
  tile_kernel<false><<<tiles(a.N, a.K), 256, 0, stream>>>(dgt, xt, dgt, xt, a.N, a.K, a.M, 1, static_cast<uint16_t*>(dWg),
                                                          nullptr, nullptr, a.bf16 != 0, a.act);
  tile_kernel<false><<<tiles(a.N, a.K), 256, 0, stream>>>(dut, xt, dut, xt, a.N, a.K, a.M, 1, static_cast<uint16_t*>(dWu),
                                                          nullptr, nullptr, a.bf16 != 0, a.act);
  return check_launch("gated_f16_backward");
}

}  // namespace fgf8
