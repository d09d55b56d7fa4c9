// gated_f16.cu -- the gated feed-forward block in 16-bit types and its backward pass.
//
// Forward:   G = X Wg^T, U = X Wu^T, H = a(G) * U, one launch.
// Backward:  dG = dH * U * a'(G), dU = dH * a(G) element by element, then
//            dX = dG Wg + dU Wu, dWg = dG^T X and dWu = dU^T X in one launch.
// The products are gated_gemm.cuh's; this file holds the elementwise kernel, the tensor
// maps, the choice of tile and the launches.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "activation.cuh"
#include "gated.h"
#include "gated_gemm.cuh"
#include "gated_thin.cuh"
#include "per_device.h"

namespace fgf8 {
namespace {

// dG, dU from dH, G, U.  Eight elements (16 bytes) per thread; n8 = M * N / 8.  A stream of
// three reads and two writes, bound by memory latency: 13.5 us at 4096 x 2048 (84 MB).
template <int ACT, bool BF16>
__global__ void __launch_bounds__(256) slope_kernel(const uint4* __restrict__ dh, const uint4* __restrict__ g,
                                                    const uint4* __restrict__ u, uint4* __restrict__ dg,
                                                    uint4* __restrict__ du, long long n8) {
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n8; i += gridDim.x * 256LL) {
    const uint4 a = dh[i], b = g[i], c = u[i];
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w}, cw[4] = {c.x, c.y, c.z, c.w};
    uint32_t gw[4], uw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float dgv[2], duv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float d = act::to_float((aw[j] >> (16 * h)) & 0xFFFFu, BF16);
        float v, s;
        act::value_slope<ACT>(act::to_float((bw[j] >> (16 * h)) & 0xFFFFu, BF16), v, s);
        dgv[h] = d * act::to_float((cw[j] >> (16 * h)) & 0xFFFFu, BF16) * s;
        duv[h] = d * v;
      }
      gw[j] = pack_2x16(dgv[0], dgv[1], BF16);
      uw[j] = pack_2x16(duv[0], duv[1], BF16);
    }
    dg[i] = make_uint4(gw[0], gw[1], gw[2], gw[3]);
    du[i] = make_uint4(uw[0], uw[1], uw[2], uw[3]);
  }
}

// ----------------------------------------------------------------- launches
// Launch configuration with a cluster of `cluster` CTAs and, for the forward pass when
// enabled, programmatic stream serialization.
struct Launch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  Launch(unsigned grid, unsigned threads, size_t smem, int cluster, cudaStream_t stream, bool pdl) {
    std::memset(&cfg, 0, sizeof(cfg));
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
  }
};

// Time of one tile beside its K blocks (set-up and the part of the epilogue that no other
// tile's MMAs cover), in K blocks.
constexpr int kTileCost = 6;

template <GatedOp OP, int ACT, int NCTA, int BN, int STAGES>
int launch_gemm(const GatedMaps& tm, GatedGemmArgs args, cudaStream_t stream) {
  using C = GatedCfg<OP, NCTA, BN, STAGES>;
  static_assert(C::SMEM_BYTES <= 232448, "shared memory budget");
  auto* fn = &gated_gemm<OP, ACT, NCTA, BN, STAGES>;
  static PerDevice<int> max_clusters;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  const int* fit = nullptr;
  const int r = max_clusters.get(dev, &fit, [&](int& clusters) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    clusters = device_sm_count();
    if (e == cudaSuccess && NCTA > 1) {
      Launch probe(static_cast<unsigned>(device_sm_count() / NCTA * NCTA), C::THREADS, C::SMEM_BYTES, NCTA, stream, false);
      e = cudaOccupancyMaxActiveClusters(&clusters, fn, &probe.cfg);
    }
    return e == cudaSuccess && clusters > 0 ? 0 : set_error(4, "gated_f16 occupancy: %s", cudaGetErrorString(e));
  });
  if (r) return r;
  auto up = [](long long v, long long by) { return (v + by - 1) / by; };
  const long long n1 = up(C::kFwd ? args.N : args.K, C::OUT_N);
  const long long tiles1 = up(args.M, C::TILE_M) * n1, tiles2 = C::kFwd ? 0 : 2 * up(args.N, C::TILE_M) * n1;
  if (tiles1 + tiles2 > 0x7F000000LL) return set_error(2, "gated_f16: problem too large");
  const long long clusters = persistent_clusters(tiles1 + tiles2, NCTA, device_sm_count(), *fit, C::kFwd && sm_cap_enabled());
  args.long_clusters = 0;
  args.early_tiles = 0;
  if (!C::kFwd && tiles1 % clusters != 0) {
    // the clusters without a last tile of dX do as many tiles of dWg, dWu as take its time
    const long long cost1 = 2 * up(args.N, 64) + kTileCost, cost2 = up(args.M, 64) + kTileCost;
    args.long_clusters = static_cast<int>(tiles1 % clusters);
    const long long early = (clusters - args.long_clusters) * (cost1 / cost2);
    args.early_tiles = static_cast<int>(early < tiles2 ? early : tiles2);
  }
  set_last_tile("f16", C::kFwd ? "gated" : "gated_grad", NCTA, BN);
  Launch l(static_cast<unsigned>(clusters * NCTA), C::THREADS, C::SMEM_BYTES, NCTA, stream, C::kFwd && pdl_enabled());
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, fn, tm, args);
  return e == cudaSuccess ? 0 : set_error(4, "gated_f16 launch: %s", cudaGetErrorString(e));
}

// A map of a row-major 16-bit matrix: K-major operand boxes of 64 columns x box_rows,
// or MN-major boxes of 64 x 64, both 128 bytes wide and swizzled.
bool operand_map(CUtensorMap* m, const GatedArgs& a, const void* p, long long rows, long long cols, int box_rows) {
  return encode_tmap_2d(m, a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p, cols, rows, cols * 2, 64,
                        box_rows, true);
}
bool output_map(CUtensorMap* m, const void* p, long long rows, long long cols, int box_cols) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, p, cols, rows, cols * 2, box_cols, 32, false);
}

int gemm_args(GatedGemmArgs& g, const GatedArgs& a) {
  std::memset(&g, 0, sizeof(g));
  g.M = a.M;
  g.N = a.N;
  g.K = a.K;
  g.a_box_rows = a.M >= 128 ? 128 : (a.M + 7) / 8 * 8;
  g.bf16 = a.bf16;
  g.status = device_status_ptr();
  g.timeout_ns = wait_timeout_ns();
  return g.status ? 0 : 4;
}

// One tile configuration and its relative time.
struct Choice {
  int ncta, bn;
  double t_kb;
};
// The candidate that FGF8_FORCE_TILE="<ctas per cluster>x<bn>" names; -1: none of these.
int forced(const Choice* c, int n) {
  if (const char* f = std::getenv("FGF8_FORCE_TILE")) {
    int nc = 0, bn = 0;
    char more = 0;                                         // a suffix names a tile of another kernel
    if (std::sscanf(f, "%dx%d%c", &nc, &bn, &more) == 2)
      for (int i = 0; i < n; ++i)
        if (c[i].ncta == nc && c[i].bn == bn) return i;
  }
  return -1;
}
// The thin forward pass (gated_thin.cuh): shares S of the reduction per tile of 64 weight
// rows and its time in units of 128-byte rows through one CTA's copy engine.
struct ThinPlan {
  int S, cta_kb;
  double cost;
};
template <int ACT>
int plan_thin(ThinPlan& p, const GatedArgs& a) {
  struct Fit {
    int clusters[9];                                       // by S: clusters that fit
  };
  static PerDevice<Fit> fits;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  const Fit* fit = nullptr;
  const int r = fits.get(dev, &fit, [](Fit& f) {
    auto* fn = &gated_thin<ACT>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, thin::kSmemCap);
    for (int s = 8; e == cudaSuccess && s >= 1; --s) {
      Launch l(static_cast<unsigned>(device_sm_count() / s * s), thin::kThreads, thin::kSmemCap, s, nullptr, false);
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, fn, &l.cfg);
      if (e == cudaSuccess && n <= 0) e = cudaErrorInvalidConfiguration;
      f.clusters[s] = n;
    }
    return e == cudaSuccess ? 0 : set_error(4, "gated_f16 occupancy: %s", cudaGetErrorString(e));
  });
  if (r) return r;
  const int tiles = (a.N + thin::kRows - 1) / thin::kRows, nkb = (a.K + 63) / 64, nb = (a.M + 15) / 16 * 16;
  p.cost = -1.0;
  for (int s = 1; s <= 8; ++s) {
    const int per = (nkb + s - 1) / s;
    if ((s - 1) * per >= nkb) continue;                    // a CTA without work
    const int waves = (tiles + fit->clusters[s] - 1) / fit->clusters[s];
    const double t = waves * (static_cast<double>(per) * (128 + nb) + (s > 1 ? 1500.0 : 500.0));
    if (p.cost < 0 || t < p.cost) {
      p.S = s;
      p.cta_kb = per;
      p.cost = t;
    }
  }
  return 0;
}

template <int ACT>
int launch_thin(const ThinPlan& p, const GatedArgs& a, const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                cudaStream_t stream) {
  GatedThinArgs t;
  std::memset(&t, 0, sizeof(t));
  t.M = a.M;
  t.N = a.N;
  t.K = a.K;
  t.nb = (a.M + 15) / 16 * 16;
  const int stage = thin::kABytes + t.nb * 128;
  const int fit = (thin::kSmemCap - 1024) / stage / thin::kKpu * thin::kKpu;
  t.stages = fit < thin::kMaxStages ? fit : thin::kMaxStages;
  t.cta_kb = p.cta_kb;
  t.bf16 = a.bf16;
  t.out = H;
  t.keep[0] = G;
  t.keep[1] = U;
  t.status = device_status_ptr();
  t.timeout_ns = wait_timeout_ns();
  if (!t.status) return 4;
  CUtensorMap tx, tg, tu;
  if (!operand_map(&tx, a, X, a.M, a.K, t.nb) || !operand_map(&tg, a, Wg, a.N, a.K, thin::kRows) || !operand_map(&tu, a, Wu, a.N, a.K, thin::kRows))
    return 4;
  const int tiles = (a.N + thin::kRows - 1) / thin::kRows;
  set_last_tile("f16", "gated_thin", p.S, t.nb);
  Launch l(static_cast<unsigned>(tiles * p.S), thin::kThreads, 1024 + static_cast<size_t>(t.stages) * stage, p.S, stream, pdl_enabled());
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, &gated_thin<ACT>, tx, tg, tu, t);
  return e == cudaSuccess ? 0 : set_error(4, "gated_f16 launch: %s", cudaGetErrorString(e));
}

template <int ACT>
int forward(const GatedArgs& a, const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U, cudaStream_t stream) {
  // time of a tile per K block, in 128-byte rows that a CTA copies (1.0 to 1.4 ns): the
  // rows loaded bound the one-CTA tiles, the MMA the pair (512 tokens at 7168 x 2048, one
  // wave each: 40 us on 2 x 256, 32 on 1 x 128, 48 for two waves of 1 x 64; 331 tokens at
  // 1800 x 2744: 18.1, 15.9 and 21.7 us)
  static const Choice c[] = {{2, 256, 320.0}, {1, 128, 256.0}, {1, 64, 200.0}};
  int best = 0;
  double cost = -1.0;
  for (int i = 0; i < 3; ++i) {
    const long long tm = 128LL * c[i].ncta, tn = c[i].bn / 2;
    const long long tiles = ((a.M + tm - 1) / tm) * ((a.N + tn - 1) / tn), units = device_sm_count() / c[i].ncta;
    const double t = static_cast<double>((tiles + units - 1) / units) * c[i].t_kb;
    if (cost < 0 || t < cost) {
      cost = t;
      best = i;
    }
  }
  const int kb = (a.K + 63) / 64, force = forced(c, 3);
  if (a.M <= 256 && force < 0) {
    ThinPlan p;
    if (int r = plan_thin<ACT>(p, a)) return r;
    if (p.cost < cost * kb + 500.0) return launch_thin<ACT>(p, a, X, Wg, Wu, H, G, U, stream);
  }
  const Choice& ch = c[force >= 0 ? force : best];
  GatedGemmArgs g;
  if (gemm_args(g, a)) return 4;
  g.save = G != nullptr;
  GatedMaps tm;
  std::memset(&tm, 0, sizeof(tm));
  const int half = ch.bn / 2, cw = half / 2 < 32 ? half / 2 : 32;   // columns of a staged output chunk
  if (!operand_map(&tm.a[0], a, X, a.M, a.K, g.a_box_rows) || !operand_map(&tm.b[0], a, Wg, a.N, a.K, half) ||
      !operand_map(&tm.b[1], a, Wu, a.N, a.K, half) || !output_map(&tm.d[0], H, a.M, a.N, cw))
    return 4;
  if (g.save && (!output_map(&tm.d[1], G, a.M, a.N, cw) || !output_map(&tm.d[2], U, a.M, a.N, cw))) return 4;
  if (ch.ncta == 2) return launch_gemm<GatedOp::Forward, ACT, 2, 256, 6>(tm, g, stream);
  if (ch.bn == 128) return launch_gemm<GatedOp::Forward, ACT, 1, 128, 6>(tm, g, stream);
  return launch_gemm<GatedOp::Forward, ACT, 1, 64, 8>(tm, g, stream);
}

int grads(const GatedArgs& a, const void* dG, const void* dU, const void* X, const void* Wg, const void* Wu, void* dX, void* dWg, void* dWu,
          cudaStream_t stream) {
  // Time of the launch in 128-byte rows that a CTA copies (1.0 to 1.4 ns): the longer of
  // one dX tile's reduction and an SM's share of all tiles; a tile's stores and set-up
  // count as `t_kb` further rows.  Measured (us) on 2x256 / 1x128 / 1x64: 17 x 7168 x 2048
  // 36.1 / 36.6 / 40.7, 67 x 2048 x 1368 24.3 / 21.3 / 19.2, 100 x 2048 x 8192 95 / 86 / 75,
  // 512 x 7168 x 2048 52 / 72 / 109, 1000 x 4096 x 4096 92 / 144 / 231.
  static const Choice c[] = {{2, 256, 2300.0}, {1, 128, 1300.0}, {1, 64, 750.0}};
  double cost = -1.0;
  int best = 0;
  const double a_rows = a.M >= 128 ? 128.0 : (a.M + 7) / 8 * 8;
  for (int i = 0; i < 3; ++i) {
    auto up = [](double v, double by) { return std::ceil(v / by); };
    const double units = device_sm_count() / c[i].ncta, b_rows = c[i].bn / c[i].ncta;
    const double n1 = up(a.K, c[i].bn), t1 = up(a.M, 128.0 * c[i].ncta) * n1, t2 = 2 * up(a.N, 128.0 * c[i].ncta) * n1;
    const double c1 = 2 * up(a.N, 64) * (a_rows + b_rows) + c[i].t_kb, c2 = up(a.M, 64) * (128.0 + b_rows) + c[i].t_kb;
    const double whole = (t1 * c1 + t2 * c2) / units, longest = c1 > whole ? c1 : whole;
    if (cost < 0 || longest < cost) {
      cost = longest;
      best = i;
    }
  }
  const int force = forced(c, 3);
  if (force >= 0) best = force;
  GatedGemmArgs g;
  if (gemm_args(g, a)) return 4;
  GatedMaps tm;
  std::memset(&tm, 0, sizeof(tm));
  if (!operand_map(&tm.a[0], a, dG, a.M, a.N, g.a_box_rows) || !operand_map(&tm.a[1], a, dU, a.M, a.N, g.a_box_rows) ||
      !operand_map(&tm.at[0], a, dG, a.M, a.N, 64) || !operand_map(&tm.at[1], a, dU, a.M, a.N, 64) || !operand_map(&tm.b[0], a, Wg, a.N, a.K, 64) ||
      !operand_map(&tm.b[1], a, Wu, a.N, a.K, 64) || !operand_map(&tm.b[2], a, X, a.M, a.K, 64) || !output_map(&tm.d[0], dX, a.M, a.K, 32) ||
      !output_map(&tm.d[1], dWg, a.N, a.K, 32) || !output_map(&tm.d[2], dWu, a.N, a.K, 32))
    return 4;
  if (c[best].ncta == 2) return launch_gemm<GatedOp::Grad, act::kSilu, 2, 256, 6>(tm, g, stream);
  if (c[best].bn == 64) return launch_gemm<GatedOp::Grad, act::kSilu, 1, 64, 8>(tm, g, stream);
  return launch_gemm<GatedOp::Grad, act::kSilu, 1, 128, 6>(tm, g, stream);
}

template <int ACT>
int slopes(const GatedArgs& a, const void* dH, const void* G, const void* U, void* dG, void* dU, cudaStream_t stream) {
  const long long n8 = static_cast<long long>(a.M) * a.N / 8;
  const long long want = (n8 + 255) / 256, cap = 8LL * device_sm_count();
  Launch l(static_cast<unsigned>(want < cap ? want : cap), 256, 0, 1, stream, false);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, a.bf16 ? slope_kernel<ACT, true> : slope_kernel<ACT, false>, static_cast<const uint4*>(dH),
                                           static_cast<const uint4*>(G), static_cast<const uint4*>(U), static_cast<uint4*>(dG),
                                           static_cast<uint4*>(dU), n8);
  return e == cudaSuccess ? 0 : set_error(4, "gated_f16_backward launch: %s", cudaGetErrorString(e));
}

}  // namespace

int launch_gated_forward(const GatedArgs& a, const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                         cudaStream_t stream) {
  if (a.M <= kGemvMaxRows) return launch_gated_gemv_f16(a, X, Wg, Wu, H, G, U, stream);
  return a.act == act::kSilu ? forward<act::kSilu>(a, X, Wg, Wu, H, G, U, stream) : forward<act::kGeluTanh>(a, X, Wg, Wu, H, G, U, stream);
}

int launch_gated_backward(const GatedArgs& a, const void* dH, const void* X, const void* Wg, const void* Wu,
                          const void* G, const void* U, void* dX, void* dWg, void* dWu, void* dG, void* dU,
                          cudaStream_t stream) {
  int r = a.act == act::kSilu ? slopes<act::kSilu>(a, dH, G, U, dG, dU, stream) : slopes<act::kGeluTanh>(a, dH, G, U, dG, dU, stream);
  if (r == 0) r = grads(a, dG, dU, X, Wg, Wu, dX, dWg, dWu, stream);
  return r;
}

}  // namespace fgf8
