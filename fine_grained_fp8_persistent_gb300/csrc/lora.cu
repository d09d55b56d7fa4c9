// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + s_g (X[t] A_g^T) B_g^T,   g the adapter of token t,
// A_g (r, K), B_g (N, r) with r up to 128, tokens grouped by adapter in tiles of 16 rows.
//
// One launch.  A cluster takes a run of tiles.  First its CTAs split K: a warp multiplies
// the 16 tokens of a tile with the adapter's rows over its share of K, the shares' sums meet
// in distributed shared memory, and P = s X A^T goes to every CTA of the cluster.  Then the
// CTAs split N.  P never leaves the chip, X and base are read once, out is written once.
// With few tiles, several clusters take the same tiles and each its part of N; they all
// compute P, from A that then comes from L2.
//
// The products run on mma.sync m16n8k16 with tokens as M: the call is bound by the reading
// and writing of X, base and out (for one token by that of A and B), not by the r = 16 .. 128
// multiplications that each of those elements meets.  Operands come from global memory
// straight into the registers of the MMA: the order of the reduction is free, so lane
// 4 q + c takes the elements 8 c .. 8 c + 7 of a row as its k indices of two instructions,
// which is one 16-byte load and 64 contiguous bytes of each row.  In the second product the
// columns of B are permuted in the same way so that a lane's results are 8 neighbours of a
// token's row.
//
// P is the left operand of the second product, in 16 bits.  It is split into a rounded value
// and the rounded rest, two instructions instead of one, so that it keeps 16 (bf16) or 22
// (fp16) bits and the only rounding to the operands' type is that of out.  In fp16 each row
// of P is first scaled by a power of two, so that no sum over K leaves the type's range.
#include <cstring>

#include "gemv.cuh"
#include "routed.h"

namespace fgf8 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kFull = 0xFFFFFFFFu;

struct LoraKArgs {
  LoraArgs a;
  int tiles;       // tiles of a CTA: 1, 2, 4 or 8; its other warps split K and N further
  int copy;        // clusters behind the tiles' that fill the rows of tokens without an adapter
};

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_global_v2(const void* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Rounded value and rounded rest of two FP32 values, each pair packed.  A value that is not
// finite has no rest; a finite one that would round to infinity keeps the largest value and
// its rest.
template <bool BF16>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const float top = BF16 ? __uint_as_float(0x7F7F0000u) : 65504.0f;
  float v[2] = {x, y}, h[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    h[i] = act::to_float(act::from_float(v[i], BF16), BF16);
    const bool finite = fabsf(v[i]) <= 3.4028235e38f;
    if (finite && fabsf(h[i]) > top) h[i] = copysignf(top, v[i]);
    l[i] = finite ? v[i] - h[i] : 0.0f;
  }
  hi = pack_2x16(h[0], h[1], BF16);
  lo = pack_2x16(l[0], l[1], BF16);
}

// Rows of tokens without an adapter: base, or zeros.  A warp's item is 2 KB of 32 tokens.
__device__ __forceinline__ void fill_others(const LoraArgs& a, long long worker, long long workers, int lane) {
  constexpr int kPart = 4;
  const int vecs = a.N / 8, parts = (vecs + 32 * kPart - 1) / (32 * kPart);
  const long long items = (static_cast<long long>(a.T) + 31) / 32 * parts;
  for (long long it = worker; it < items; it += workers) {
    const int t0 = static_cast<int>(it / parts) * 32, v0 = static_cast<int>(it % parts) * 32 * kPart + lane;
    const bool other = t0 + lane < a.T && ptx::ld_global(a.rows + t0 + lane) < 0;
    for (uint32_t left = __ballot_sync(kFull, other); left != 0; left &= left - 1) {
      const size_t t = static_cast<size_t>(t0 + __ffs(left) - 1);
      uint4 v[kPart] = {};
#pragma unroll
      for (int u = 0; u < kPart; ++u)
        if (a.base != nullptr && v0 + 32 * u < vecs)
          v[u] = ptx::ld_global_v4(static_cast<const uint16_t*>(a.base) + t * a.ldb + 8 * static_cast<size_t>(v0 + 32 * u));
#pragma unroll
      for (int u = 0; u < kPart; ++u)
        if (v0 + 32 * u < vecs) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + t * a.ldo + 8 * static_cast<size_t>(v0 + 32 * u)) = v[u];
    }
  }
}

// RP: the rank rounded up to 16, 32, 64 or 128.  Blocks of rank rows past r load nothing.
template <bool BF16, int RP>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) lora_f16_kernel(LoraKArgs args) {
  constexpr int NB = RP / 8;                                // blocks of 8 rank rows
  constexpr int UNROLL = RP <= 16 ? 4 : RP <= 32 ? 3 : RP <= 64 ? 2 : 1;
  constexpr int LDP = RP + 4;                               // floats of a row of sums in shared memory
  constexpr int LDH = RP + 8;                               // 16-bit values of a row of P
  const LoraArgs& a = args.a;
  extern __shared__ __align__(16) uint8_t smem[];
  const int WT = args.tiles, WK = kWarps / WT;
  float* part = reinterpret_cast<float*>(smem);             // [WK][16 WT][LDP] sums over a share of K
  uint16_t* hi = reinterpret_cast<uint16_t*>(part + kWarps * 16 * LDP);  // [16 WT][LDH]
  uint16_t* lo = hi + WT * 16 * LDH;
  float* power = reinterpret_cast<float*>(lo + WT * 16 * LDH);           // [16 WT] what a row of P is to be multiplied by
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int q = lane >> 2, c = lane & 3;
  const int C = static_cast<int>(gridDim.z), rank = static_cast<int>(blockIdx.z);      // the cluster is (1, 1, C)
  __shared__ float tile_scale[kWarps];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  const int groups = static_cast<int>(gridDim.x) - args.copy;
  if (static_cast<int>(blockIdx.x) >= groups) {
    if (blockIdx.y == 0)
      fill_others(a, (static_cast<long long>(blockIdx.x - groups) * C + rank) * kWarps + warp, static_cast<long long>(args.copy) * C * kWarps, lane);
    return;                                                 // whole clusters
  }

  // the tile of this warp: its adapter and tokens
  const int wt = warp % WT, wk = warp / WT;
  const long long row0 = (static_cast<long long>(blockIdx.x) * WT + wt) * 16;
  int g = -1, token = -1;
  if (row0 < a.M) {                                         // M is a multiple of 16
    int id = -1;
    if (lane < 16) {
      id = ptx::ld_global(a.m_indices + row0 + lane);
      token = ptx::ld_global(a.src + row0 + lane);
    }
    g = __shfl_sync(kFull, id, 0);
    // rows of another adapter, adapters and tokens out of range are reported and left alone
    bool bad = false;
    if (g >= a.G) {
      bad = lane == 0;
      g = -1;
    }
    if (id < 0 || token < 0 || g < 0) {
      token = -1;
    } else if (id != g || token >= a.T) {
      bad = true;
      token = -1;
    }
    if (bad) atomicOr(a.status, FGF8_DEVERR_INPUT);
  }
  if (__syncthreads_or(g >= 0) == 0) return;                // the same for every CTA of the cluster
  const int t0 = __shfl_sync(kFull, token, q), t1 = __shfl_sync(kFull, token, q + 8);

  // ------------------------------------------------------------ X A^T over a share of K
  const int share = rank * WK + wk, shares = C * WK;
  const int kblocks = (a.K + 31) / 32;
  const int kb0 = static_cast<int>(static_cast<long long>(kblocks) * share / shares);
  const int kb1 = static_cast<int>(static_cast<long long>(kblocks) * (share + 1) / shares);
  float acc[NB][4] = {};
  if (g >= 0) {
    const uint16_t* x0 = static_cast<const uint16_t*>(a.X) + static_cast<size_t>(t0 < 0 ? 0 : t0) * a.ldx;
    const uint16_t* x1 = static_cast<const uint16_t*>(a.X) + static_cast<size_t>(t1 < 0 ? 0 : t1) * a.ldx;
    const uint16_t* w = static_cast<const uint16_t*>(a.A) + (static_cast<size_t>(g) * a.r + q) * a.K;
    for (int kb = kb0; kb < kb1; kb += UNROLL) {
      uint4 xv[UNROLL][2], wv[UNROLL][NB];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int k = (kb + u) * 32 + 8 * c;
        const bool in = kb + u < kb1 && k < a.K;
        xv[u][0] = in && t0 >= 0 ? ptx::ld_global_v4(x0 + k) : make_uint4(0u, 0u, 0u, 0u);
        xv[u][1] = in && t1 >= 0 ? ptx::ld_global_v4(x1 + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          wv[u][b] = in && 8 * b < a.r ? ptx::ld_global_v4(w + static_cast<size_t>(8 * b) * a.K + k) : make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();                                         // the instructions below are whole-warp ones
#pragma unroll
      for (int u = 0; u < UNROLL; ++u)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          gemv::mma16816<BF16>(acc[b], xv[u][0].x, xv[u][1].x, xv[u][0].y, xv[u][1].y, wv[u][b].x, wv[u][b].y);
          gemv::mma16816<BF16>(acc[b], xv[u][0].z, xv[u][1].z, xv[u][0].w, xv[u][1].w, wv[u][b].z, wv[u][b].w);
        }
    }
  }
  if (wk == 0 && lane == 0) tile_scale[wt] = a.scale != nullptr && g >= 0 ? ptx::ld_global(a.scale + g) : 1.0f;
  {
    float* p = part + (wk * WT + wt) * 16 * LDP;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      *reinterpret_cast<float2*>(p + q * LDP + 8 * b + 2 * c) = make_float2(acc[b][0], acc[b][1]);
      *reinterpret_cast<float2*>(p + (q + 8) * LDP + 8 * b + 2 * c) = make_float2(acc[b][2], acc[b][3]);
    }
  }
  __syncthreads();
  if (WK > 1) {
    for (int i = tid; i < WT * 16 * RP; i += kThreads) {
      const int at = i / RP * LDP + i % RP;
      float s = part[at];
      for (int k = 1; k < WK; ++k) s += part[k * WT * 16 * LDP + at];
      part[at] = s;
    }
  }
  if (C > 1) cluster_sync_all(); else __syncthreads();

  // ------------------------------------------------------------ P, a warp per row
  // each CTA sums every C-th row over the cluster and hands it to all of them
  for (int row = rank + C * warp; row < WT * 16; row += C * kWarps) {
    const float scale = tile_scale[row / 16];
    constexpr int PAIRS = (RP + 63) / 64;
    float2 v[PAIRS];
    float top = 0.0f;
#pragma unroll
    for (int u = 0; u < PAIRS; ++u) {
      const int col = 2 * (lane + 32 * u);
      v[u] = make_float2(0.0f, 0.0f);
      if (col < RP) {
        const uint32_t at = ptx::smem_u32(part + row * LDP + col);
        for (int r = 0; r < C; ++r) {
          const float2 s = ld_cluster_f32x2(map_to_rank(at, static_cast<uint32_t>(r)));
          v[u].x += s.x;
          v[u].y += s.y;
        }
        v[u].x *= scale;
        v[u].y *= scale;
        if (!BF16) top = fmaxf(top, fmaxf(fabsf(v[u].x), fabsf(v[u].y)));
      }
    }
    float up = 1.0f;
    if (!BF16) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
      // the largest goes to [2^14, 2^15): exponents stay where 2^e and 2^-e are normal numbers
      int e = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14;
      e = e < -126 ? -126 : e;
      if (top == 0.0f || top > 3.4028235e38f) e = 0;
      up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int u = 0; u < PAIRS; ++u) {
        v[u].x *= down;
        v[u].y *= down;
      }
    }
#pragma unroll
    for (int u = 0; u < PAIRS; ++u) {
      const int col = 2 * (lane + 32 * u);
      if (col < RP) {
        uint32_t h, l;
        split2<BF16>(v[u].x, v[u].y, h, l);
        const uint32_t at_h = ptx::smem_u32(hi + row * LDH + col), at_l = ptx::smem_u32(lo + row * LDH + col);
        for (int r = 0; r < C; ++r) {
          st_cluster_u32(map_to_rank(at_h, static_cast<uint32_t>(r)), h);
          st_cluster_u32(map_to_rank(at_l, static_cast<uint32_t>(r)), l);
        }
      }
    }
    if (lane < C) st_cluster_f32(map_to_rank(ptx::smem_u32(power + row), static_cast<uint32_t>(lane)), up);
  }
  if (C > 1) cluster_sync_all(); else __syncthreads();      // and nothing remote is touched behind this
  if (g < 0) return;

  // ------------------------------------------------------------ P B^T over a share of N
  constexpr int KS = RP >= 32 ? RP / 32 : 1;                // steps of 32 rank rows (of 16 when there are no more)
  uint32_t ph[KS][8], pl[KS][8];                            // [row q: 4 words][row q + 8: 4 words]
  {
    const uint16_t *h0 = hi + (wt * 16 + q) * LDH, *l0 = lo + (wt * 16 + q) * LDH;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint16_t *h = h0 + half * 8 * LDH, *l = l0 + half * 8 * LDH;
        if constexpr (RP >= 32) {
          const uint4 vh = *reinterpret_cast<const uint4*>(h + 32 * s + 8 * c), vl = *reinterpret_cast<const uint4*>(l + 32 * s + 8 * c);
          ph[s][4 * half] = vh.x, ph[s][4 * half + 1] = vh.y, ph[s][4 * half + 2] = vh.z, ph[s][4 * half + 3] = vh.w;
          pl[s][4 * half] = vl.x, pl[s][4 * half + 1] = vl.y, pl[s][4 * half + 2] = vl.z, pl[s][4 * half + 3] = vl.w;
        } else {
          const uint2 vh = *reinterpret_cast<const uint2*>(h + 4 * c), vl = *reinterpret_cast<const uint2*>(l + 4 * c);
          ph[s][4 * half] = vh.x, ph[s][4 * half + 1] = vh.y, ph[s][4 * half + 2] = 0u, ph[s][4 * half + 3] = 0u;
          pl[s][4 * half] = vl.x, pl[s][4 * half + 1] = vl.y, pl[s][4 * half + 2] = 0u, pl[s][4 * half + 3] = 0u;
        }
      }
  }
  const float up0 = power[wt * 16 + q], up1 = power[wt * 16 + q + 8];
  const int nblocks = (a.N + 31) / 32;
  const long long nshare = static_cast<long long>(blockIdx.y) * C + rank, nshares = static_cast<long long>(gridDim.y) * C;
  const int nb0 = static_cast<int>(nblocks * nshare / nshares), nb1 = static_cast<int>(nblocks * (nshare + 1) / nshares);
  const uint16_t* bg = static_cast<const uint16_t*>(a.B) + static_cast<size_t>(g) * a.N * a.r;
  for (int nb = nb0 + wk; nb < nb1; nb += WK) {
    const int n0 = nb * 32 + 8 * c;                         // this lane's 8 columns of out
    const bool in = n0 < a.N;
    uint4 base0 = make_uint4(0u, 0u, 0u, 0u), base1 = base0;
    if (a.base != nullptr && in) {
      const uint16_t* b = static_cast<const uint16_t*>(a.base);
      if (t0 >= 0) base0 = ptx::ld_global_v4(b + static_cast<size_t>(t0) * a.ldb + n0);
      if (t1 >= 0) base1 = ptx::ld_global_v4(b + static_cast<size_t>(t1) * a.ldb + n0);
    }
    float d[4][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = nb * 32 + 8 * (q >> 1) + 2 * j + (q & 1);
      const uint16_t* bn = bg + static_cast<size_t>(n < a.N ? n : 0) * a.r;
      uint4 bv[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        bv[s] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (RP >= 32) {
          if (n < a.N && 32 * s + 8 * c < a.r) bv[s] = ptx::ld_global_v4(bn + 32 * s + 8 * c);
        } else {
          if (n < a.N && 4 * c < a.r) {
            const uint2 v = ld_global_v2(bn + 4 * c);
            bv[s].x = v.x;
            bv[s].y = v.y;
          }
        }
      }
      __syncwarp();
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        gemv::mma16816<BF16>(d[j], ph[s][0], ph[s][4], ph[s][1], ph[s][5], bv[s].x, bv[s].y);
        gemv::mma16816<BF16>(d[j], pl[s][0], pl[s][4], pl[s][1], pl[s][5], bv[s].x, bv[s].y);
        if constexpr (RP >= 32) {
          gemv::mma16816<BF16>(d[j], ph[s][2], ph[s][6], ph[s][3], ph[s][7], bv[s].z, bv[s].w);
          gemv::mma16816<BF16>(d[j], pl[s][2], pl[s][6], pl[s][3], pl[s][7], bv[s].z, bv[s].w);
        }
      }
    }
    if (in) {
      uint16_t* o = static_cast<uint16_t*>(a.out);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int t = half ? t1 : t0;
        if (t < 0) continue;
        const float up = half ? up1 : up0;
        const uint4& b = half ? base1 : base0;
        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
        uint32_t ow[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ow[j] = pack_2x16(fmaf(up, d[j][2 * half], act::to_float(bw[j] & 0xFFFFu, BF16)),
                            fmaf(up, d[j][2 * half + 1], act::to_float(bw[j] >> 16, BF16)), BF16);
        *reinterpret_cast<uint4*>(o + static_cast<size_t>(t) * a.ldo + n0) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
      }
    }
  }
}

// Shared memory of a CTA with `tiles` tiles.
template <int RP>
constexpr int smem_bytes(int tiles) {
  return kWarps * 16 * (RP + 4) * 4 + 2 * tiles * 16 * (RP + 8) * 2 + tiles * 16 * 4;
}

template <bool BF16, int RP>
int launch(LoraKArgs& k, int cluster, int parts, cudaStream_t stream) {
  auto* fn = &lora_f16_kernel<BF16, RP>;
  static PerDevice<int> ready;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  const int* set = nullptr;
  const int r = ready.get(dev, &set, [&](int& v) {
    v = smem_bytes<RP>(kWarps);
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
    return e == cudaSuccess ? 0 : set_error(4, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  });
  if (r) return r;
  const long long groups = (k.a.M / 16 + k.tiles - 1) / k.tiles;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = static_cast<unsigned>(cluster);
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(groups + k.copy), static_cast<unsigned>(parts), static_cast<unsigned>(cluster));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes<RP>(k.tiles));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, k);
  return e == cudaSuccess ? 0 : set_error(4, "lora_f16 launch: %s", cudaGetErrorString(e));
}

template <bool BF16>
int by_rank(LoraKArgs& k, int cluster, int parts, cudaStream_t stream) {
  if (k.a.r <= 16) return launch<BF16, 16>(k, cluster, parts, stream);
  if (k.a.r <= 32) return launch<BF16, 32>(k, cluster, parts, stream);
  if (k.a.r <= 64) return launch<BF16, 64>(k, cluster, parts, stream);
  return launch<BF16, 128>(k, cluster, parts, stream);
}

}  // namespace

int launch_lora_f16(const LoraArgs& a, int bf16, cudaStream_t stream) {
  LoraKArgs k;
  k.a = a;
  const long long tiles = a.M / 16, sms = device_sm_count();
  const long long nblocks = (a.N + 31) / 32;
  // a cluster's CTAs split K and N: eight, fewer where there is too little to split
  int cluster = 8;
  while (cluster > 1 && (a.K + 31) / 32 < 2 * cluster && nblocks < 2 * cluster) cluster /= 2;
  // tiles share a CTA as soon as there are two CTAs per SM without
  k.tiles = 8;
  while (k.tiles > 1 && (tiles + k.tiles - 1) / k.tiles * cluster < 2 * sms) k.tiles /= 2;
  // few tiles: several clusters per tile, each a part of N
  long long parts = 1;
  const long long ctas = (tiles + k.tiles - 1) / k.tiles * cluster;
  while (parts < 64 && 2 * parts * ctas <= sms && 2 * parts * cluster <= nblocks) parts *= 2;
  k.copy = 0;
  if (a.base != a.out) {
    const long long items = (a.T + 31LL) / 32 * ((a.N / 8 + 127) / 128), want = (items + cluster * kWarps - 1) / (cluster * kWarps);
    const long long most = (2 * sms + cluster - 1) / cluster;
    k.copy = static_cast<int>(want < most ? want : most);
  }
  return bf16 ? by_rank<true>(k, cluster, static_cast<int>(parts), stream) : by_rank<false>(k, cluster, static_cast<int>(parts), stream);
}

}  // namespace fgf8
