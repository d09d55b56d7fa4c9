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
constexpr int kMaxCluster = 8;
constexpr uint32_t kFull = 0xFFFFFFFFu;

struct LoraKArgs {
  LoraArgs a;
  int tiles;       // tiles of a CTA: 1, 2, 4 or 8; its other warps split K and N further
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

// P from the sums over the shares of K: each CTA of the cluster sums every C-th row of `part`
// over all of them, a warp per row, and hands value, rest and power to all of them.
template <bool BF16, int RP>
__device__ __forceinline__ void exchange_rows(const float* part, uint16_t* hi, uint16_t* lo, float* power, int rows, const float* scale_of,
                                              int scale_rows, int C, int rank) {
  constexpr int LDP = RP + 4, LDH = RP + 8;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  for (int row = rank + C * warp; row < rows; row += C * kWarps) {
    const float scale = scale_of[row / scale_rows];
    constexpr int PAIRS = (RP + 63) / 64;
    float2 v[PAIRS];
    float top = 0.0f;
#pragma unroll
    for (int u = 0; u < PAIRS; ++u) {
      const int col = 2 * (lane + 32 * u);
      v[u] = make_float2(0.0f, 0.0f);
      if (col < RP) {
        const uint32_t at = ptx::smem_u32(part + row * LDP + col);
        float2 s[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < C) s[r] = ld_cluster_f32x2(map_to_rank(at, static_cast<uint32_t>(r)));
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < C) {
            v[u].x += s[r].x;
            v[u].y += s[r].y;
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
}

// Rows of tokens without an adapter: base, or zeros.  An item is 2 KB of 32 tokens; every warp
// of the grid takes its share when its other work is done, and looks at the tokens of its
// first item as it starts.  In place there is nothing to do.
struct Others {
  const LoraArgs& a;
  const uint32_t worker, workers, parts, items;
  bool first;
  static constexpr int kPart = 4;

  __device__ __forceinline__ Others(const LoraArgs& args, uint32_t w, uint32_t n)
      : a(args), worker(w), workers(n), parts((static_cast<uint32_t>(args.N) / 8 + 32 * kPart - 1) / (32 * kPart)),
        items(args.base == args.out ? 0u : (static_cast<uint32_t>(args.T) + 31) / 32 * parts) {
    first = worker < items && look(worker);
  }
  // whether this lane's token of an item is one
  __device__ __forceinline__ bool look(uint32_t it) const {
    const uint32_t t = it / parts * 32 + (threadIdx.x & 31);
    return t < static_cast<uint32_t>(a.T) && ptx::ld_global(a.rows + t) < 0;
  }
  __device__ __forceinline__ void fill() const {
    const int lane = static_cast<int>(threadIdx.x & 31), vecs = a.N / 8;
    for (uint32_t it = worker; it < items; it += workers) {
      const int v0 = static_cast<int>(it % parts) * 32 * kPart + lane;
      for (uint32_t left = __ballot_sync(kFull, it == worker ? first : look(it)); left != 0; left &= left - 1) {
        const size_t t = static_cast<size_t>(it / parts) * 32 + __ffs(left) - 1;
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
};
__device__ __forceinline__ uint32_t cta_of_grid() { return (blockIdx.x * gridDim.y + blockIdx.y) * gridDim.z + blockIdx.z; }

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

  const Others others(a, cta_of_grid() * kWarps + warp, gridDim.x * gridDim.y * gridDim.z * kWarps);

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
  if (__syncthreads_or(g >= 0) == 0) {                      // the same for every CTA of the cluster
    others.fill();
    return;
  }
  const int t0 = __shfl_sync(kFull, token, q), t1 = __shfl_sync(kFull, token, q + 8);

  // this CTA's part of N, whose rows of B are asked into L2 while A is read
  const int nblocks = (a.N + 31) / 32;
  const long long nshare = static_cast<long long>(blockIdx.y) * C + rank, nshares = static_cast<long long>(gridDim.y) * C;
  const int nb0 = static_cast<int>(nblocks * nshare / nshares), nb1 = static_cast<int>(nblocks * (nshare + 1) / nshares);
  const uint16_t* bg = static_cast<const uint16_t*>(a.B) + static_cast<size_t>(g < 0 ? 0 : g) * a.N * a.r;
  if (g >= 0) {
    const char *from = reinterpret_cast<const char*>(bg + static_cast<size_t>(nb0) * 32 * a.r),
               *to = reinterpret_cast<const char*>(bg + static_cast<size_t>(min(nb1 * 32, a.N)) * a.r);
    for (const char* p = from + 128 * (wk * 32 + lane); p < to; p += 128 * 32 * WK) gemv::prefetch_l2(p);
  }

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
  exchange_rows<BF16, RP>(part, hi, lo, power, WT * 16, tile_scale, 16, C, rank);
  if (C > 1) cluster_sync_all(); else __syncthreads();      // and nothing remote is touched behind this
  if (g < 0) {
    others.fill();
    return;
  }

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
  __syncwarp();
  others.fill();
}

// ----------------------------------------------------------------- many tokens of an adapter
// The same two products for blocks of 128 rows with one adapter, in which a byte of A or B
// serves 128 tokens.  X, A and B go through shared memory by cp.async, kStages blocks deep, so
// that enough of X and base is on its way without holding registers; four groups of warps
// take 32 tokens each and read A and B by ldmatrix, two warps of a group halve K, then N.
// Rows of a stage are 128 bytes in 16-byte pieces, piece p of row i at p ^ (i & 7).
constexpr int kStages = 3, kWideRows = 128;

template <int RP>
struct WideCfg {
  static constexpr int LDP = RP + 4, LDH = RP + 8;
  static constexpr int KSTAGE = (kWideRows + RP) * 128;     // 64 columns of X and A
  static constexpr int NB = 64;                             // rows of B in a block
  static constexpr int LDB = 2 * RP + 16;                   // bytes between them: ldmatrix without conflicts
  static constexpr int NSTAGE = NB * LDB;
  static constexpr int BSTAGE = kWideRows * 2 * NB;         // a block of base
  static constexpr int PART = kWideRows * LDP * 4;
  // [part, then stages of base | stages of B], over the stages of X and A; then P
  static constexpr int OFF_B = PART > kStages * BSTAGE ? PART : kStages * BSTAGE;
  static constexpr int FRONT = kStages * KSTAGE > OFF_B + kStages * NSTAGE ? kStages * KSTAGE : OFF_B + kStages * NSTAGE;
  static constexpr int OFF_HI = FRONT, OFF_LO = OFF_HI + kWideRows * LDH * 2, OFF_POWER = OFF_LO + kWideRows * LDH * 2;
  static constexpr int SMEM = OFF_POWER + kWideRows * 4;
};

__device__ __forceinline__ void ldmatrix_x4_at(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(addr) : "memory");
}

template <bool BF16, int RP>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) lora_f16_wide_kernel(LoraKArgs args) {
  using Cf = WideCfg<RP>;
  constexpr int NB8 = RP / 8;
  const LoraArgs& a = args.a;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int tokens[kWideRows];
  __shared__ float block_scale;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int q = lane >> 2, c = lane & 3;
  const int C = static_cast<int>(gridDim.z), rank = static_cast<int>(blockIdx.z);
  float* part = reinterpret_cast<float*>(smem);
  uint16_t *hi = reinterpret_cast<uint16_t*>(smem + Cf::OFF_HI), *lo = reinterpret_cast<uint16_t*>(smem + Cf::OFF_LO);
  float* power = reinterpret_cast<float*>(smem + Cf::OFF_POWER);
  const uint32_t base_s = ptx::smem_u32(smem);
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  const Others others(a, cta_of_grid() * kWarps + warp, gridDim.x * gridDim.y * gridDim.z * kWarps);
  // the block's adapter and tokens
  const long long row0 = static_cast<long long>(blockIdx.x) * kWideRows;
  int g = ptx::ld_global(a.m_indices + row0);
  bool bad = tid == 0 && (g >= a.G);
  if (g >= a.G) g = -1;
  if (tid < kWideRows) {
    const int id = ptx::ld_global(a.m_indices + row0 + tid);
    int t = ptx::ld_global(a.src + row0 + tid);
    if (id < 0 || t < 0 || g < 0) {
      t = -1;
    } else if (id != g || t >= a.T) {
      bad = true;
      t = -1;
    }
    tokens[tid] = t;
  }
  if (bad) atomicOr(a.status, FGF8_DEVERR_INPUT);
  if (tid == 0) block_scale = a.scale != nullptr && g >= 0 ? ptx::ld_global(a.scale + g) : 1.0f;
  __syncthreads();
  if (g < 0) {                                              // the same for every CTA of the cluster
    others.fill();
    return;
  }

  const uint16_t* ag = static_cast<const uint16_t*>(a.A) + static_cast<size_t>(g) * a.r * a.K;
  const uint16_t* bg = static_cast<const uint16_t*>(a.B) + static_cast<size_t>(g) * a.N * a.r;
  const int wm = warp & 3, wh = warp >> 2;                  // this warp's 32 tokens, its half of K or N

  // ------------------------------------------------------------ X A^T over a share of K
  const int ksteps = (a.K + 63) / 64;
  const int ks0 = static_cast<int>(static_cast<long long>(ksteps) * rank / C), ks1 = static_cast<int>(static_cast<long long>(ksteps) * (rank + 1) / C);
  const int prow = tid >> 3, pcol = tid & 7;                // the piece that this thread copies of every 32 rows
  const uint16_t* xrow[kWideRows / 32];
#pragma unroll
  for (int i = 0; i < kWideRows / 32; ++i) {
    const int t = tokens[prow + 32 * i];
    xrow[i] = t < 0 ? nullptr : static_cast<const uint16_t*>(a.X) + static_cast<size_t>(t) * a.ldx;
  }
  auto load_k = [&](int ks, int stage) {
    const int k = ks * 64 + pcol * 8;
    const bool in = ks < ks1 && k < a.K;
    const uint32_t to = base_s + static_cast<uint32_t>(stage * Cf::KSTAGE) + static_cast<uint32_t>(prow * 128 + ((pcol ^ (prow & 7)) << 4));
    if (ks < ks1) {
#pragma unroll
      for (int i = 0; i < kWideRows / 32; ++i) {
        const bool have = in && xrow[i] != nullptr;
        gemv::cp16(to + static_cast<uint32_t>(i * 32 * 128), have ? xrow[i] + k : static_cast<const uint16_t*>(a.X), have);
      }
#pragma unroll
      for (int i = 0; i < (RP + 31) / 32; ++i) {
        const int row = prow + 32 * i;
        if (row < RP) {
          const bool have = in && row < a.r;
          gemv::cp16(to + static_cast<uint32_t>((kWideRows + i * 32) * 128), have ? ag + static_cast<size_t>(row) * a.K + k : ag, have);
        }
      }
    }
    gemv::cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load_k(ks0 + s, s);
  float acc[2][NB8][4] = {};
  int stage = 0;
  for (int ks = ks0; ks < ks1; ++ks) {
    gemv::cp_wait<kStages - 2>();
    __syncthreads();                                        // the stage is there, and everybody is done with the one before
    load_k(ks + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
    const uint32_t sx = base_s + static_cast<uint32_t>(stage * Cf::KSTAGE), sa = sx + kWideRows * 128;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int piece = 4 * wh + 2 * kk;                    // the two 16-byte pieces of 16 columns
      uint32_t xf[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int row = 32 * wm + 16 * m + (lane & 15);
        ldmatrix_x4_at(sx + static_cast<uint32_t>(row * 128 + (((piece + (lane >> 4)) ^ (row & 7)) << 4)), xf[m][0], xf[m][1], xf[m][2], xf[m][3]);
      }
#pragma unroll
      for (int b = 0; b < NB8; b += 2) {
        const int row = 8 * b + (lane & 7) + ((lane >> 4) << 3);
        uint32_t w0, w1, w2, w3;
        ldmatrix_x4_at(sa + static_cast<uint32_t>(row * 128 + (((piece + ((lane >> 3) & 1)) ^ (row & 7)) << 4)), w0, w1, w2, w3);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          gemv::mma16816<BF16>(acc[m][b], xf[m][0], xf[m][1], xf[m][2], xf[m][3], w0, w1);
          gemv::mma16816<BF16>(acc[m][b + 1], xf[m][0], xf[m][1], xf[m][2], xf[m][3], w2, w3);
        }
      }
    }
    if (++stage == kStages) stage = 0;
  }
  gemv::cp_wait<0>();
  __syncthreads();
  // the halves of K meet in shared memory
#pragma unroll
  for (int half = 1; half >= 0; --half) {
    if (wh == half) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int b = 0; b < NB8; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float2* p = reinterpret_cast<float2*>(part + (32 * wm + 16 * m + 8 * e + q) * Cf::LDP + 8 * b + 2 * c);
            float2 v = make_float2(acc[m][b][2 * e], acc[m][b][2 * e + 1]);
            if (half == 0) {
              const float2 o = *p;
              v.x += o.x;
              v.y += o.y;
            }
            *p = v;
          }
    }
    __syncthreads();
  }

  // ------------------------------------------------------------ P B^T over a share of N
  const int nblocks = (a.N + Cf::NB - 1) / Cf::NB;
  const int nb0 = static_cast<int>(static_cast<long long>(nblocks) * rank / C), nb1 = static_cast<int>(static_cast<long long>(nblocks) * (rank + 1) / C);
  // row 8 x + 2 j + e of 32 goes to 8 j + 2 x + e: the eight rows of an MMA side by side, and a
  // lane's results of four MMAs are eight neighbours
  auto load_n = [&](int nb, int s) {
    constexpr int PIECES = RP / 8;                          // of a row
    if (nb < nb1) {
#pragma unroll
      for (int i = tid; i < Cf::NB * PIECES; i += kThreads) {
        const int row = i / PIECES, piece = i % PIECES, n = nb * Cf::NB + row;
        const int at = (row & 32) + ((row >> 1) & 3) * 8 + ((row >> 3) & 3) * 2 + (row & 1);
        const bool have = n < a.N && 8 * piece < a.r;
        gemv::cp16(base_s + Cf::OFF_B + static_cast<uint32_t>(s * Cf::NSTAGE + at * Cf::LDB + piece * 16),
                   have ? bg + static_cast<size_t>(n) * a.r + 8 * piece : bg, have);
      }
    }
    gemv::cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load_n(nb0 + s, s);
  if (C > 1) cluster_sync_all();
  exchange_rows<BF16, RP>(part, hi, lo, power, kWideRows, &block_scale, kWideRows, C, rank);
  if (C > 1) cluster_sync_all(); else __syncthreads();      // and nothing remote is touched behind this

  int t[4];                                                 // tokens of rows q, q + 8, q + 16, q + 24 of the 32
  float up[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = tokens[32 * wm + 8 * i + q];
    up[i] = power[32 * wm + 8 * i + q];
  }
  const int off = 32 * wh + 8 * c;                          // this lane's columns of a block
  // 16-byte piece p of row i of a block of base stands at p ^ turn(i): the pieces that eight
  // lanes read together are in different banks
  auto turn = [](int row) { return ((row & 1) << 2) | ((row >> 1) & 3); };
  int brow[kWideRows / 32];
#pragma unroll
  for (int i = 0; i < kWideRows / 32; ++i) brow[i] = a.base != nullptr ? tokens[prow + 32 * i] : -1;
  auto load_base = [&](int nb, int s) {
    const int n0 = nb * Cf::NB + 8 * pcol;
    if (nb < nb1) {
#pragma unroll
      for (int i = 0; i < kWideRows / 32; ++i) {
        const bool have = n0 < a.N && brow[i] >= 0;
        const uint16_t* from = have ? static_cast<const uint16_t*>(a.base) + static_cast<size_t>(brow[i]) * a.ldb + n0 : bg;
        gemv::cp16(base_s + static_cast<uint32_t>(s * Cf::BSTAGE + (prow + 32 * i) * 128 + ((pcol ^ turn(prow)) << 4)), from, have);
      }
    }
    gemv::cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load_base(nb0 + s, s);
  const uint32_t sh = base_s + Cf::OFF_HI + static_cast<uint32_t>((32 * wm + (lane & 15)) * Cf::LDH * 2 + (lane >> 4) * 16);
  stage = 0;
  for (int nb = nb0; nb < nb1; ++nb) {
    // groups in order: two of B, two of base, then for each block its B and base together
    if (nb == nb0)
      gemv::cp_wait<kStages - 2>();
    else
      gemv::cp_wait<2 * (kStages - 2)>();
    __syncthreads();
    const int ahead = stage == 0 ? kStages - 1 : stage - 1;
    load_n(nb + kStages - 1, ahead);
    load_base(nb + kStages - 1, ahead);
    const uint32_t sb = base_s + Cf::OFF_B + static_cast<uint32_t>(stage * Cf::NSTAGE + (32 * wh + (lane & 7) + ((lane >> 4) << 3)) * Cf::LDB + ((lane >> 3) & 1) * 16);
    float d[2][4][4] = {};
#pragma unroll
    for (int k = 0; k < RP / 16; ++k) {
      uint32_t bf[4][2];
      ldmatrix_x4_at(sb + static_cast<uint32_t>(k * 32), bf[0][0], bf[0][1], bf[1][0], bf[1][1]);
      ldmatrix_x4_at(sb + static_cast<uint32_t>(16 * Cf::LDB + k * 32), bf[2][0], bf[2][1], bf[3][0], bf[3][1]);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int part_of = 0; part_of < 2; ++part_of) {     // P rounded, and its rest
          uint32_t pf[4];
          ldmatrix_x4_at(sh + static_cast<uint32_t>((part_of ? Cf::OFF_LO - Cf::OFF_HI : 0) + m * 16 * Cf::LDH * 2 + k * 32), pf[0], pf[1], pf[2], pf[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) gemv::mma16816<BF16>(d[m][j], pf[0], pf[1], pf[2], pf[3], bf[j][0], bf[j][1]);
        }
    }
    const int n0 = nb * Cf::NB + off;
    if (n0 < a.N) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t[i] < 0) continue;
        const int row = 32 * wm + 8 * i + q;
        uint32_t bw[4], ow[4];
        gemv::lds128(smem + stage * Cf::BSTAGE + row * 128 + (((4 * wh + c) ^ turn(row)) << 4), bw);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ow[j] = pack_2x16(fmaf(up[i], d[i >> 1][j][2 * (i & 1)], act::to_float(bw[j] & 0xFFFFu, BF16)),
                            fmaf(up[i], d[i >> 1][j][2 * (i & 1) + 1], act::to_float(bw[j] >> 16, BF16)), BF16);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + static_cast<size_t>(t[i]) * a.ldo + n0) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
      }
    }
    __syncwarp();                                           // whole-warp instructions follow
    if (++stage == kStages) stage = 0;
  }
  gemv::cp_wait<0>();
  others.fill();
}

// Shared memory of a CTA with `tiles` tiles.
template <int RP>
constexpr int smem_bytes(int tiles) {
  return kWarps * 16 * (RP + 4) * 4 + 2 * tiles * 16 * (RP + 8) * 2 + tiles * 16 * 4;
}

struct LoraLaunch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  LoraLaunch(long long groups, int parts, int cluster, size_t smem, cudaStream_t stream) {
    std::memset(&cfg, 0, sizeof(cfg));
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = static_cast<unsigned>(cluster);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(groups), static_cast<unsigned>(parts), static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
  }
};

// Opens the kernel's shared memory once per device, then launches it.
template <typename K>
int launch(K* fn, PerDevice<int>& ready, int most_smem, int smem, const LoraKArgs& k, long long groups, int parts, int cluster, cudaStream_t stream) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  const int* set = nullptr;
  const int r = ready.get(dev, &set, [&](int& v) {
    v = most_smem;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
    return e == cudaSuccess ? 0 : set_error(4, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  });
  if (r) return r;
  LoraLaunch l(groups, parts, cluster, static_cast<size_t>(smem), stream);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, fn, k);
  return e == cudaSuccess ? 0 : set_error(4, "lora_f16 launch: %s", cudaGetErrorString(e));
}

template <bool BF16, int RP>
int launch_tiles(const LoraArgs& a, cudaStream_t stream) {
  static PerDevice<int> ready;
  LoraKArgs k;
  k.a = a;
  const long long tiles = a.M / 16, sms = device_sm_count();
  const long long nblocks = (a.N + 31) / 32;
  // a cluster's CTAs split K and N: eight, fewer where there is too little to split
  int cluster = kMaxCluster;
  while (cluster > 1 && (a.K + 31) / 32 < 2 * cluster && nblocks < 2 * cluster) cluster /= 2;
  // tiles share a CTA as soon as there are two CTAs per SM without
  k.tiles = 8;
  while (k.tiles > 1 && (tiles + k.tiles - 1) / k.tiles * cluster < 2 * sms) k.tiles /= 2;
  // few tiles: several clusters per tile, each a part of N
  const long long groups = (tiles + k.tiles - 1) / k.tiles;
  int parts = 1;
  while (parts < 64 && 2 * parts * groups * cluster <= sms && 2 * parts * cluster <= nblocks) parts *= 2;
  return launch(&lora_f16_kernel<BF16, RP>, ready, smem_bytes<RP>(kWarps), smem_bytes<RP>(k.tiles), k, groups, parts, cluster, stream);
}

template <bool BF16, int RP>
int launch_wide(const LoraArgs& a, cudaStream_t stream) {
  static PerDevice<int> ready;
  static_assert(WideCfg<RP>::SMEM <= 232448 - 1024, "shared memory budget");
  LoraKArgs k;
  k.a = a;
  k.tiles = 8;
  // the cluster that takes the least time in waves of what fits the device, each as long as the
  // share of a CTA and, for the start and the exchange of P, a fortieth of a whole block
  const long long groups = a.M / kWideRows, slots = static_cast<long long>(device_sm_count()) * (RP <= 64 ? 2 : 1);
  int cluster = 1;
  double best = 0.0;
  for (int c = 1; c <= kMaxCluster; c *= 2) {
    if (c > 1 && (a.K + 63) / 64 < 2 * c && (a.N + 63) / 64 < 2 * c) break;
    const double time = static_cast<double>((groups * c + slots - 1) / slots) * (1.0 / c + 0.025);
    if (c == 1 || time < best) {
      best = time;
      cluster = c;
    }
  }
  return launch(&lora_f16_wide_kernel<BF16, RP>, ready, WideCfg<RP>::SMEM, WideCfg<RP>::SMEM, k, groups, 1, cluster, stream);
}

template <bool BF16, int RP>
int by_align(const LoraArgs& a, cudaStream_t stream) {
  return a.align % kWideRows == 0 ? launch_wide<BF16, RP>(a, stream) : launch_tiles<BF16, RP>(a, stream);
}

template <bool BF16>
int by_rank(const LoraArgs& a, cudaStream_t stream) {
  if (a.r <= 16) return by_align<BF16, 16>(a, stream);
  if (a.r <= 32) return by_align<BF16, 32>(a, stream);
  if (a.r <= 64) return by_align<BF16, 64>(a, stream);
  return by_align<BF16, 128>(a, stream);
}

}  // namespace

int launch_lora_f16(const LoraArgs& a, int bf16, cudaStream_t stream) {
  return bf16 ? by_rank<true>(a, stream) : by_rank<false>(a, stream);
}

}  // namespace fgf8
