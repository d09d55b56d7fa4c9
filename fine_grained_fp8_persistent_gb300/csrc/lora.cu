// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + s_g (X[t] A_g^T) B_g^T,   g the adapter of token t,
// A_g (r, K), B_g (N, r) with r up to 128, tokens grouped by adapter in tiles of 16 rows.
//
// One launch, in two forms: tiles of 16 rows (below) and, where the rows of an adapter come in
// blocks of 128, those (further down).  A cluster takes a tile or block.  First its CTAs split
// K: X A^T over a share of K, whose sums meet in distributed shared memory.  Then they split
// N.  P = s X A^T never leaves the chip, X and base are read once, out is written once.
//
// Tiles of 16 are for few tokens per adapter, where the adapter's own bytes and the latency of
// a chain of dependent steps are the time: ids, X and A, sums, B, out.  Warps multiply on
// mma.sync m16n8k16 with tokens as M, operands straight from global memory into the registers
// of the MMA: the order of the reduction is free, so lane 4 q + c takes the elements
// 8 c .. 8 c + 7 of a row as its k indices of two instructions, which is one 16-byte load and
// 64 contiguous bytes of each row.  In the second product the columns of B are permuted in the
// same way so that a lane's results are 8 neighbours of a token's row.  While A is read, the
// CTA's part of B is asked into L2, and its first blocks come while the sums meet.  Where SMs
// are left, several clusters take the same tile and each its part of N; they all compute P,
// from A that then comes from L2.
//
// P is the left operand of the second product, in 16 bits.  It is split into a value rounded
// toward zero and the rounded rest, two instructions instead of one, so that it keeps 16 (bf16)
// or 22 (fp16) bits and the only rounding to the operands' type is that of out.  In fp16 each row
// of P is first scaled by a power of two, so that no sum over K leaves the type's range.  The rest
// has P's sign and is never zero beside a value that is not: both parts times an infinity of B
// are then the infinity that P times it is.  (Rounded to nearest, P would keep one bit more and
// have NaN there.  Sums that come out NaN taken again from the whole P instead: 2 % of the time in
// blocks of 128 rows and up to 12 % in tiles of 16, for the look at each.)
#include <cstdlib>
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
  uint64_t timeout_ns;
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

// Value rounded toward zero and rounded rest of two FP32 values, each pair packed.  Where the
// rest would be zero beside a value that is not (an exact or infinite one), it is the type's
// smallest number: 2^-133 (bf16), 2^-24 (fp16, 2^-39 of what rows are scaled to).
template <bool BF16>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const float least = BF16 ? __uint_as_float(0x00010000u) : 0x1p-24f;
  float v[2] = {x, y}, h[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool finite = fabsf(v[i]) <= 3.4028235e38f;
    h[i] = v[i];
    if (finite) h[i] = BF16 ? __uint_as_float(__float_as_uint(v[i]) & 0xFFFF0000u) : __half2float(__float2half_rz(v[i]));
    l[i] = finite ? act::to_float(act::from_float(v[i] - h[i], BF16), BF16) : 0.0f;
    if (l[i] == 0.0f && h[i] != 0.0f) l[i] = copysignf(least, h[i]);
  }
  hi = pack_2x16(h[0], h[1], BF16);
  lo = pack_2x16(l[0], l[1], BF16);
}
// |x| of a finite x, else 0.
__device__ __forceinline__ float finite_size(float x) { return fabsf(x) <= 3.4028235e38f ? fabsf(x) : 0.0f; }

// P from the sums over the shares of K, as value, rest and power.  With ALL every CTA of the
// cluster sums all rows over `part` of all CTAs and keeps them; otherwise it sums every C-th row
// and hands it to all of them.  place(row, column, value's address, rest's) says where two
// columns go.  A row is summed by as many lanes as it has pairs of columns, up to 32.  Columns
// from the rank on do not exist: they are zeros here, whatever stands in `part` (an infinity of X
// by nothing is NaN there) and whatever the scale is.
template <bool BF16, int RP, bool ALL, typename Place>
__device__ __forceinline__ void exchange_rows(const float* part, float* power, int rows, int columns, const float* scale_at, int C,
                                              int rank, Place&& place) {
  constexpr int LDP = RP + 4, LANES = RP >= 64 ? 32 : RP / 2, PAIRS = RP / 2 / LANES, TOGETHER = 32 / LANES;
  constexpr int ROWS = ALL || RP == 16 ? 1 : RP == 128 ? 2 : 4;   // rows of a lane whose loads are in flight together
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31), at_lane = lane % LANES;
  const int first = ALL ? 0 : rank, step = ALL ? 1 : C;
  const float scale = *scale_at;
  for (int i = warp * TOGETHER; first + step * i < rows; i += kWarps * TOGETHER * ROWS) {
    float2 v[ROWS][PAIRS];
    int row[ROWS];
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
      row[m] = first + step * (i + m * kWarps * TOGETHER + lane / LANES);
      if (row[m] >= rows) row[m] = -1;
#pragma unroll
      for (int u = 0; u < PAIRS; ++u) v[m][u] = make_float2(0.0f, 0.0f);
    }
    // over the cluster in its order, two CTAs at a time
    for (int r = 0; r < C; r += 2) {
      float2 s[2][ROWS][PAIRS];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < ROWS; ++m)
#pragma unroll
          for (int u = 0; u < PAIRS; ++u) {
            s[h][m][u] = make_float2(0.0f, 0.0f);
            if (row[m] >= 0 && r + h < C)
              s[h][m][u] = ld_cluster_f32x2(map_to_rank(ptx::smem_u32(part + row[m] * LDP + 2 * (at_lane + LANES * u)), static_cast<uint32_t>(r + h)));
          }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < ROWS; ++m)
#pragma unroll
          for (int u = 0; u < PAIRS; ++u) {
            v[m][u].x += s[h][m][u].x;
            v[m][u].y += s[h][m][u].y;
          }
    }
    __syncwarp();
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
      float top = 0.0f, up = 1.0f;
#pragma unroll
      for (int u = 0; u < PAIRS; ++u) {
        if (2 * (at_lane + LANES * u) < columns) {
          v[m][u].x *= scale;
          v[m][u].y *= scale;
        } else {
          v[m][u] = make_float2(0.0f, 0.0f);
        }
        if (!BF16) top = fmaxf(top, fmaxf(finite_size(v[m][u].x), finite_size(v[m][u].y)));
      }
      if (!BF16) {
#pragma unroll
        for (int off = LANES / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
        // the largest finite one goes to [2^15, 2^16), of which rounding toward zero leaves the type's
        // largest number at most: exponents stay where 2^e and 2^-e are normal numbers
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 15;
        e = e < -126 ? -126 : e;
        if (top == 0.0f) e = 0;
        up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int u = 0; u < PAIRS; ++u) {
          v[m][u].x *= down;
          v[m][u].y *= down;
        }
      }
      if (row[m] >= 0) {
        const int to0 = ALL ? rank : 0, to1 = ALL ? rank + 1 : C;
#pragma unroll
        for (int u = 0; u < PAIRS; ++u) {
          uint32_t h, l, at_h, at_l;
          split2<BF16>(v[m][u].x, v[m][u].y, h, l);
          place(row[m], 2 * (at_lane + LANES * u), at_h, at_l);
          for (int r = to0; r < to1; ++r) {
            st_cluster_u32(map_to_rank(at_h, static_cast<uint32_t>(r)), h);
            st_cluster_u32(map_to_rank(at_l, static_cast<uint32_t>(r)), l);
          }
        }
        if (at_lane == 0)
          for (int r = to0; r < to1; ++r) st_cluster_f32(map_to_rank(ptx::smem_u32(power + row[m]), static_cast<uint32_t>(r)), up);
      }
      __syncwarp();
    }
  }
}

// Rows of tokens without an adapter: base, or zeros.  An item is 2 KB of 32 tokens; every warp
// of the grid takes its share when its other work is done, and looks at the tokens of its
// first item as it starts.  A row out of range is reported and counts as none.  In place the
// tokens are looked at for that alone.
struct Others {
  const LoraArgs& a;
  const bool in_place;
  const uint32_t worker, workers, parts, items;
  bool first;
  static constexpr int kPart = 4;

  __device__ __forceinline__ Others(const LoraArgs& args, uint32_t w, uint32_t n)
      : a(args), in_place(args.base == args.out), worker(w), workers(n),
        parts(in_place ? 1u : (static_cast<uint32_t>(args.N) / 8 + 32 * kPart - 1) / (32 * kPart)),
        items(n == 0u ? 0u : (static_cast<uint32_t>(args.T) + 31) / 32 * parts) {
    first = worker < items && look(worker);
  }
  // whether this lane's token of an item is one
  __device__ __forceinline__ bool look(uint32_t it) const {
    const uint32_t t = it / parts * 32 + (threadIdx.x & 31);
    if (t >= static_cast<uint32_t>(a.T)) return false;
    const int row = ptx::ld_global(a.rows + t);
    if (row < -1 || row >= a.M) atomicOr(a.status, FGF8_DEVERR_INPUT);
    return row < 0 || row >= a.M;
  }
  __device__ __forceinline__ void fill() const {
    const int lane = static_cast<int>(threadIdx.x & 31), vecs = a.N / 8;
    for (uint32_t it = worker; it < items; it += workers) {
      const int v0 = static_cast<int>(it % parts) * 32 * kPart + lane;
      for (uint32_t left = __ballot_sync(kFull, (it == worker ? first : look(it)) && !in_place); left != 0; left &= left - 1) {
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
  constexpr int UNROLL = RP <= 32 ? 4 : RP <= 64 ? 2 : 1;    // steps of 32 columns of K in flight
  constexpr int LDP = RP + 4;                               // floats of a row of sums in shared memory
  constexpr int LDH = RP + 8;                               // 16-bit values of a row of P
  const LoraArgs& a = args.a;
  extern __shared__ __align__(16) uint8_t smem[];
  float* part = reinterpret_cast<float*>(smem);             // [warp][16][LDP] sums over a share of K
  uint16_t* hi = reinterpret_cast<uint16_t*>(part + kWarps * 16 * LDP);  // [16][LDH]
  uint16_t* lo = hi + 16 * LDH;
  float* power = reinterpret_cast<float*>(lo + 16 * LDH);   // [16] what a row of P is to be multiplied by
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int q = lane >> 2, c = lane & 3;
  const int C = static_cast<int>(gridDim.z), rank = static_cast<int>(blockIdx.z);      // the cluster is (1, 1, C)
  __shared__ float tile_scale;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  const Others others(a, cta_of_grid() * kWarps + warp, gridDim.x * gridDim.y * gridDim.z * kWarps);

  // the tile's adapter and tokens
  const long long row0 = static_cast<long long>(blockIdx.x) * 16;
  int id = -1, token = -1;
  if (lane < 16) {
    id = ptx::ld_global(a.m_indices + row0 + lane);
    token = ptx::ld_global(a.src + row0 + lane);
  }
  int g = __shfl_sync(kFull, id, 0);
  // rows of another adapter, adapters and tokens out of range are reported and left alone
  bool bad = id < -1 || token < -1 || id >= a.G || (id >= 0 && token >= 0 && (id != g || token >= a.T));
  if (g >= a.G) g = -1;
  if (bad || id < 0 || token < 0) token = -1;
  if (bad) atomicOr(a.status, FGF8_DEVERR_INPUT);
  if (g < 0) {                                              // the same for every warp of the cluster
    others.fill();
    return;
  }
  const int t0 = __shfl_sync(kFull, token, q), t1 = __shfl_sync(kFull, token, q + 8);

  // this CTA's part of N, whose rows of B are asked into L2 while A is read
  const int nblocks = (a.N + 31) / 32;
  const long long nshare = static_cast<long long>(blockIdx.y) * C + rank, nshares = static_cast<long long>(gridDim.y) * C;
  const int nb0 = static_cast<int>(nblocks * nshare / nshares), nb1 = static_cast<int>(nblocks * (nshare + 1) / nshares);
  const uint16_t* bg = static_cast<const uint16_t*>(a.B) + static_cast<size_t>(g) * a.N * a.r;
  {
    const char *from = reinterpret_cast<const char*>(bg + static_cast<size_t>(nb0) * 32 * a.r),
               *to = reinterpret_cast<const char*>(bg + static_cast<size_t>(min(nb1 * 32, a.N)) * a.r);
    for (const char* p = from + 128 * tid; p < to; p += 128 * kThreads) gemv::prefetch_l2(p);
  }

  // ------------------------------------------------------------ X A^T over a share of K
  const int share = rank * kWarps + warp, shares = C * kWarps;
  const int kblocks = (a.K + 31) / 32;
  const int kb0 = static_cast<int>(static_cast<long long>(kblocks) * share / shares);
  const int kb1 = static_cast<int>(static_cast<long long>(kblocks) * (share + 1) / shares);
  float acc[NB][4] = {};
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
  if (tid == 0) tile_scale = a.scale != nullptr ? ptx::ld_global(a.scale + g) : 1.0f;
  {
    float* p = part + warp * 16 * LDP;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      *reinterpret_cast<float2*>(p + q * LDP + 8 * b + 2 * c) = make_float2(acc[b][0], acc[b][1]);
      *reinterpret_cast<float2*>(p + (q + 8) * LDP + 8 * b + 2 * c) = make_float2(acc[b][2], acc[b][3]);
    }
  }
  __syncthreads();
  for (int i = tid; i < 16 * RP; i += kThreads) {
    const int at = i / RP * LDP + i % RP;
    float sum = part[at];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum += part[w * 16 * LDP + at];
    part[at] = sum;
  }

  // a block of 32 columns of out: what it adds to and B's rows for it, at this lane's columns
  constexpr int KS = RP >= 32 ? RP / 32 : 1;                // steps of 32 rank rows (of 16 when there are no more)
  struct Block {
    uint4 base[2];
    uint4 b[4][KS];
  };
  auto load_block = [&](int nb, Block& v) {
    const int n0 = nb * 32 + 8 * c;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int t = half ? t1 : t0;
      v.base[half] = make_uint4(0u, 0u, 0u, 0u);
      if (a.base != nullptr && nb < nb1 && n0 < a.N && t >= 0)
        v.base[half] = ptx::ld_global_v4(static_cast<const uint16_t*>(a.base) + static_cast<size_t>(t) * a.ldb + n0);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = nb * 32 + 8 * (q >> 1) + 2 * j + (q & 1);
      const uint16_t* bn = bg + static_cast<size_t>(n) * a.r;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        v.b[j][s] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (RP >= 32) {
          if (nb < nb1 && n < a.N && 32 * s + 8 * c < a.r) v.b[j][s] = ptx::ld_global_v4(bn + 32 * s + 8 * c);
        } else {
          if (nb < nb1 && n < a.N && 4 * c < a.r) {
            const uint2 w = ld_global_v2(bn + 4 * c);
            v.b[j][s].x = w.x;
            v.b[j][s].y = w.y;
          }
        }
      }
    }
  };
  // the first block, and where registers allow the second, come while P is exchanged
  constexpr bool kTwo = RP <= 32;
  Block even, odd;
  load_block(nb0 + warp, even);
  if (kTwo) load_block(nb0 + warp + kWarps, odd);
  // every CTA sums all rows, and they meet once
  if (C > 1) cluster_sync_all(); else __syncthreads();
  exchange_rows<BF16, RP, true>(part, power, 16, a.r, &tile_scale, C, rank, [&](int row, int col, uint32_t& at_h, uint32_t& at_l) {
    at_h = ptx::smem_u32(hi + row * LDH + col);
    at_l = ptx::smem_u32(lo + row * LDH + col);
  });
  cluster_arrive();                                         // behind this nothing remote is touched
  __syncthreads();

  // ------------------------------------------------------------ P B^T over a share of N
  uint32_t ph[KS][8], pl[KS][8];                            // [row q: 4 words][row q + 8: 4 words]
  {
    const uint16_t *h0 = hi + q * LDH, *l0 = lo + q * LDH;
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
  const float up0 = power[q], up1 = power[q + 8];
  auto finish = [&](int nb, const Block& v) {
    __syncwarp();                                           // the instructions below are whole-warp ones
    float d[4][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        gemv::mma16816<BF16>(d[j], ph[s][0], ph[s][4], ph[s][1], ph[s][5], v.b[j][s].x, v.b[j][s].y);
        gemv::mma16816<BF16>(d[j], pl[s][0], pl[s][4], pl[s][1], pl[s][5], v.b[j][s].x, v.b[j][s].y);
        if constexpr (RP >= 32) {
          gemv::mma16816<BF16>(d[j], ph[s][2], ph[s][6], ph[s][3], ph[s][7], v.b[j][s].z, v.b[j][s].w);
          gemv::mma16816<BF16>(d[j], pl[s][2], pl[s][6], pl[s][3], pl[s][7], v.b[j][s].z, v.b[j][s].w);
        }
      }
    const int n0 = nb * 32 + 8 * c;                         // this lane's 8 columns of out
    if (n0 < a.N) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int t = half ? t1 : t0;
        if (t < 0) continue;
        const float up = half ? up1 : up0;
        const uint32_t bw[4] = {v.base[half].x, v.base[half].y, v.base[half].z, v.base[half].w};
        uint32_t ow[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ow[j] = pack_2x16(fmaf(up, d[j][2 * half], act::to_float(bw[j] & 0xFFFFu, BF16)),
                            fmaf(up, d[j][2 * half + 1], act::to_float(bw[j] >> 16, BF16)), BF16);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + static_cast<size_t>(t) * a.ldo + n0) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
      }
    }
  };
  if constexpr (kTwo) {
    for (int nb = nb0 + warp; nb < nb1; nb += 2 * kWarps) {
      finish(nb, even);
      load_block(nb + 2 * kWarps, even);
      if (nb + kWarps < nb1) finish(nb + kWarps, odd);
      load_block(nb + 3 * kWarps, odd);
    }
  } else {
    for (int nb = nb0 + warp; nb < nb1; nb += kWarps) {
      finish(nb, even);
      load_block(nb + kWarps, even);
    }
  }
  __syncwarp();
  others.fill();
  cluster_wait();                                           // a CTA stays until all have read its sums
}

// ----------------------------------------------------------------- many tokens of an adapter
// The same two products for blocks of 128 rows with one adapter, on tcgen05: a byte of A or B
// serves 128 tokens, and the multiplications (2 r of them, with P in two parts 3 r, for each
// element of X, base and out) are off the warps' hands.
//   X A^T  [128 x r] in TMEM, K in steps of 64 through a ring of KSTAGES: the tokens' rows of X
//          by cp.async from four warps, a tile of A by TMA.  (TMA's tile::gather4 takes some 80
//          cycles for four rows of 128 bytes: 137 us for the calls below, whatever the rank.)
//   P      over the cluster as above, written as two more operands.
//   P B^T  [128 x 64] twice in TMEM, through another ring in its place: B and the tokens' rows
//          of base by cp.async.  Four warps add base to the even blocks and four to the odd ones,
//          a row per thread as TMEM gives it, put the sums where base stood, and store 128 bytes
//          of four rows at a time.
// All operands are K-major with 128-byte swizzle, rows of 64 columns.  Warps that copy, multiply
// and add wait for one another on mbarriers only: with a block-wide barrier for each step the
// same work took 86 us, and a third of that went to threads whose proxy fence waited for their
// own copies.  8192 tokens of 8 adapters, 7168 x 7168: 64 us at rank 16, 72 at 64 (5.1 TB/s),
// 95 at 128, where one CTA fills the SM; the bytes alone take 54 to 57.  At rank 64 X A^T is done
// after 28 us and P after 34, and the rest streams at 7 TB/s.  No gain from columns dealt to the
// cluster's CTAs in turn, nor from asking base into L2 while P is exchanged.
constexpr int kStages = 3, kWideRows = 128, kCopyWarps = 4;
constexpr int kWideThreads = kThreads + 32 * kCopyWarps + 32;   // sums and adding, copies, MMAs

template <int RP>
struct WideCfg {
  static constexpr int LDP = RP + 4;
  static constexpr int XBYTES = kWideRows * 128, KSTAGE = XBYTES + RP * 128;   // 64 columns of X and of A
  static constexpr int KB = (RP + 63) / 64;                 // blocks of 64 rank columns
  static constexpr int NB = 64;                             // rows of B in a block
  static constexpr int NSTAGE = KB * NB * 128, BSTAGE = kWideRows * NB * 2;    // a block of B, of base
  static constexpr int PART = (kWideRows * LDP * 4 + 1023) / 1024 * 1024;
  // stages of base, the sums over the later ones of them, stages of B, the two parts of P; the
  // stages of X and A lie over all of it
  static constexpr int EARLY = RP == 64 ? 1 : 2;            // stages of base before the sums
  static constexpr int OFF_PART = EARLY * BSTAGE;
  static constexpr int OFF_B = OFF_PART + PART > kStages * BSTAGE ? OFF_PART + PART : kStages * BSTAGE;
  static constexpr int PBYTES = KB * kWideRows * 128;
  static constexpr int OFF_HI = OFF_B + kStages * NSTAGE, OFF_LO = OFF_HI + PBYTES, OFF_POWER = OFF_LO + PBYTES;
  static constexpr int KSTAGES = OFF_POWER / KSTAGE;
  static constexpr int SMEM = OFF_POWER + kWideRows * 4 + 1024;   // the layout starts on 1024 bytes
  static_assert(KSTAGES >= 3 && SMEM <= (RP <= 64 ? 112 : 224) * 1024, "shared memory of one or two CTAs");
  static constexpr int COL_D = 128;                         // TMEM: X A^T from column 0, two blocks of P B^T from here
  static constexpr int TMEM = 256;
};

// Stage and parity of the uses of a ring, one after the other.
template <int STAGES>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == STAGES) s = 0, phase ^= 1u;
  }
};

// Byte of 16-bit column `col` of row `row` in blocks of 64 columns, 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int rows, int row, int col) {
  return static_cast<uint32_t>((col >> 6) * rows * 128 + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2);
}
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
// 16 bytes of a row into shared memory, zeros where there are none; the row's next bytes are
// asked into L2 with them.
__device__ __forceinline__ void cp16_row(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// This thread's arrival on a barrier, when all its cp.async so far have come.
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <bool BF16, int RP>
__global__ void __launch_bounds__(kWideThreads, RP <= 64 ? 2 : 1) lora_f16_wide_kernel(const __grid_constant__ CUtensorMap map_a,
                                                                                       const __grid_constant__ LoraKArgs args) {
  using Cf = WideCfg<RP>;
  const LoraArgs& a = args.a;
  extern __shared__ __align__(128) uint8_t raw[];
  __shared__ int tokens[kWideRows];                         // -1 where a row has none
  __shared__ float block_scale;
  __shared__ uint64_t bars[2 * Cf::KSTAGES + 2 * kStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_word;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int C = static_cast<int>(gridDim.z), rank = static_cast<int>(blockIdx.z);
  uint8_t* smem = raw + ((1024u - (ptx::smem_u32(raw) & 1023u)) & 1023u);   // the same offset in every CTA
  float* part = reinterpret_cast<float*>(smem + Cf::OFF_PART);
  float* power = reinterpret_cast<float*>(smem + Cf::OFF_POWER);
  const uint32_t base_s = ptx::smem_u32(smem);
  auto bar = [&](int i) { return ptx::smem_u32(&bars[i]); };
  constexpr int NBARS = 2 * Cf::KSTAGES, DBARS = NBARS + 2 * kStages;
  auto kfull = [&](int s) { return bar(s); };               // a stage of X and A has come, has been read
  auto kfree = [&](int s) { return bar(Cf::KSTAGES + s); };
  auto nfull = [&](int s) { return bar(NBARS + s); };       // a stage of B and base
  auto nfree = [&](int s) { return bar(NBARS + kStages + s); };
  auto dfull = [&](int d) { return bar(DBARS + d); };       // a block of P B^T is in TMEM, has been taken out
  auto dfree = [&](int d) { return bar(DBARS + 2 + d); };
  const uint32_t kdone = bar(DBARS + 4);                    // X A^T is in TMEM
  if (tid == 0) {
    for (int s = 0; s < Cf::KSTAGES; ++s) {
      ptx::mbar_init(kfull(s), 1 + 32 * kCopyWarps);
      ptx::mbar_init(kfree(s), 1);
    }
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(nfull(s), 32 * kCopyWarps);
      ptx::mbar_init(nfree(s), 1 + kWarps / 2);
    }
    for (int d = 0; d < 2; ++d) {
      ptx::mbar_init(dfull(d), 1);
      ptx::mbar_init(dfree(d), kWarps / 2);
    }
    ptx::mbar_init(kdone, 1);
    abort_word = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == kWarps && lane == 0) ptx::prefetch_tmap(&map_a);
  ptx::griddep_wait();

  const Others others(a, cta_of_grid() * kWarps + warp, warp < kWarps ? gridDim.x * gridDim.y * gridDim.z * kWarps : 0u);
  // the block's adapter and tokens
  const long long row0 = static_cast<long long>(blockIdx.x) * kWideRows;
  int g = ptx::ld_global(a.m_indices + row0);
  if (tid < kWideRows) {
    const int id = ptx::ld_global(a.m_indices + row0 + tid), t = ptx::ld_global(a.src + row0 + tid);
    const bool bad = id < -1 || t < -1 || id >= a.G || (id >= 0 && t >= 0 && (id != g || t >= a.T));
    tokens[tid] = bad || id < 0 ? -1 : t;                   // t is -1 where there is none
    if (bad) atomicOr(a.status, FGF8_DEVERR_INPUT);
  }
  if (g >= a.G) g = -1;
  if (tid == 0) block_scale = a.scale != nullptr && g >= 0 ? ptx::ld_global(a.scale + g) : 1.0f;
  if (g < 0) {                                              // the same for every CTA of the cluster
    others.fill();
    return;
  }
  if (warp == kWarps + kCopyWarps) {
    tc_alloc<1>(ptx::smem_u32(&tmem_slot), Cf::TMEM);
    ptx::tc_fence_before();
  }
  __syncthreads();
  // Not before this CTA holds its tensor memory: the next kernel's CTAs take theirs before they
  // wait for this grid, and one that fitted beside this CTA would hold what it waits for.
  ptx::griddep_launch_dependents();
  ptx::tc_fence_after();
  const uint32_t tmem = *const_cast<volatile uint32_t*>(&tmem_slot);
  PairWaitCtl ctl{&abort_word, 0u, a.status, args.timeout_ns, 0u};
  constexpr uint32_t kFmt = BF16 ? 1u : 0u;

  const int ksteps = (a.K + 63) / 64, nblocks = (a.N + Cf::NB - 1) / Cf::NB;
  const int ks0 = static_cast<int>(static_cast<long long>(ksteps) * rank / C), ks1 = static_cast<int>(static_cast<long long>(ksteps) * (rank + 1) / C);
  const int nb0 = static_cast<int>(static_cast<long long>(nblocks) * rank / C), nb1 = static_cast<int>(static_cast<long long>(nblocks) * (rank + 1) / C);
  if (warp >= kWarps && warp < kWarps + kCopyWarps) {
    // ---------------------------------------------------------- copies
    ctl.role_bit = FGF8_DEVERR_ROLE_PRODUCER;
    constexpr int kRows = 4 * kCopyWarps;                   // copied together: 8 pieces of a row by 8 lanes
    const int me = tid - kThreads, prow = me >> 3, pcol = me & 7;
    const bool first = me == 0;                             // who also asks for the tiles of A
    const uint16_t* from[kWideRows / kRows];                // this lane's pieces of its rows, at column 0
    int bytes[kWideRows / kRows];                           // 16, or 0 for a row without a token
    auto rows_of = [&](const void* matrix, long long ld) {
#pragma unroll
      for (int i = 0; i < kWideRows / kRows; ++i) {
        const int t = tokens[prow + kRows * i];
        bytes[i] = t >= 0 ? 16 : 0;
        from[i] = static_cast<const uint16_t*>(matrix) + (t >= 0 ? static_cast<long long>(t) * ld : 0) + 8 * pcol;
      }
    };
    // 64 columns from `col` on
    auto copy_rows = [&](uint32_t to, int col, int cols) {
      const uint32_t at = to + swizzled(0, prow, 8 * pcol);
      const bool in = col + 8 * pcol < cols;
#pragma unroll
      for (int i = 0; i < kWideRows / kRows; ++i)
        cp16_row(at + static_cast<uint32_t>(i * kRows * 128), in ? from[i] + col : from[i], in ? bytes[i] : 0);
    };
    rows_of(a.X, a.ldx);
    bool ok = true;
    Ring<Cf::KSTAGES> r;
    for (int ks = ks0; ks < ks1; ++ks) {
      ok = pwait(kfree(r.s), r.phase ^ 1u, ctl);
      if (!ok) break;
      const uint32_t to = base_s + static_cast<uint32_t>(r.s * Cf::KSTAGE);
      if (first) {
        ptx::mbar_arrive_expect_tx(kfull(r.s), static_cast<uint32_t>(a.r * 128));
        ptx::tma_load_2d(to + Cf::XBYTES, &map_a, kfull(r.s), ks * 64, g * a.r);
      }
      copy_rows(to, ks * 64, a.K);
      cp_arrive(kfull(r.s));
      r.next();
    }
    // shared memory changes hands: B's stages when X A^T is done, base's when P has been exchanged
    if (ok && ks1 > ks0) ok = pwait(kdone, 0u, ctl);
    const uint16_t* bg = static_cast<const uint16_t*>(a.B) + static_cast<size_t>(g) * a.N * a.r;
    auto load_b = [&](int nb, int s) {
      constexpr int PIECES = RP / 8;                        // of a row
#pragma unroll
      for (int i = 0; i < Cf::NB * PIECES / (32 * kCopyWarps); ++i) {
        const int at = me + 32 * kCopyWarps * i, brow = at / PIECES, piece = at % PIECES, n = nb * Cf::NB + brow;
        const bool have = n < a.N && 8 * piece < a.r;
        gemv::cp16(base_s + static_cast<uint32_t>(Cf::OFF_B + s * Cf::NSTAGE) + swizzled(Cf::NB, brow, 8 * piece),
                   have ? bg + static_cast<size_t>(n) * a.r + 8 * piece : bg, have);
      }
    };
    for (int s = 0; ok && s < kStages && nb0 + s < nb1; ++s) load_b(nb0 + s, s);
    rows_of(a.base, a.ldb);
    Ring<kStages> n;
    auto load_base = [&](int nb) {
      if (a.base != nullptr) copy_rows(base_s + static_cast<uint32_t>(n.s * Cf::BSTAGE), nb * Cf::NB, a.N);
      cp_arrive(nfull(n.s));
      n.next();
    };
    int nb = nb0;
    for (; ok && nb < nb1 && nb < nb0 + Cf::EARLY; ++nb) load_base(nb);
    __syncwarp();
    cluster_sync_all();
    cluster_sync_all();
    for (; ok && nb < nb1; ++nb) {
      if (nb >= nb0 + kStages) {
        ok = pwait(nfree(n.s), n.phase ^ 1u, ctl);
        if (!ok) break;
        load_b(nb, n.s);
      }
      load_base(nb);
    }
    gemv::cp_commit();
    gemv::cp_wait<0>();
    __syncwarp();
  } else if (warp == kWarps + kCopyWarps) {
    // ---------------------------------------------------------- MMAs
    ctl.role_bit = FGF8_DEVERR_ROLE_MMA;
    bool ok = true;
    Ring<Cf::KSTAGES> r;
    for (int ks = ks0; ks < ks1; ++ks) {
      ok = pwait(kfull(r.s), r.phase, ctl);
      if (!ok) break;
      ptx::tc_fence_after();
      if (lane == 0) {
        // the copies are for the tensor core; here, because a thread that fences waits for all
        // its own copies under way
        ptx::fence_proxy_async_smem();
        const uint32_t s = base_s + static_cast<uint32_t>(r.s * Cf::KSTAGE);
        const uint64_t xd = smem_desc_sw128(s), ad = smem_desc_sw128(s + Cf::XBYTES);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ptx::mma_f16(tmem, xd + 2 * k, ad + 2 * k, idesc_dense(kFmt, kFmt, RP, 128), ks > ks0 || k > 0 ? 1u : 0u);
        ptx::mma_commit(kfree(r.s));
        if (ks + 1 == ks1) ptx::mma_commit(kdone);
      }
      __syncwarp();
      r.next();
    }
    cluster_sync_all();
    cluster_sync_all();
    fence_proxy_async_all();                                // P is read by the tensor core
    Ring<kStages> n;
    for (int nb = nb0; ok && nb < nb1; ++nb) {
      const int d = (nb - nb0) & 1;
      ok = pwait(nfull(n.s), n.phase, ctl) && (nb < nb0 + 2 || pwait(dfree(d), (static_cast<uint32_t>(nb - nb0 - 2) >> 1) & 1u, ctl));
      if (!ok) break;
      ptx::tc_fence_after();
      if (lane == 0) {
        ptx::fence_proxy_async_smem();
        const uint32_t s = base_s + Cf::OFF_B + static_cast<uint32_t>(n.s * Cf::NSTAGE);
        const uint32_t to = tmem + static_cast<uint32_t>(Cf::COL_D + Cf::NB * d);
#pragma unroll
        for (int k = 0; k < RP / 16; ++k) {
          const uint64_t bd = smem_desc_sw128(s + static_cast<uint32_t>((k >> 2) * Cf::NB * 128)) + 2 * (k & 3);
          const uint32_t p = base_s + Cf::OFF_HI + static_cast<uint32_t>((k >> 2) * kWideRows * 128);
          ptx::mma_f16(to, smem_desc_sw128(p) + 2 * (k & 3), bd, idesc_dense(kFmt, kFmt, Cf::NB, 128), k > 0 ? 1u : 0u);
          ptx::mma_f16(to, smem_desc_sw128(p + Cf::PBYTES) + 2 * (k & 3), bd, idesc_dense(kFmt, kFmt, Cf::NB, 128), 1u);
        }
        ptx::mma_commit(nfree(n.s));
        ptx::mma_commit(dfull(d));
      }
      __syncwarp();
      n.next();
    }
  } else {
    // ---------------------------------------------------------- sums, exchange, adding
    ctl.role_bit = FGF8_DEVERR_ROLE_EPILOGUE;
    const int row = 32 * (warp & 3) + lane, half = warp >> 2;   // this thread's row, and half of the columns
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    bool ok = ks1 == ks0 || pwait(kdone, 0u, ctl);
    ptx::tc_fence_after();
    if (RP >= 32 || half == 0) {
      constexpr int COLS = RP >= 32 ? RP / 2 : 16, STEP = COLS < 32 ? COLS : 32;
#pragma unroll
      for (int c = 0; c < COLS; c += STEP) {
        uint32_t v[STEP];
        tmem_ld_chunk(lanes + static_cast<uint32_t>(half * COLS + c), v);
        ptx::tmem_wait_ld();
        ptx::reg_fence(v);
        float4* to = reinterpret_cast<float4*>(part + row * Cf::LDP + half * COLS + c);
        // rank columns from r on hold what the stage's last rows happened to be
#pragma unroll
        for (int i = 0; i < STEP / 4; ++i)
          to[i] = ks1 > ks0
                      ? make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]))
                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    }
    cluster_sync_all();
    exchange_rows<BF16, RP, false>(part, power, kWideRows, a.r, &block_scale, C, rank, [&](int r, int col, uint32_t& at_h, uint32_t& at_l) {
      at_h = base_s + Cf::OFF_HI + swizzled(kWideRows, r, col);
      at_l = at_h + Cf::PBYTES;
    });
    fence_proxy_async_all();                                // the MMAs of every CTA read P; copies overwrite the sums
    cluster_sync_all();                                     // and nothing remote is touched behind this
    const float up = power[row];
    // four warps take the even blocks, four the odd ones
    int token[8];                                           // of rows 4 i + lane / 8, of which this lane stores 16 bytes
#pragma unroll
    for (int i = 0; i < 8; ++i) token[i] = tokens[32 * (warp & 3) + 4 * i + (lane >> 3)];
    Ring<kStages> n;
    if (half == 1) n.next();
    for (int nb = nb0 + half; ok && nb < nb1; nb += 2) {
      const int d = half;
      ok = pwait(dfull(d), (static_cast<uint32_t>(nb - nb0) >> 1) & 1u, ctl) && pwait(nfull(n.s), n.phase, ctl);
      if (!ok) break;
      ptx::tc_fence_after();
      uint8_t* mine = smem + n.s * Cf::BSTAGE;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
        tmem_ld_chunk(lanes + static_cast<uint32_t>(Cf::COL_D + Cf::NB * d + 32 * c), v);
        ptx::tmem_wait_ld();
        ptx::reg_fence(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint8_t* p = mine + swizzled(0, row, 32 * c + 8 * i);
          uint32_t b[4] = {0u, 0u, 0u, 0u}, o[4];
          if (a.base != nullptr) gemv::lds128(p, b);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = pack_2x16(fmaf(up, __uint_as_float(v[8 * i + 2 * j]), act::to_float(b[j] & 0xFFFFu, BF16)),
                             fmaf(up, __uint_as_float(v[8 * i + 2 * j + 1]), act::to_float(b[j] >> 16, BF16)), BF16);
          *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(dfree(d));
      const int col = nb * Cf::NB + 8 * (lane & 7);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (token[i] >= 0 && col < a.N) {
          uint32_t o[4];
          gemv::lds128(mine + swizzled(0, 32 * (warp & 3) + 4 * i + (lane >> 3), 8 * (lane & 7)), o);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + static_cast<size_t>(token[i]) * a.ldo + col) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(nfree(n.s));
      n.next();
      n.next();
    }
    __syncwarp();
    others.fill();
  }
  // everything asked for has come and has been read, unless a wait ran out: then it gets a while
  // before shared memory and TMEM are given back
  if (__syncthreads_or(abort_word != 0u ? 1 : 0)) {
    const uint64_t since = ptx::globaltimer();
    while (ptx::globaltimer() - since < 200000ull) __nanosleep(1000);
  }
  if (warp == kWarps + kCopyWarps) {
    ptx::tc_fence_after();
    tc_dealloc<1>(tmem, Cf::TMEM);
  }
}

// Tiles of 16 rows with a token in them: all of them in segments of 16 rows; in longer ones, which
// end in empty tiles, at most a partly filled one for each adapter.
long long used_tiles(const LoraArgs& a) {
  const long long most = a.M / 16, est = a.T / 16 + (a.T < a.G ? a.T : a.G) + 1;
  return est < most ? est : most;
}

// Shared memory of a CTA with one tile.
template <int RP>
constexpr int kTileSmem = kWarps * 16 * (RP + 4) * 4 + 2 * 16 * (RP + 8) * 2 + 16 * 4;

struct LoraLaunch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  LoraLaunch(long long groups, int parts, int cluster, int threads, int smem, cudaStream_t stream, bool pdl) {
    std::memset(&cfg, 0, sizeof(cfg));
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = static_cast<unsigned>(cluster);
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(groups), static_cast<unsigned>(parts), static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
  }
};

template <bool BF16, int RP>
int launch_tiles(const LoraArgs& a, cudaStream_t stream) {
  auto* fn = &lora_f16_kernel<BF16, RP>;
  static PerDevice<int> ready;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  const int* set = nullptr;
  const int r = ready.get(dev, &set, [&](int& v) {
    v = kTileSmem<RP>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
    return e == cudaSuccess ? 0 : set_error(4, "lora_f16 set-up: %s", cudaGetErrorString(e));
  });
  if (r) return r;
  // A cluster's CTAs split K and N: eight, unless a warp's share of K falls below 32 columns or
  // the tiles' CTAs are a third more than run together (some tiles are empty).  Clusters that
  // share a tile's N, and each compute P, help up to 64 CTAs with 4 KB of B each.  Over 15
  // shapes of 1 to 2000 tokens this is within 4 % of the best of all splits at eleven and at most
  // 15 % slower (7.8 us for 6.8, 24 tokens of 32 adapters, 2048 x 8192).  Empty
  // tiles have CTAs too, so a layout of more than kMostCtas with these splits goes without: launching
  // them is the time there, and their warps are counted in 32 bits.
  const long long tiles = used_tiles(a), slots = (RP <= 64 ? 2LL : 1LL) * device_sm_count(), bytes = 2LL * a.N * a.r;
  int cluster = kMaxCluster, parts = 1;
  while (cluster > 1 && (256 * cluster > a.K || 3 * tiles * cluster > 4 * slots)) cluster /= 2;
  while (2 * parts * cluster <= (a.N + 31) / 32 && 2 * parts * cluster * tiles <= 64 && bytes / (2 * parts * cluster) >= 4096) parts *= 2;
  constexpr long long kMostCtas = 1 << 24;
  if (a.M / 16 * parts > kMostCtas / cluster) cluster = parts = 1;
  LoraKArgs k;
  k.a = a;
  k.timeout_ns = 0;                                         // this form waits on no mbarrier
  set_last_tile("f16", "lora", cluster, 16);
  LoraLaunch l(a.M / 16, parts, cluster, kThreads, kTileSmem<RP>, stream, pdl_enabled());
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, fn, k);
  return e == cudaSuccess ? 0 : set_error(4, "lora_f16 launch: %s", cudaGetErrorString(e));
}

// Clusters of 1, 2, 4 and 8 CTAs that run on the device together.
struct Fit {
  int clusters[4];
};
template <typename K>
int find_fit(K* fn, PerDevice<Fit>& fits, int threads, int smem, const Fit** out) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  return fits.get(dev, out, [&](Fit& f) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    for (int i = 0; e == cudaSuccess && i < 4; ++i) {
      LoraLaunch l(device_sm_count(), 1, 1 << i, threads, smem, nullptr, false);
      e = cudaOccupancyMaxActiveClusters(&f.clusters[i], fn, &l.cfg);
      if (e == cudaSuccess && f.clusters[i] <= 0) e = cudaErrorInvalidConfiguration;
    }
    return e == cudaSuccess ? 0 : set_error(4, "lora_f16 set-up: %s", cudaGetErrorString(e));
  });
}

template <bool BF16, int RP>
int launch_wide(const LoraArgs& a, cudaStream_t stream) {
  using Cf = WideCfg<RP>;
  static_assert(Cf::SMEM <= 232448 - 2048, "shared memory budget");
  static PerDevice<Fit> fits;
  const Fit* fit = nullptr;
  if (const int r = find_fit(&lora_f16_wide_kernel<BF16, RP>, fits, kWideThreads, Cf::SMEM, &fit)) return r;
  LoraKArgs k;
  k.a = a;
  k.timeout_ns = wait_timeout_ns();
  // The cluster whose CTAs take the least time, in units of a whole block alone on an SM: each
  // takes its share and 0.08 for the start and the exchange of P, 1.28 times as long where two
  // are on an SM (up to rank 64; the occupancy query counts one CTA per SM for a kernel with
  // tensor memory).  At 7168 x 7168, rank 64, clusters of 1, 2, 4 and 8: 153, 91, 73 and 84 us
  // for 71 blocks, 155, 94, 114 and 107 for 76, which do not fit the device as fours.
  constexpr int kPerSm = RP <= 64 ? 2 : 1;
  constexpr double kShared = RP <= 64 ? 1.28 : 1.0;
  const long long groups = a.M / kWideRows;
  int cluster = 1;
  double best = 0.0;
  for (int i = 0; i < 4; ++i) {
    const int c = 1 << i;
    if (c > 1 && (a.K + 63) / 64 < 2 * c && (a.N + 63) / 64 < 2 * c) break;
    const long long alone = fit->clusters[i], waves = groups / (kPerSm * alone), rest = groups % (kPerSm * alone);
    const double time = (1.0 / c + 0.08) * (static_cast<double>(waves) * kShared + (rest == 0 ? 0.0 : rest <= alone ? 1.0 : kShared));
    if (c == 1 || time < best) {
      best = time;
      cluster = c;
    }
  }
  const CUtensorMapDataType dt = BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUtensorMap m;
  const uint64_t K = static_cast<uint64_t>(a.K);
  if (!encode_tmap_2d(&m, dt, a.A, K, static_cast<uint64_t>(a.G) * a.r, 2 * K, 64, static_cast<uint32_t>(a.r), true)) return 4;
  set_last_tile("f16", "lora", cluster, kWideRows);
  LoraLaunch l(groups, 1, cluster, kWideThreads, Cf::SMEM, stream, pdl_enabled());
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, &lora_f16_wide_kernel<BF16, RP>, m, k);
  return e == cudaSuccess ? 0 : set_error(4, "lora_f16 launch: %s", cudaGetErrorString(e));
}

// Blocks of 128 rows or tiles of 16, by the time each takes, in us.  Tiles: 5 and the bytes that
// leave L2, at 8.2 TB/s: X, base and out once, A and B once for every 16 tokens.  Blocks: 17 for
// the start, the exchange and the filling of the rings, and the bytes from memory at 6.3 TB/s, a
// third less where one CTA fills an SM.  Against times of both forms at 108 shapes (4 to 8192
// tokens of 4 and 32 adapters, 1024 x 1024 to 7168 x 7168, rank 16 to 128) the choice is the better
// one at 99 and within 8 % of it at all but three, where it is 13, 21 and 42 % slower (34 us for 24,
// 4096 tokens of 32 adapters, 1024 x 1024, rank 128); 4096 tokens of 32 adapters, 4096 x 4096: 29
// and 35 us at rank 16, 51 and 43 at 64.
// FGF8_FORCE_TILE=1x16 or 1x128 takes a form where the rows allow it.
bool wide_form(const LoraArgs& a) {
  // the copy engine counts the rows of all adapters' A in 32 bits
  if (a.align % kWideRows != 0 || static_cast<long long>(a.G) * a.r > kRouteMaxSize) return false;
  if (const char* f = std::getenv("FGF8_FORCE_TILE")) {
    if (std::strcmp(f, "1x16") == 0) return false;
    if (std::strcmp(f, "1x128") == 0) return true;
  }
  const double rows = 2.0 * a.T * (static_cast<double>(a.K) + 2.0 * a.N), adapter = 2.0 * a.r * (static_cast<double>(a.K) + a.N);
  const double tiles = 5.0 + (rows + used_tiles(a) * adapter) / 8.2e6;
  const double blocks = 17.0 + (rows + (a.T < a.G ? a.T : a.G) * adapter) / (a.r <= 64 ? 6.3e6 : 4.3e6);
  return blocks < tiles;
}

template <bool BF16, int RP>
int by_form(const LoraArgs& a, cudaStream_t stream) {
  return wide_form(a) ? launch_wide<BF16, RP>(a, stream) : launch_tiles<BF16, RP>(a, stream);
}

template <bool BF16>
int by_rank(const LoraArgs& a, cudaStream_t stream) {
  if (a.r <= 16) return by_form<BF16, 16>(a, stream);
  if (a.r <= 32) return by_form<BF16, 32>(a, stream);
  if (a.r <= 64) return by_form<BF16, 64>(a, stream);
  return by_form<BF16, 128>(a, stream);
}

}  // namespace

int launch_lora_f16(const LoraArgs& a, int bf16, cudaStream_t stream) {
  return bf16 ? by_rank<true>(a, stream) : by_rank<false>(a, stream);
}

}  // namespace fgf8
