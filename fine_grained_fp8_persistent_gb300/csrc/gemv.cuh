// gemv.cuh -- products of at most 16 rows of X with a weight matrix (or, gated, two),
// bound by reading the weights: Y[m][n] = sum_k X[m][k] W[n][k].
//
// The weights are the M operand of mma.sync m16n8k16 (16 weight rows per warp tile), the
// rows of X its N = 8 columns, so one to eight tokens cost the same; FP32 accumulation.
// Decoding is what the CUDA cores do:
//   16-bit   none: the weights go from shared memory into the MMA.
//   NVFP4    code * scale in fp16: an E2M1 value has 2 significant bits, an E4M3 scale 4,
//            and the product lies in 2^-10 .. 2688, so it is exact; the MMA accumulates
//            over the whole reduction.
//   MXFP4    the codes in fp16 (exact), one FP32 partial sum per group of 32, then
//            acc += partial * 2^e: scales reach 2^+-127, which no fp16 product holds.
// A 16-byte piece of a weight row holds 32 codes.  ldmatrix hands lane 4 g + t of the warp
// the 8 codes 8 t .. 8 t + 7 of row g; taken as two K = 16 instructions, instruction i
// multiplies codes 8 t + 4 i + {0, 1} and {2, 3} of lane t as its k = 2 t + {0, 1} and
// 2 t + 8 + {0, 1}.  The sum over k does not care for the order, so X needs no shuffle
// either: lane t's share of a row of X is 16 contiguous bytes.
//
// bf16 X is scaled, for each row and chunk of 256 columns, by the power of two that puts
// the largest finite |x| there into [2^14, 2^15), and converted to fp16, the type E2M1
// decodes to.  That is exact for every |x| of at least 2^-31 of the largest.  The chunk's
// sums are multiplied by the power's inverse as they are added to the totals.  Where a row
// of X holds smaller |x| too (they may be all that its weights leave: code 0 is common),
// it stays bf16, and a chunk with such a row is multiplied in bf16, where decoded weights
// are exact as well, at two to three times the instructions.
//
// Work split.  One CTA per SM, walking tiles of 16 weight rows in rounds; a warp takes one
// tile (of one of the two matrices, when gated) of the round, or, when there are fewer
// tiles than warps, every KS-th of the tile's 128-byte pieces ("chunks").  X (or as much of
// it as fits: a "piece") is converted and kept in shared memory once per CTA.  Each warp streams its chunks through a ring of its
// own with cp.async, which goes on across pieces and rounds, so the loop has no barrier,
// and keeps its sums in registers to the round's end.  The KS shares of a tile are then
// added in shared memory, in order.  With few rows, or with much more of X than fits, a
// cluster of CTAs splits the reduction further and adds its sums through distributed
// shared memory, also in order.
#pragma once
#include <cstring>

#include "activation.cuh"
#include "gated.h"
#include "gemm_persistent.cuh"
#include "per_device.h"

namespace fgf8 {

enum class WType : int { W16 = 0, MX = 1, NV = 2 };

struct GemvKArgs {
  const void* X;
  const void* W[2];
  const void* SF[2];
  void* out;
  void* keep[2];     // gated 16-bit: G and U, or null
  int M, N, K;
  int act;
  int cta_tiles;     // tiles of 16 weight rows per cluster, one more for the first `extra`
  int extra;
  int round_tiles;   // tiles of one round
  int ks;            // warps per tile and matrix
  int chunks;        // chunks of the whole reduction
  int cta_chunks;    // chunks of one CTA's share of it (every CTA has at least one)
  int x_chunks;      // chunks of X in shared memory at a time
  int x_stride;      // bytes between rows of X in shared memory
  int off_slots;     // offsets of the warps' sums [warp][M][16], of 2^p of each chunk
  int off_scale;     //   and row of X, and of X
  int off_x;
  int prefetch;      // chunks per warp to ask into L2 ahead of the previous kernel's end
};

// DEEP: 16 warps with as many bytes in flight as fit; else 12 warps with rings of three and
// half an SM's registers, so that the next kernel's CTAs can start beside it where the
// shared memory that the plan takes for X (up to all of it) leaves them room.
template <WType WT, int NT, bool DEEP>
struct GemvCfg {
  static constexpr int WARPS = DEEP ? 16 : 12;               // at most
  static constexpr int MIN_CTAS = DEEP ? 1 : 2;              // per SM: bounds the registers
  static constexpr int CK = WT == WType::W16 ? 64 : 256;     // elements of K per chunk (128 bytes of a row)
  static constexpr int WPC = WT == WType::MX ? 2 : 4;        // scale words per row and chunk
  static constexpr int SF_BYTES = WT == WType::W16 ? 0 : WPC * 64;
  static constexpr int STAGE = 2048 + SF_BYTES;
  static constexpr int DEPTH = DEEP && NT == 1 ? 5 : 3;   // ring slots of a warp
};

namespace gemv {

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp16_full(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4_full(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A B, no addend.
__device__ __forceinline__ void mma16816_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Eight E2M1 codes (low nibble first) to four fp16 pairs.
__device__ __forceinline__ void e2m1x8(uint32_t v, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(v));
}
// Four E8M0 bytes to FP32 (0 is 2^-127, 255 is NaN).
__device__ __forceinline__ void e8m0x4(uint32_t w, float (&s)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, l;\n\tcvt.rn.bf16x2.ue8m0x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
  s[0] = __uint_as_float(lo << 16);
  s[1] = __uint_as_float(lo & 0xFFFF0000u);
  s[2] = __uint_as_float(hi << 16);
  s[3] = __uint_as_float(hi & 0xFFFF0000u);
}
// An fp16 pair as a bf16 pair, times f; exact for decoded weights and for X scaled to fp16.
__device__ __forceinline__ uint32_t bf16_pair(uint32_t h, float f) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_2x16(v.x * f, v.y * f, true);
}
// The E4M3 byte `i` of w as an fp16 pair (value, value).
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, int i) {
  uint32_t h;
  const uint16_t two = static_cast<uint16_t>(__byte_perm(w, 0u, static_cast<uint32_t>(i | (i << 4))));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return h;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void lds128(const uint8_t* p, uint32_t (&r)[4]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  r[0] = v.x;
  r[1] = v.y;
  r[2] = v.z;
  r[3] = v.w;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

}  // namespace gemv

__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x;
  a.y += b.y;
  a.z += b.z;
  a.w += b.w;
}
// Four outputs (weight rows n .. n + 3, token m) from their FP32 sums.
__device__ __forceinline__ void store4(void* base, const GemvKArgs& args, int n, int m, const float4& v, bool bf16) {
  uint16_t* p = static_cast<uint16_t*>(base) + static_cast<size_t>(m) * args.N + n;
  const uint32_t lo = pack_2x16(v.x, v.y, bf16), hi = pack_2x16(v.z, v.w, bf16);
  if (args.N % 4 == 0) {                                  // 8-byte aligned, and all four rows or none
    *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
    return;
  }
  p[0] = static_cast<uint16_t>(lo);
  if (n + 1 < args.N) p[1] = static_cast<uint16_t>(lo >> 16);
  if (n + 2 < args.N) p[2] = static_cast<uint16_t>(hi);
  if (n + 3 < args.N) p[3] = static_cast<uint16_t>(hi >> 16);
}
template <bool BF16, int MATS>
__device__ __forceinline__ void gemv_store(const GemvKArgs& args, int n, int m, float4 (&v)[MATS]) {
  if (n >= args.N) return;
  if constexpr (MATS == 2) {
    if (args.keep[0] != nullptr) {
      store4(args.keep[0], args, n, m, v[0], BF16);
      store4(args.keep[1], args, n, m, v[1], BF16);
    }
    auto a = [&](float g) { return args.act == act::kSilu ? act::value<act::kSilu>(g) : act::value<act::kGeluTanh>(g); };
    v[0] = make_float4(a(v[0].x) * v[1].x, a(v[0].y) * v[1].y, a(v[0].z) * v[1].z, a(v[0].w) * v[1].w);
  }
  store4(args.out, args, n, m, v[0], BF16);
}

template <WType WT, bool BF16, int MATS, int NT, bool DEEP>
__global__ void __launch_bounds__(32 * GemvCfg<WT, NT, DEEP>::WARPS, GemvCfg<WT, NT, DEEP>::MIN_CTAS) gemv_kernel(const GemvKArgs args) {
  using C = GemvCfg<WT, NT, DEEP>;
  using namespace gemv;
  constexpr bool kScaleX = WT != WType::W16 && BF16;   // bf16 X against fp16 weight values
  constexpr bool kMmaBf16 = WT == WType::W16 && BF16;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int W = static_cast<int>(blockDim.x) / 32;
  const int g = lane >> 2, t = lane & 3;
  const int S = static_cast<int>(gridDim.y);            // CTAs of the cluster: shares of the reduction
  const int rank = static_cast<int>(blockIdx.y);
  const int M = args.M, N = args.N, K = args.K, KS = args.ks;
  const int tile0 = static_cast<int>(blockIdx.x) * args.cta_tiles + min(static_cast<int>(blockIdx.x), args.extra);
  const int my_tiles = args.cta_tiles + (static_cast<int>(blockIdx.x) < args.extra ? 1 : 0);
  // this warp's tile of the round, matrix and share of it
  const int wm = warp / KS, ks = warp - wm * KS, wt = wm / MATS;
  const uint8_t* const weights = static_cast<const uint8_t*>(MATS == 2 && wm % 2 != 0 ? args.W[1] : args.W[0]);
  const uint32_t* const scale_words = static_cast<const uint32_t*>(MATS == 2 && wm % 2 != 0 ? args.SF[1] : args.SF[0]);
  const int c0 = rank * args.cta_chunks;                 // first chunk of this CTA
  const int nc = min(args.cta_chunks, args.chunks - c0);
  constexpr int ELEM_BITS = WT == WType::W16 ? 16 : 4;
  const size_t row_bytes = static_cast<size_t>(K) * ELEM_BITS / 8;
  constexpr int SV = WT == WType::MX ? 32 : 16;
  const int sf_words = WT == WType::W16 ? 0 : (K / SV + 3) / 4;
  const int sf_ld = (N + 3) / 4 * 4;

  // Under a programmatic dependent launch the previous kernel may still be running.  Its
  // outputs (X, perhaps the weights) are read only after the wait below; until then this
  // warp asks for the weights of its first run to be brought into L2, the memory's point of
  // coherence, which reads nothing into the kernel.
  if (args.prefetch > 0 && wt < my_tiles) {
    const int row = (tile0 + wt) * 16 + (lane & 15);       // a row per lane, two chunks at a time
    for (int i = lane >> 4; i < args.prefetch && ks + i * KS < nc; i += 2) {
      const int gc = c0 + ks + i * KS;
      if (row < N) prefetch_l2(weights + static_cast<size_t>(row) * row_bytes + static_cast<size_t>(gc) * 128);
      if (WT != WType::W16 && (lane & 15) < C::WPC && gc * C::WPC + (lane & 15) < sf_words)
        prefetch_l2(scale_words + static_cast<size_t>(gc * C::WPC + (lane & 15)) * sf_ld + (tile0 + wt) * 16);
    }
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  // ------------------------------------------------------------ weight stream
  const uint32_t ring = sbase + static_cast<uint32_t>(warp * C::DEPTH * C::STAGE);
  // copies: lane = row l / 8 (and + 4, + 8, + 12), piece l % 8; piece p of row r is stored
  // at p ^ (r % 8) so that ldmatrix reads eight rows without bank conflicts
  const int cr = lane >> 3, cp = lane & 7;
  const uint32_t dst_a = static_cast<uint32_t>(cr * 128 + ((cp ^ cr) << 4)), dst_b = dst_a ^ 64u;
  const size_t rows4 = 4 * row_bytes;
  const int full_chunks = static_cast<int>(row_bytes / 128);   // chunks with no column past K
  const size_t sf_step = static_cast<size_t>(sf_ld) * C::WPC * KS;
  int pf_tile = wt, pf_q = ks;                             // tile (of this CTA's) and chunk (of its share) to load next
  int pf_slot = 0, row0 = 0;
  bool pf_rows = false, pf_new = true;
  const uint8_t* wp = nullptr;
  const uint32_t* sp = nullptr;
  if (pf_q >= nc) pf_tile = my_tiles;                      // more shares than chunks: nothing to do
  auto issue = [&]() {
    if (pf_tile < my_tiles) {
      const int gc = c0 + pf_q;
      if (pf_new) {                                       // a new tile: row pointers
        row0 = (tile0 + pf_tile) * 16;
        pf_rows = row0 + 16 <= N;
        wp = weights + static_cast<size_t>(row0 + cr) * row_bytes + static_cast<size_t>(gc) * 128 + cp * 16;
        if constexpr (WT != WType::W16) sp = scale_words + static_cast<size_t>(gc * C::WPC + (lane >> 4)) * sf_ld + row0 + (lane & 15);
        pf_new = false;
      }
      const uint32_t st = ring + static_cast<uint32_t>(pf_slot * C::STAGE);
      if (pf_rows && gc < full_chunks) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cp16_full(st + (i & 1 ? dst_b : dst_a) + 512 * i, wp + i * rows4);
        if constexpr (WT != WType::W16) {
#pragma unroll
          for (int i = 0; i < C::WPC / 2; ++i) cp4_full(st + 2048 + lane * 4 + 128 * i, sp + static_cast<size_t>(2 * i) * sf_ld);
        }
      } else {                                            // rows past N and columns past K are zero
        const bool in_k = static_cast<size_t>(gc) * 128 + cp * 16 < row_bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool ok = in_k && row0 + cr + 4 * i < N;
          cp16(st + (i & 1 ? dst_b : dst_a) + 512 * i, ok ? wp + i * rows4 : weights, ok);
        }
        if constexpr (WT != WType::W16) {
#pragma unroll
          for (int i = 0; i < C::WPC / 2; ++i) {
            const bool ok = gc * C::WPC + (lane >> 4) + 2 * i < sf_words && row0 + (lane & 15) < N;
            cp4(st + 2048 + lane * 4 + 128 * i, ok ? sp + static_cast<size_t>(2 * i) * sf_ld : scale_words, ok);
          }
        }
      }
      wp += 128 * KS;
      if constexpr (WT != WType::W16) sp += sf_step;
      pf_q += KS;
      if (pf_q >= nc) {
        pf_q = ks;
        pf_tile += args.round_tiles;
        pf_new = true;
      }
      if (++pf_slot == C::DEPTH) pf_slot = 0;
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < C::DEPTH - 1; ++i) issue();

  const uint32_t xs = sbase + static_cast<uint32_t>(args.off_x);
  float* xscale = reinterpret_cast<float*>(smem + args.off_scale);   // [chunk][M]: the power's inverse, negative: kept in bf16
  int slot = 0;                                           // ring slot of the next chunk
  [[maybe_unused]] bool wide = false;                     // the piece of X holds rows kept in bf16

  // this lane's rows of X (columns of the MMA); columns past M repeat the last row and
  // are never stored
  const uint8_t* xl[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xl[n] = smem + args.off_x + static_cast<uint32_t>(min(8 * n + g, M - 1) * args.x_stride + t * 16);

  for (int round = 0; round < my_tiles; round += args.round_tiles) {
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
    int q = round + wt < my_tiles ? ks : nc;              // this warp's next chunk
    // MXFP4: bit 7 of the scale bytes that count in the word this lane looks at; in the last
    // chunk, if it is not a whole one, only of groups before K
    [[maybe_unused]] const uint32_t look = (tile0 + round + wt) * 16 + (lane & 15) < N ? 0x80808080u : 0u;
    [[maybe_unused]] const int left = K / SV - ((args.chunks - 1) * C::WPC + (lane >> 4)) * 4;
    [[maybe_unused]] const uint32_t look_last = left >= 4 ? look : left > 0 ? look >> (8 * (4 - left)) : 0u;
    for (int x0 = 0; x0 < nc; x0 += args.x_chunks) {
      // -------------------------------------------------------- a piece of X
      if (round == 0 || nc > args.x_chunks) {
        if (round > 0 || x0 > 0) __syncthreads();         // the previous piece has been read
        const int xn = min(args.x_chunks, nc - x0);
        const int k0 = (c0 + x0) * C::CK;
        wide = false;
        // one warp takes 256 columns of a row, 8 per lane (zeros past K)
        const int blocks = (xn * C::CK + 255) / 256;
        // loads in flight per lane: 4, or 8 where 16 rows make the staging long (NVFP4
        // 16 x 32768 x 7168 47.2 -> 46.2 us, MXFP4 48.3 -> 45.3 when this was taken; one token
        // gets 10 % slower)
        constexpr int XL = NT == 2 ? 8 : 4;
        auto load_x = [&](int m, int v) -> uint4 {        // zeros past K
          if (k0 + 8 * v >= K) return make_uint4(0u, 0u, 0u, 0u);
          return ptx::ld_global_v4(static_cast<const uint16_t*>(args.X) + static_cast<size_t>(m) * K + k0 + 8 * v);
        };
        for (int it0 = warp; it0 < M * blocks; it0 += XL * W) {
          uint4 w[XL];
#pragma unroll
          for (int q = 0; q < XL; ++q) {
            const int it = it0 + q * W, m = it / blocks, v = (it - m * blocks) * 32 + lane;
            w[q] = it < M * blocks ? load_x(m, v) : make_uint4(0u, 0u, 0u, 0u);
          }
          // 8 columns of row m per lane into shared memory
          auto put = [&](int m, int v, const uint32_t (&u)[4]) {
            st_shared_v4(xs + static_cast<uint32_t>(m * args.x_stride + v * 16), u[0], u[1], u[2], u[3]);
          };
          // x * 2^sh is exact for |x| of bits `a` and 31 powers of two below; 2^sh is not an
          // FP32 value above sh = 127 (it reaches 141), where 2^14 of it is applied first;
          // 2^-sh always is one, a subnormal from sh = 127 on
          auto put_scaled = [&](int m, int blk, int v, uint32_t (&u)[4], uint32_t a) {
            const int sh = 141 - (a ? static_cast<int>(a >> 7) : 127);
            const float f = __uint_as_float(static_cast<uint32_t>(127 + (sh > 127 ? sh - 14 : sh)) << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float lo = __uint_as_float(u[j] << 16), hi = __uint_as_float(u[j] & 0xFFFF0000u);
              if (sh > 127) {
                lo *= 16384.0f;
                hi *= 16384.0f;
              }
              u[j] = pack_2x16(lo * f, hi * f, false);
            }
            if (lane == 0) xscale[blk * M + m] = sh < 127 ? __uint_as_float(static_cast<uint32_t>(127 - sh) << 23) : __uint_as_float(1u << (149 - sh));
            put(m, v, u);
          };
          bool again = false;
#pragma unroll
          for (int q = 0; q < XL; ++q) {
            const int it = it0 + q * W;
            if (it >= M * blocks) break;
            const int m = it / blocks, blk = it - m * blocks, v = blk * 32 + lane;
            uint32_t u[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
            if constexpr (WT == WType::W16) {
              // element 8 s + 2 t + i of each 32 goes to 8 t + 2 s + i: lane t's four pairs side by side
              if (8 * v < xn * C::CK) {
                const uint32_t d = xs + static_cast<uint32_t>(m * args.x_stride + (v >> 2) * 64 + (v & 3) * 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) asm volatile("st.shared.b32 [%0], %1;" ::"r"(d + 16 * j), "r"(u[j]) : "memory");
              }
            } else if constexpr (kScaleX) {
              // largest and, in this lane, least non-zero |x| of the 256 columns as bf16 bits;
              // for the least, as 16-bit integers, |x| - 1 - 2^15, where zero is the largest
              uint32_t a2 = 0u, z2 = 0x7FFF7FFFu;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                a2 = __vmaxu2(a2, u[j] & 0x7FFF7FFFu);
                z2 = __vmins2(z2, (u[j] | 0x80008000u) - 0x00010001u);
              }
              const uint32_t a = __reduce_max_sync(0xffffffffu, max(a2 & 0xFFFFu, a2 >> 16));
              // an |x| of bits below `low` would lose digits in fp16
              const int low = static_cast<int>(a & 0x7F80u) - (31 << 7);
              const uint32_t limit = __byte_perm(static_cast<uint32_t>(max(low, 1) - 1) | 0x8000u, 0u, 0x1010);
              again = again || a >= 0x7F80u || __vmins2(z2, limit) != limit;
              put_scaled(m, blk, v, u, a);
            } else {
              put(m, v, u);
            }
          }
          if constexpr (kScaleX) {
            // infinities, NaN or |x| too small for the scale: these rows once more, with only
            // finite values in the largest
            if (__any_sync(0xffffffffu, again)) {
#pragma unroll 1
              for (int it = it0; it < M * blocks && it < it0 + XL * W; it += W) {
                const int m = it / blocks, blk = it - m * blocks, v = blk * 32 + lane;
                const uint4 x = load_x(m, v);
                uint32_t u[4] = {x.x, x.y, x.z, x.w};
                uint32_t a = 0u, z = 0x7F80u;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const uint32_t e = (u[j / 2] >> (16 * (j & 1))) & 0x7FFFu;
                  if (e < 0x7F80u && e != 0u) {
                    a = max(a, e);
                    z = min(z, e);
                  }
                }
                a = __reduce_max_sync(0xffffffffu, a);
                z = __reduce_min_sync(0xffffffffu, z);
                if (static_cast<int>(z) < static_cast<int>(a & 0x7F80u) - (31 << 7)) {
                  wide = true;
                  if (lane == 0) xscale[blk * M + m] = -1.0f;
                  put(m, v, u);
                } else {
                  put_scaled(m, blk, v, u, a);
                }
              }
            }
          }
        }
        if constexpr (kScaleX) wide = __syncthreads_or(wide ? 1 : 0) != 0;
        else __syncthreads();
      }

      // -------------------------------------------------------- this warp's chunks of it
      const int lr = (lane & 7) + ((lane >> 3) & 1) * 8;  // ldmatrix: row and piece this lane addresses
      const uint32_t la = static_cast<uint32_t>(lr * 128 + (((lane >> 4) ^ (lr & 7)) << 4));
      for (const int end = min(nc, x0 + args.x_chunks); q < end; q += KS) {
        cp_wait<C::DEPTH - 2>();
        __syncwarp();
        issue();
        const uint32_t so = static_cast<uint32_t>((warp * C::DEPTH + slot) * C::STAGE);
        const uint32_t st = sbase + so;
        if (++slot == C::DEPTH) slot = 0;
        const uint32_t xc = static_cast<uint32_t>((q - x0) * (C::CK * 2));
        if constexpr (WT == WType::W16) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {                   // 32 columns
            uint32_t b[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) lds128(xl[n] + xc + 64 * h, b[n]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t a[4];
              ldmatrix_x4(st + (la ^ ((2 * h + i) << 5)), a);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816<kMmaBf16>(acc[n], a[0], a[1], a[2], a[3], b[n][2 * i], b[n][2 * i + 1]);
            }
          }
        } else {
          float xp[NT][2];                                // 2^p of this lane's columns
          if constexpr (kScaleX) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j) xp[n][j] = xscale[(q - x0) * M + min(8 * n + 2 * t + j, M - 1)];
          }
          // the chunk's sums: of scaled X where X is scaled, else straight into the totals
          float part_acc[NT][4];
          float(&sums)[NT][4] = kScaleX ? part_acc : acc;
          if constexpr (kScaleX) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) part_acc[n][e] = 0.0f;
          }
          const uint8_t* scales = smem + so + 2048;
          // MXFP4 on scaled X: sums of scaled X times 2^-63 .. 2^64 are plain FP32 values.  A
          // scale outside of that (E8M0 bits 7 and 6 alike) could overflow or lose digits
          // before the power's inverse is back, so its chunk is multiplied in bf16.  Rows
          // past N and groups past K do not count.
          bool in_bf16 = false;
          if constexpr (kScaleX && WT == WType::MX) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(scales + lane * 4);
            in_bf16 = (~(w ^ (w << 1)) & (c0 + q >= full_chunks ? look_last : look)) != 0u;
          }
          // The chunk in bf16: X as it was, weights decoded as below and converted.  MXFP4
          // scales each group's sum; one that overflows (|x| near 2^128) is taken again
          // from weights times 2^-9.  Rare, so the loop is short rather than fast.
          [[maybe_unused]] auto bf16_chunk = [&]() {
            float back[NT];                               // of row 8 n + g of X
#pragma unroll
            for (int n = 0; n < NT; ++n) back[n] = xscale[(q - x0) * M + min(8 * n + g, M - 1)];
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {                 // 32 codes of each row
              uint32_t a[4], lo[4], hi[4];
              ldmatrix_x4(st + (la ^ static_cast<uint32_t>((i >> 1) << 5)), a);
              e2m1x8(i & 1 ? a[2] : a[0], lo);
              e2m1x8(i & 1 ? a[3] : a[1], hi);
              const uint8_t* w = scales + (i >> 2) * (C::WPC * 32) + g * 4 + (WT == WType::NV ? ((i >> 1) & 1) * 64 : 0);
              const int at = WT == WType::NV ? 2 * (i & 1) + (t >> 1) : i & 3;
              const uint32_t w0 = *reinterpret_cast<const uint32_t*>(w) >> (8 * at), w1 = *reinterpret_cast<const uint32_t*>(w + 32) >> (8 * at);
              [[maybe_unused]] float sf[4], sf1[4];
              if constexpr (WT == WType::NV) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  lo[e] = mul2(lo[e], e4m3_pair(w0, 0));
                  hi[e] = mul2(hi[e], e4m3_pair(w1, 0));
                }
              } else {
                e8m0x4(w0, sf);
                e8m0x4(w1, sf1);
                sf[1] = sf1[0];
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                uint32_t b[4];
                lds128(xl[n] + xc + 64 * i, b);
                if (back[n] > 0.0f) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) b[e] = bf16_pair(b[e], back[n]);
                }
                auto mma = [&](float (&d)[4], float f) {
                  uint32_t wl[4], wh[4];
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    wl[e] = bf16_pair(lo[e], f);
                    wh[e] = bf16_pair(hi[e], f);
                  }
                  __syncwarp();
                  mma16816<true>(d, wl[0], wh[0], wl[1], wh[1], b[0], b[1]);
                  mma16816<true>(d, wl[2], wh[2], wl[3], wh[3], b[2], b[3]);
                };
                if constexpr (WT == WType::NV) {
                  mma(acc[n], 1.0f);
                } else {
                  float p[4] = {}, after = 1.0f;
                  mma(p, 1.0f);
                  const bool lost = !(fabsf(p[0]) + fabsf(p[1]) <= 3.0e38f && fabsf(p[2]) + fabsf(p[3]) <= 3.0e38f);
                  if (__any_sync(0xffffffffu, lost)) {
                    p[0] = p[1] = p[2] = p[3] = 0.0f;
                    mma(p, 1.0f / 512.0f);
                    after = 512.0f;
                  }
#pragma unroll
                  for (int e = 0; e < 4; ++e) acc[n][e] = after == 1.0f ? fmaf(p[e], sf[e >> 1], acc[n][e]) : fmaf(p[e] * sf[e >> 1], after, acc[n][e]);
                }
              }
            }
          };
          auto body = [&]() {
#pragma unroll
            for (int f = 0; f < 2; ++f) {                 // 128 codes of each row
              // scales of rows g and g + 8
              uint32_t sw[2][2];
              [[maybe_unused]] float sf[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint8_t* p = scales + f * (C::WPC * 32) + (g + 8 * h) * 4;
                sw[h][0] = *reinterpret_cast<const uint32_t*>(p);
                if constexpr (WT == WType::NV) {
                  sw[h][1] = *reinterpret_cast<const uint32_t*>(p + 64);
                  sw[h][0] >>= 8 * (t >> 1);
                  sw[h][1] >>= 8 * (t >> 1);
                } else {
                  e8m0x4(sw[h][0], sf[h]);
                }
              }
#pragma unroll
              for (int p2 = 0; p2 < 2; ++p2) {            // 64 codes
                uint32_t a[4];
                ldmatrix_x4(st + (la ^ ((2 * f + p2) << 5)), a);
#pragma unroll
                for (int s2 = 0; s2 < 2; ++s2) {          // 32 codes
                  const int s = 2 * p2 + s2;
                  uint32_t b[NT][4];
#pragma unroll
                  for (int n = 0; n < NT; ++n) lds128(xl[n] + xc + 256 * f + 64 * s, b[n]);
                  uint32_t lo[4], hi[4];
                  e2m1x8(a[2 * s2], lo);
                  e2m1x8(a[2 * s2 + 1], hi);
                  if constexpr (WT == WType::NV) {
                    // lanes t = 0, 1 hold the piece's first group, t = 2, 3 its second
                    const uint32_t s0 = e4m3_pair(sw[0][p2], 2 * s2), s1 = e4m3_pair(sw[1][p2], 2 * s2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      lo[e] = mul2(lo[e], s0);
                      hi[e] = mul2(hi[e], s1);
                    }
                  }
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    if constexpr (WT == WType::NV) {
                      mma16816<false>(sums[n], lo[0], hi[0], lo[1], hi[1], b[n][0], b[n][1]);
                      mma16816<false>(sums[n], lo[2], hi[2], lo[3], hi[3], b[n][2], b[n][3]);
                    } else {
                      float p[4];
                      mma16816_f16_zero(p, lo[0], hi[0], lo[1], hi[1], b[n][0], b[n][1]);
                      mma16816<false>(p, lo[2], hi[2], lo[3], hi[3], b[n][2], b[n][3]);
#pragma unroll
                      for (int e = 0; e < 4; ++e) sums[n][e] = fmaf(p[e], sf[e >> 1][s], sums[n][e]);
                    }
                  }
                }
              }
            }
            if constexpr (kScaleX) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][e] = fmaf(part_acc[n][e], xp[n][e & 1], acc[n][e]);
            }
          };
          if constexpr (kScaleX) {
            if (__builtin_expect(wide, 0)) {
#pragma unroll
              for (int n = 0; n < NT; ++n) in_bf16 = in_bf16 || xp[n][0] < 0.0f || xp[n][1] < 0.0f;
            }
            if (WT == WType::MX || wide) in_bf16 = __any_sync(0xffffffffu, in_bf16);
          }
          if (__builtin_expect(kScaleX && in_bf16, 0)) bf16_chunk();
          else body();
        }
      }
    }

    // ---------------------------------------------------------- the round's outputs
    // four weight rows of one token per thread: cell = token * 4 + row / 4 of a tile
    float* slots = reinterpret_cast<float*>(smem + args.off_slots);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = 8 * n + 2 * t + (e & 1), row = g + 8 * (e >> 1);
        if (col < M) slots[(warp * M + col) * 16 + row] = acc[n][e];
      }
    const int T = min(args.round_tiles, my_tiles - round), cells = 4 * M;
    float4* slots4 = reinterpret_cast<float4*>(slots);
    if (MATS == 1 && KS == 1 && S == 1) {                 // a warp's own tile
      __syncwarp();
      if (wt < T)
        for (int cell = lane; cell < cells; cell += 32) {
          float4 v[MATS];
          v[0] = slots4[warp * cells + cell];
          gemv_store<BF16, MATS>(args, (tile0 + round + wt) * 16 + (cell & 3) * 4, cell >> 2, v);
        }
      __syncwarp();
      continue;
    }
    __syncthreads();
    for (int o = threadIdx.x; o < T * cells; o += static_cast<int>(blockDim.x)) {
      const int tile = o / cells, cell = o - tile * cells;
      float4 v[MATS];
#pragma unroll
      for (int j = 0; j < MATS; ++j) {
        float4* first = slots4 + (tile * MATS + j) * KS * cells + cell;
        v[j] = *first;
        for (int k = 1; k < KS; ++k) add4(v[j], first[k * cells]);
        if (S > 1) *first = v[j];
      }
      if (S == 1) gemv_store<BF16, MATS>(args, (tile0 + round + tile) * 16 + (cell & 3) * 4, cell >> 2, v);
    }
    if (S > 1) {
      cluster_sync_all();                                 // every share's sums are there
      for (int o = rank * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x); o < T * cells; o += S * static_cast<int>(blockDim.x)) {
        const int tile = o / cells, cell = o - tile * cells;
        float4 v[MATS];
#pragma unroll
        for (int j = 0; j < MATS; ++j) {
          const uint32_t at = ptx::smem_u32(slots4 + (tile * MATS + j) * KS * cells + cell);
          v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int r = 0; r < S; ++r) add4(v[j], ld_cluster_f32x4(map_to_rank(at, static_cast<uint32_t>(r))));
        }
        gemv_store<BF16, MATS>(args, (tile0 + round + tile) * 16 + (cell & 3) * 4, cell >> 2, v);
      }
      cluster_sync_all();                                 // and stay until every CTA has read them
    } else {
      __syncthreads();                                    // the slots are free again
    }
  }
  cp_wait<0>();
}

// How a call is laid out: log2 of the cluster, clusters, shared memory, tiles and X per CTA.
struct GemvPlan {
  double ns;
  int log_s, clusters, threads, smem;
  int rounds, pieces;   // of the CTA with most tiles
  GemvKArgs a;
};

template <WType WT, bool BF16, int MATS, int NT, bool DEEP>
struct GemvLaunch {
  using C = GemvCfg<WT, NT, DEEP>;
  static constexpr int kSmem = 232448;
  static constexpr auto kernel = &gemv_kernel<WT, BF16, MATS, NT, DEEP>;

  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  GemvLaunch(int log_s, int clusters, int threads, int smem, cudaStream_t stream, bool pdl) {
    std::memset(&cfg, 0, sizeof(cfg));
    // a cluster of one needs no attribute
    int n = 0;
    if (log_s > 0) {
      attr[n].id = cudaLaunchAttributeClusterDimension;
      attr[n].val.clusterDim.x = 1;
      attr[n].val.clusterDim.y = 1u << log_s;
      attr[n++].val.clusterDim.z = 1;
    }
    if (pdl) {
      attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(clusters), 1u << log_s, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(n);
  }

  // Clusters of 2^log_s CTAs that fit the device at one CTA per SM; null on an error.
  struct Fit {
    int clusters[4];
  };
  static const int* max_clusters() {
    static PerDevice<Fit> fits;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) {
      set_error(2, "device id %d", dev);
      return nullptr;
    }
    const Fit* fit = nullptr;
    fits.get(dev, &fit, [](Fit& f) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      for (int i = 3; e == cudaSuccess && i >= 0; --i) {
        GemvLaunch l(i, device_sm_count() >> i, 32 * C::WARPS, kSmem, nullptr, false);
        int n = device_sm_count();
        if (i > 0) e = cudaOccupancyMaxActiveClusters(&n, kernel, &l.cfg);
        if (e == cudaSuccess && n <= 0) e = cudaErrorInvalidConfiguration;
        f.clusters[i] = n;
      }
      return e == cudaSuccess ? 0 : set_error(4, "matrix-vector set-up: %s", cudaGetErrorString(e));
    });
    return fit != nullptr ? fit->clusters : nullptr;
  }

  // The layout with the least time by a simple model (ns): the chunks of the busiest SM, X
  // to stage, a cluster's joins.  Its constants were searched for the least
  // loss against the best layout, over device times of both variants with clusters of 1, 2,
  // 4 and 8, forced in turn (GB300; 32 shapes, up to 7 numbers of tokens, each type): 1.1 %
  // on average, 19 % at most (0.7 us, 512 rows).  On ten further shapes it is 1.044 times
  // faster than the model before it (geometric mean; 0.90 to 1.61).  They stand for more than their names (a
  // rate also holds part of the latency).  Staging runs on all warps and costs latency per
  // piece, so few warps, many tokens and pieces are what a cluster is for: each of its CTAs
  // stages its own share of X.  Eight tokens of bf16 at 2048 x 7168 in NVFP4 take 10.8 us
  // on one CTA per tile and 6.1 us on four; one token in MXFP4 takes 8.39 us shallow and
  // 8.54 us deep at 7168 x 7168, 34.4 and 25.2 us at 32768 x 7168.  (Times of that search; what
  // bf16 X has needed since, for rows and scales far apart, costs 0 to 5 % of either form.)
  static bool plan(GemvPlan& best, const GemvKArgs& args) {
    const int* fit = max_clusters();
    if (fit == nullptr) return false;
    const int chunks = (args.K + C::CK - 1) / C::CK, all_tiles = (args.N + 15) / 16;
    for (int i = 0; i < 4; ++i) {
      const int s = 1 << i, per = (chunks + s - 1) / s;
      if ((s - 1) * per >= chunks) continue;              // a CTA without work
      // tiles per round and warps per tile: all warps busy, as few rounds as can be, and no
      // more shares of a tile than shorten the longest one
      const int tiles = (all_tiles + fit[i] - 1) / fit[i];
      constexpr int kMost = C::WARPS / MATS;              // tiles of a round
      const int rounds = (tiles + kMost - 1) / kMost;
      const int round_tiles = (tiles + rounds - 1) / rounds;
      int ks = kMost / round_tiles < per ? kMost / round_tiles : per;
      const int longest = (per + ks - 1) / ks;
      ks = (per + longest - 1) / longest;
      const int warps = round_tiles * MATS * ks;
      // shared memory: ring, sums, X (rows an odd number of 64-byte units apart) and scales
      const int slots = warps * C::DEPTH * C::STAGE;
      const int scale = slots + warps * args.M * 64;
      const int fit_x = ((kSmem - scale - 128) / args.M - 64) / (C::CK * 2 + 4);
      if (fit_x < 1) continue;
      const int pieces = (per + fit_x - 1) / fit_x;
      const double stagings = pieces > 1 ? pieces * rounds : 1.0;
      constexpr double kRate = DEEP ? (WT == WType::W16 ? (NT == 1 ? 67.0 : 54.0) : (NT == 1 ? 42.0 : 32.5))
                                    : (WT == WType::W16 ? 40.0 : 23.0);      // bytes per ns and SM
      constexpr double kStage = BF16 && WT != WType::W16 ? 1.2 : 0.43;       // ns per element and warp
      const double x_elements = static_cast<double>(per) / pieces * C::CK * args.M;
      double ns = static_cast<double>(rounds) * longest * warps * C::STAGE / kRate +
                  stagings * (1280.0 + kStage * x_elements / warps) + (DEEP ? 170.0 : 0.0);
      if (s > 1) ns += 1000.0 + 2040.0 * (rounds - 1) + 8.0 * rounds * round_tiles * args.M + (s == 8 ? 200.0 : 0.0);
      if (best.ns >= 0 && ns >= best.ns) continue;
      best.ns = ns;
      best.log_s = i;
      best.rounds = rounds;
      best.pieces = pieces;
      best.threads = 32 * warps;
      best.clusters = all_tiles < fit[i] ? all_tiles : fit[i];
      GemvKArgs& a = best.a;
      a = args;
      a.cta_tiles = all_tiles / best.clusters;
      a.extra = all_tiles % best.clusters;
      a.round_tiles = round_tiles;
      a.ks = ks;
      a.chunks = chunks;
      a.cta_chunks = per;
      a.x_chunks = (per + pieces - 1) / pieces;
      a.x_stride = (a.x_chunks * (C::CK * 2 / 64) | 1) * 64;
      a.off_slots = slots;
      a.off_scale = scale;
      a.off_x = (scale + a.x_chunks * args.M * 4 + 127) / 128 * 128;
      a.prefetch = pdl_enabled() ? 4 : 0;
      best.smem = a.off_x + args.M * a.x_stride;
    }
    return true;
  }

  static int launch(const GemvPlan& p, cudaStream_t stream) {
    set_last_gemv(WT == WType::W16 ? "f16" : WT == WType::MX ? "mxf4" : "nvf4", MATS == 2, 1 << p.log_s, 8 * NT, DEEP, p.rounds, p.pieces);
    GemvLaunch l(p.log_s, p.clusters, p.threads, p.smem, stream, pdl_enabled());
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, p.a);
    return e == cudaSuccess ? 0 : set_error(4, "matrix-vector launch: %s", cudaGetErrorString(e));
  }
};

template <WType WT, bool BF16, int MATS, int NT>
int launch_gemv(const GemvKArgs& args, cudaStream_t stream) {
  GemvPlan p;
  p.ns = -1.0;
  if constexpr (NT == 2) {
    using D = GemvLaunch<WT, BF16, MATS, NT, true>;
    if (!D::plan(p, args)) return 4;
    if (p.ns < 0) return set_error(2, "matrix-vector: no room for X");
    return D::launch(p, stream);
  } else {
    using D = GemvLaunch<WT, BF16, MATS, NT, true>;
    using L = GemvLaunch<WT, BF16, MATS, NT, false>;
    if (!L::plan(p, args)) return 4;
    const double shallow = p.ns;
    if (!D::plan(p, args)) return 4;
    if (p.ns < 0) return set_error(2, "matrix-vector: no room for X");
    return p.ns < shallow || shallow < 0 ? D::launch(p, stream) : L::launch(p, stream);
  }
}

}  // namespace fgf8
