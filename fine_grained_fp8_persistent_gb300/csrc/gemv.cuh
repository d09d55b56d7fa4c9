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
//            acc += partial * 2^e: scales reach 2^+-127, which no 16-bit product holds.
// A 16-byte piece of a weight row holds 32 codes.  ldmatrix hands lane 4 g + t of the warp
// the 8 codes 8 t .. 8 t + 7 of row g; taken as two K = 16 instructions, instruction i
// multiplies codes 8 t + 4 i + {0, 1} and {2, 3} of lane t as its k = 2 t + {0, 1} and
// 2 t + 8 + {0, 1}.  The sum over k does not care for the order, so X needs no shuffle
// either: lane t's share of a row of X is 16 contiguous bytes.
//
// bf16 X is scaled per row by the power of two that puts its largest finite |x| into
// [2^14, 2^15) and rounded to fp16, the type E2M1 decodes to.  Every |x| of at least 2^-31
// of that largest one stays exact; smaller ones move by at most 2^-39 of it, below the FP32
// accumulation's own rounding.
//
// Work split.  A CTA is 8 warps: WR groups of 16 weight rows times WK = 8 / WR interleaved
// shares of the reduction; a cluster of CTAs splits the reduction further when there
// are few rows.  Each warp streams 64-byte pieces of its 16 rows (one "chunk") through a
// ring of its own with cp.async, so the main loop has no barrier.  The partial sums are
// joined in shared memory, then over the cluster, always in the same order.
#pragma once
#include <cstring>

#include "activation.cuh"
#include "gated.h"
#include "gemm_persistent.cuh"

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
  int chunks;        // chunks of the whole reduction
  int per_cta;       // chunks of one CTA (a multiple of WK)
  int x_chunks;      // chunks of X in shared memory at a time (a multiple of WK)
  int x_stride;      // bytes between rows of X in shared memory
};

template <WType WT, bool BF16, int MATS, int NT, int WR>
struct GemvCfg {
  static constexpr int WARPS = 8, THREADS = 32 * WARPS;
  static constexpr int WK = WARPS / WR;
  static constexpr int ROWS = 16 * WR;
  static constexpr int CK = WT == WType::W16 ? 32 : 128;     // elements of K per chunk (64 bytes of a row)
  static constexpr int SF_BYTES = WT == WType::MX ? 64 : WT == WType::NV ? 128 : 0;
  static constexpr int STAGE = MATS * (1024 + SF_BYTES);
  static constexpr int DEPTH = MATS == 2 ? 4 : 6;            // chunks in flight per warp
  static constexpr int RING = WARPS * DEPTH * STAGE;
  static constexpr int COLS = 8 * NT;
  static constexpr int RED = WARPS * MATS * 16 * COLS * 4;   // partial sums, over the ring
  static_assert(RED <= RING, "the partial sums reuse the ring");
  static constexpr int SUM = MATS * ROWS * COLS * 4;         // joined sums of the CTA, read by the cluster
  static constexpr int OFF_SUM = RING;
  static constexpr int OFF_MISC = OFF_SUM + SUM;             // per row of X: largest |x| bits, then 2^p
  static constexpr int OFF_X = OFF_MISC + 128;
};

namespace gemv {

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
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
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

}  // namespace gemv

template <WType WT, bool BF16, int MATS, int NT, int WR>
__global__ void __launch_bounds__(256, MATS == 2 ? 2 : 3) gemv_kernel(const GemvKArgs args) {
  using C = GemvCfg<WT, BF16, MATS, NT, WR>;
  using namespace gemv;
  constexpr bool kScaleX = WT != WType::W16 && BF16;   // bf16 X against fp16 weight values
  constexpr bool kMmaBf16 = WT == WType::W16 && BF16;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane >> 2, t = lane & 3;
  const int wr = warp % WR, wk = warp / WR;
  const int S = static_cast<int>(gridDim.y);            // CTAs of the cluster: shares of the reduction
  const int rank = static_cast<int>(blockIdx.y);
  const int M = args.M, N = args.N, K = args.K;
  const int row0 = static_cast<int>(blockIdx.x) * C::ROWS;
  const int c0 = rank * args.per_cta;                    // first chunk of this CTA
  const int nc = min(args.per_cta, args.chunks - c0);    // may be <= 0 for the last ranks
  const int mine = nc > wk ? (nc - wk + C::WK - 1) / C::WK : 0;   // chunks of this warp: wk, wk + WK, ...
  constexpr int ELEM_BITS = WT == WType::W16 ? 16 : 4;
  const size_t row_bytes = static_cast<size_t>(K) * ELEM_BITS / 8;
  constexpr int SV = WT == WType::MX ? 32 : 16;
  const int sf_words = WT == WType::W16 ? 0 : (K / SV + 3) / 4;
  const int sf_ld = (N + 3) / 4 * 4;

  // X and the weights may come from the previous kernel
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  // ------------------------------------------------------------ weight stream
  const uint32_t ring = sbase + static_cast<uint32_t>(warp * C::DEPTH * C::STAGE);
  // copies: lane = row l / 4 (and + 8), piece l % 4; the pieces of row r are stored
  // rotated by r / 2 so that ldmatrix reads eight rows without bank conflicts
  const int cr = lane >> 2, cp = lane & 3;
  const int wrow = row0 + 16 * wr;
  auto issue = [&](int i) {                               // i-th chunk of this warp
    if (i < mine) {
      const int c = c0 + wk + i * C::WK;
      const uint32_t st = ring + static_cast<uint32_t>((i % C::DEPTH) * C::STAGE);
      const size_t at = static_cast<size_t>(c) * 64 + static_cast<size_t>(cp) * 16;
      const bool in_k = at < row_bytes;
#pragma unroll
      for (int j = 0; j < MATS; ++j) {
        const uint8_t* w = static_cast<const uint8_t*>(args.W[j]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = cr + 8 * h;
          const bool ok = in_k && wrow + r < N;
          cp16(st + j * 1024 + r * 64 + ((cp ^ ((r >> 1) & 3)) << 4), ok ? w + static_cast<size_t>(wrow + r) * row_bytes + at : w, ok);
        }
        if constexpr (WT != WType::W16) {
          // scale words of the chunk's 16 rows: one (MXFP4) or two (NVFP4) per row
          constexpr int WPC = WT == WType::MX ? 1 : 2;
          if (lane < 16 * WPC) {
            const int word = c * WPC + (lane >> 4), r = wrow + (lane & 15);
            const bool ok = word < sf_words && r < N;
            const uint32_t* sf = static_cast<const uint32_t*>(args.SF[j]);
            cp4(st + MATS * 1024 + j * C::SF_BYTES + lane * 4, ok ? sf + static_cast<size_t>(word) * sf_ld + r : sf, ok);
          }
        }
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < C::DEPTH - 1; ++i) issue(i);

  float acc[MATS][NT][4] = {};
  float tot[MATS][NT][4] = {};                            // NVFP4 with scaled X: sums over the pieces of X
  const uint32_t xs = sbase + C::OFF_X;
  uint32_t* amax = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  float* pw = reinterpret_cast<float*>(smem + C::OFF_MISC + 64);

  int i = 0;                                              // next chunk of this warp
  for (int x0 = 0; x0 < nc; x0 += args.x_chunks) {
    // ---------------------------------------------------------- a piece of X
    const int xn = min(args.x_chunks, nc - x0);           // chunks
    const int k0 = (c0 + x0) * C::CK;
    const int vecs = xn * (C::CK / 8);                    // 16-byte vectors per row, zeros past K
    const int blocks = (vecs + 31) / 32;
    if (x0 > 0) __syncthreads();                          // the previous piece has been read
    if constexpr (kScaleX) {
      if (threadIdx.x < 16) amax[threadIdx.x] = 0u;
      __syncthreads();
    }
    for (int it = warp; it < M * blocks; it += C::WARPS) {
      const int m = it / blocks, v = (it - m * blocks) * 32 + lane;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      const bool in = v < vecs;
      if (in && k0 + 8 * v < K)
        w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(args.X) + static_cast<size_t>(m) * K + k0 + 8 * v));
      if constexpr (WT == WType::W16) {
        // element 8 s + 2 t + i of each 32 goes to 8 t + 2 s + i: lane t's four pairs side by side
        if (in) {
          const uint32_t d = xs + static_cast<uint32_t>(m * args.x_stride + (v >> 2) * 64 + (v & 3) * 4);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) asm volatile("st.shared.b32 [%0], %1;" ::"r"(d + 16 * j), "r"(u[j]) : "memory");
        }
      } else if (in) {
        st_shared_v4(xs + static_cast<uint32_t>(m * args.x_stride + v * 16), w.x, w.y, w.z, w.w);
      }
      if constexpr (kScaleX) {
        // largest finite |x| of the row, as FP32 bits
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t a = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = (u[j] << 16) & 0x7FFFFFFFu, hi = u[j] & 0x7FFF0000u;
          a = max(a, lo < 0x7F800000u ? lo : 0u);
          a = max(a, hi < 0x7F800000u ? hi : 0u);
        }
        a = __reduce_max_sync(0xffffffffu, a);
        if (lane == 0) atomicMax(amax + m, a);
      }
    }
    __syncthreads();
    float xp[NT][2];                                      // 2^p of this lane's columns
#pragma unroll
    for (int n = 0; n < NT; ++n) xp[n][0] = xp[n][1] = 1.0f;
    if constexpr (kScaleX) {
      for (int it = warp; it < M * blocks; it += C::WARPS) {
        const int m = it / blocks, v = (it - m * blocks) * 32 + lane;
        // x * 2^sh in two exact steps (sh reaches 141); 2^-sh is an FP32 value
        const int e = amax[m] ? static_cast<int>(amax[m] >> 23) : 127;
        const int sh = 141 - e, s1 = sh / 2, s2 = sh - s1;
        const float f1 = __uint_as_float(static_cast<uint32_t>(127 + s1) << 23), f2 = __uint_as_float(static_cast<uint32_t>(127 + s2) << 23);
        if (v < vecs) {
          const uint32_t at = xs + static_cast<uint32_t>(m * args.x_stride + v * 16);
          uint32_t u[4];
          lds128(at, u);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            u[j] = pack_2x16(__uint_as_float(u[j] << 16) * f1 * f2, __uint_as_float(u[j] & 0xFFFF0000u) * f1 * f2, false);
          st_shared_v4(at, u[0], u[1], u[2], u[3]);
        }
        if (v == 0) {                                     // the row's first vector: record 2^-sh, subnormal from sh = 127
          pw[m] = sh < 127 ? __uint_as_float(static_cast<uint32_t>(127 - sh) << 23) : __uint_as_float(1u << (149 - sh));
        }
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int m = 8 * n + 2 * t + j;
          xp[n][j] = m < M ? pw[m] : 1.0f;
        }
    }

    // ---------------------------------------------------------- main loop
    const int lr = (lane & 7) + ((lane >> 3) & 1) * 8;    // ldmatrix: row and piece this lane addresses
    const int lp = lane >> 4, lx = (lr >> 1) & 3;
    for (; i < mine && wk + i * C::WK < x0 + xn; ++i) {
      cp_wait<C::DEPTH - 2>();
      __syncwarp();
      issue(i + C::DEPTH - 1);
      const uint32_t st = ring + static_cast<uint32_t>((i % C::DEPTH) * C::STAGE);
      const uint32_t xc = xs + static_cast<uint32_t>((wk + i * C::WK - x0) * (C::CK * 2) + t * 16);
      uint32_t a[MATS][2][4];
#pragma unroll
      for (int j = 0; j < MATS; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) ldmatrix_x4(st + j * 1024 + lr * 64 + (((2 * h + lp) ^ lx) << 4), a[j][h]);
      if constexpr (WT == WType::W16) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t b[4] = {0u, 0u, 0u, 0u};
          if (8 * n + g < M) lds128(xc + static_cast<uint32_t>((8 * n + g) * args.x_stride), b);
#pragma unroll
          for (int j = 0; j < MATS; ++j) {
            mma16816<kMmaBf16>(acc[j][n], a[j][0][0], a[j][0][1], a[j][0][2], a[j][0][3], b[0], b[1]);
            mma16816<kMmaBf16>(acc[j][n], a[j][1][0], a[j][1][1], a[j][1][2], a[j][1][3], b[2], b[3]);
          }
        }
      } else {
        // scale words of rows g and g + 8
        uint32_t sw[MATS][2][2];
        float sf[MATS][2][4];
#pragma unroll
        for (int j = 0; j < MATS; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint8_t* p = smem + (st - sbase) + MATS * 1024 + j * C::SF_BYTES + (g + 8 * r) * 4;
            sw[j][r][0] = *reinterpret_cast<const uint32_t*>(p);
            if constexpr (WT == WType::NV) {
              sw[j][r][1] = *reinterpret_cast<const uint32_t*>(p + 64);
              sw[j][r][0] >>= 8 * (t >> 1);
              sw[j][r][1] >>= 8 * (t >> 1);
            } else {
              e8m0x4(sw[j][r][0], sf[j][r]);
            }
          }
#pragma unroll
        for (int s = 0; s < 4; ++s) {                     // 32 codes of each row
          uint32_t b[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            b[n][0] = b[n][1] = b[n][2] = b[n][3] = 0u;
            if (8 * n + g < M) lds128(xc + static_cast<uint32_t>((8 * n + g) * args.x_stride + 64 * s), b[n]);
          }
#pragma unroll
          for (int j = 0; j < MATS; ++j) {
            uint32_t lo[4], hi[4];
            e2m1x8(a[j][s >> 1][2 * (s & 1)], lo);
            e2m1x8(a[j][s >> 1][2 * (s & 1) + 1], hi);
            if constexpr (WT == WType::NV) {
              // lanes t = 0, 1 hold the piece's first group, t = 2, 3 its second
              const uint32_t s0 = e4m3_pair(sw[j][0][s >> 1], 2 * (s & 1)), s1 = e4m3_pair(sw[j][1][s >> 1], 2 * (s & 1));
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                lo[q] = mul2(lo[q], s0);
                hi[q] = mul2(hi[q], s1);
              }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if constexpr (WT == WType::NV) {
                mma16816<false>(acc[j][n], lo[0], hi[0], lo[1], hi[1], b[n][0], b[n][1]);
                mma16816<false>(acc[j][n], lo[2], hi[2], lo[3], hi[3], b[n][2], b[n][3]);
              } else {
                float p[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma16816<false>(p, lo[0], hi[0], lo[1], hi[1], b[n][0], b[n][1]);
                mma16816<false>(p, lo[2], hi[2], lo[3], hi[3], b[n][2], b[n][3]);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  acc[j][n][q] = fmaf(kScaleX ? p[q] * xp[n][q & 1] : p[q], sf[j][q >> 1][s], acc[j][n][q]);
              }
            }
          }
        }
      }
    }
    if constexpr (kScaleX && WT == WType::NV) {
#pragma unroll
      for (int j = 0; j < MATS; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tot[j][n][q] = fmaf(acc[j][n][q], xp[n][q & 1], tot[j][n][q]);
            acc[j][n][q] = 0.0f;
          }
    }
  }

  // -------------------------------------------------------------- join
  cp_wait<0>();
  __syncthreads();                                        // every warp is done with its ring
  float* red = reinterpret_cast<float*>(smem);            // [wk][mat][col][ROWS]
#pragma unroll
  for (int j = 0; j < MATS; ++j)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = 8 * n + 2 * t + (q & 1), row = 16 * wr + g + 8 * (q >> 1);
        red[((wk * MATS + j) * C::COLS + col) * C::ROWS + row] = (kScaleX && WT == WType::NV) ? tot[j][n][q] : acc[j][n][q];
      }
  __syncthreads();
  float* sum = reinterpret_cast<float*>(smem + C::OFF_SUM);   // [mat][col][ROWS]
  for (int o = threadIdx.x; o < MATS * C::COLS * C::ROWS; o += C::THREADS) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < C::WK; ++k) v += red[k * MATS * C::COLS * C::ROWS + o];
    sum[o] = v;
  }
  if (S > 1) cluster_sync_all();
  else __syncthreads();
  // outputs o = m * ROWS + row, split over the cluster
  const int all = M * C::ROWS;
  for (int o = rank * C::THREADS + static_cast<int>(threadIdx.x); o < all; o += S * C::THREADS) {
    const int m = o / C::ROWS, n = row0 + o % C::ROWS;
    float v[MATS];
#pragma unroll
    for (int j = 0; j < MATS; ++j) {
      if (S > 1) {
        const uint32_t at = sbase + C::OFF_SUM + static_cast<uint32_t>(j * C::COLS * C::ROWS + o) * 4u;
        v[j] = 0.0f;
        for (int r = 0; r < S; ++r) v[j] += ld_cluster_f32(map_to_rank(at, static_cast<uint32_t>(r)));
      } else {
        v[j] = sum[j * C::COLS * C::ROWS + o];
      }
    }
    if (n < N) {
      const size_t at = static_cast<size_t>(m) * N + n;
      uint16_t* out = static_cast<uint16_t*>(args.out);
      if constexpr (MATS == 2) {
        if (args.keep[0] != nullptr) {
          static_cast<uint16_t*>(args.keep[0])[at] = act::from_float(v[0], BF16);
          static_cast<uint16_t*>(args.keep[1])[at] = act::from_float(v[1], BF16);
        }
        v[0] = (args.act == act::kSilu ? act::value<act::kSilu>(v[0]) : act::value<act::kGeluTanh>(v[0])) * v[1];
      }
      out[at] = act::from_float(v[0], BF16);
    }
  }
  if (S > 1) cluster_sync_all();                          // the sums stay until every CTA has read them
}

// Launch: rows per CTA, shares of the reduction, and how much of X stays in shared memory.
template <WType WT, bool BF16, int MATS, int NT, int WR>
int launch_gemv(GemvKArgs a, cudaStream_t stream) {
  using C = GemvCfg<WT, BF16, MATS, NT, WR>;
  auto* fn = &gemv_kernel<WT, BF16, MATS, NT, WR>;
  constexpr int kXBytes = 56 * 1024;
  constexpr int kMaxSmem = C::OFF_X + kXBytes + 16 * 64;
  static_assert(kMaxSmem <= 232448, "shared memory budget");
  static bool ready[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return set_error(2, "device id %d", dev);
  if (!ready[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return set_error(4, "matrix-vector set-up: %s", cudaGetErrorString(e));
    ready[dev] = true;
  }
  a.chunks = (a.K + C::CK - 1) / C::CK;
  const long long tiles = (a.N + C::ROWS - 1) / C::ROWS;
  // split the reduction while the CTAs do not fill the SMs twice over and every warp
  // keeps at least four chunks
  int S = 1;
  while (S < 8 && tiles * S < 2LL * device_sm_count() && a.chunks / (2 * S * C::WK) >= 4) S *= 2;
  auto round_up = [](int v, int to) { return (v + to - 1) / to * to; };
  a.per_cta = round_up((a.chunks + S - 1) / S, C::WK);
  // rows of X are an odd number of 64-byte units apart (bank conflicts); at most kXBytes of X
  const int most = kXBytes / (C::CK * 2) / a.M / C::WK * C::WK;
  a.x_chunks = a.per_cta < most ? a.per_cta : most;
  const int units = a.x_chunks * (C::CK * 2 / 64);
  a.x_stride = (units | 1) * 64;
  if (a.x_chunks <= 0) return set_error(2, "matrix-vector: no room for X");
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = static_cast<unsigned>(S);
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(S), 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(C::OFF_X) + static_cast<size_t>(a.M) * a.x_stride;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, a);
  return e == cudaSuccess ? 0 : set_error(4, "matrix-vector launch: %s", cudaGetErrorString(e));
}

}  // namespace fgf8
