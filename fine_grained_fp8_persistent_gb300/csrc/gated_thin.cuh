// gated_thin.cuh -- the gated forward pass for 17 to 256 tokens, bound by reading the
// weights: H = a(X Wg^T) * (X Wu^T).
//
// The weights are the M operand: a tile is 128 accumulator rows, 64 rows of Wg and the same
// 64 rows of Wu, by all tokens (N = tokens rounded up to 16), so each weight byte goes
// through the MMA once, whatever the number of tokens.  (With tokens as M, as for many
// tokens, the tiles that fill 152 SMs are 16 columns of each weight wide, and every one of
// them loads all of X: at 64 tokens 96 rows of 128 bytes per K block of 64, of which 32
// are weights; here 128 of 192 are.)
// A cluster of S CTAs splits the reduction of a tile; each writes its FP32 sums to shared
// memory and the cluster adds them through distributed shared memory, in order, with the
// activation, the product and the store.  Weights from memory, N = 2048, K = 7168 (59 MB,
// 8.7 us at the copy rate): 16.4 us at 64 tokens.  With the weights in L2 the same launch
// takes 12.3, and its 28 K blocks of 192 rows are 5.4 to 7.5 us of copying at the 1.0 to
// 1.4 ns per 128-byte row and CTA that wide tiles take, so neither the copying nor memory
// alone bounds it.  128 of 152 SMs work, in one wave, and launch, pipeline fill and the join are
// not hidden; how the rest divides among them is not established.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer, all warps the epilogue (warps 0-3 drain
// one TMEM lane quarter each).
#pragma once
#include "activation.cuh"
#include "gated.h"
#include "gemm_persistent.cuh"

namespace fgf8 {

struct GatedThinArgs {
  int M, N, K;
  int nb;            // MMA columns: M rounded up to 16
  int stages;        // pipeline stages of a K block (even)
  int cta_kb;        // K blocks of 64 of one CTA's share
  int bf16;
  void* out;
  void* keep[2];     // G and U, or null
  uint32_t* status;
  uint64_t timeout_ns;
};

namespace thin {
constexpr int kRows = 64;                    // weight rows of each matrix in a tile
constexpr int kABytes = 128 * 128;           // a stage's weights
constexpr int kThreads = 128;
constexpr int kMaxStages = 12;
constexpr int kKpu = 2;                      // K blocks per pipeline unit
constexpr int kSmemCap = 230400;             // bytes of stages that fit beside the barriers
}  // namespace thin

template <int ACT>
__global__ void __launch_bounds__(thin::kThreads, 1)
    gated_thin(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_g, const __grid_constant__ CUtensorMap tm_u,
               const GatedThinArgs args) {
  using namespace thin;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t bars[kMaxStages + 2];   // full and empty per unit, accumulator done
  __shared__ uint32_t tmem_slot, abort_word;
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  uint32_t S;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const int units = args.stages / kKpu;
  const int bb = args.nb * 128, stage_bytes = kABytes + bb;
  const int row0 = static_cast<int>(blockIdx.x / S) * kRows;
  const int nkb = (args.K + 63) / 64;
  const int kb0 = static_cast<int>(rank) * args.cta_kb, kb1 = min(nkb, kb0 + args.cta_kb);
  auto full = [&](int u) { return ptx::smem_u32(&bars[u]); };
  auto empty = [&](int u) { return ptx::smem_u32(&bars[kMaxStages / 2 + u]); };
  const uint32_t done = ptx::smem_u32(&bars[kMaxStages]);
  const uint32_t ncols = args.nb <= 32 ? 32u : args.nb <= 64 ? 64u : args.nb <= 128 ? 128u : 256u;

  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tm_x);
    ptx::prefetch_tmap(&tm_g);
    ptx::prefetch_tmap(&tm_u);
    for (int u = 0; u < units; ++u) {
      ptx::mbar_init(full(u), 1);
      ptx::mbar_init(empty(u), 1);
    }
    ptx::mbar_init(done, 1);
    abort_word = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    tc_alloc<1>(ptx::smem_u32(&tmem_slot), ncols);
    ptx::tc_fence_before();
  }
  ptx::griddep_wait();     // nothing above reads global memory
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *const_cast<volatile uint32_t*>(&tmem_slot);
  PairWaitCtl ctl{&abort_word, 0u, args.status, args.timeout_ns, 0};

  if (warp == 0) {
    ctl.role_bit = FGF8_DEVERR_ROLE_PRODUCER;
    int unit = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; kb += kKpu) {
      if (!pwait(empty(unit), phase ^ 1u, ctl)) break;
      if (lane == 0) {
        const int nk = min(kKpu, kb1 - kb);
        ptx::mbar_arrive_expect_tx(full(unit), static_cast<uint32_t>(nk * stage_bytes));
        for (int j = 0; j < nk; ++j) {
          const uint32_t s = sbase + static_cast<uint32_t>((unit * kKpu + j) * stage_bytes);
          ptx::tma_load_2d(s, &tm_g, full(unit), (kb + j) * 64, row0);
          ptx::tma_load_2d(s + kABytes / 2, &tm_u, full(unit), (kb + j) * 64, row0);
          ptx::tma_load_2d(s + kABytes, &tm_x, full(unit), (kb + j) * 64, 0);
        }
      }
      __syncwarp();
      if (++unit == units) { unit = 0; phase ^= 1u; }
    }
  } else if (warp == 1) {
    ctl.role_bit = FGF8_DEVERR_ROLE_MMA;
    const uint32_t fmt = args.bf16 ? 1u : 0u;
    const uint32_t idesc = idesc_dense(fmt, fmt, static_cast<uint32_t>(args.nb), 128);
    int unit = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; kb += kKpu) {
      if (!pwait(full(unit), phase, ctl)) break;
      ptx::tc_fence_after();
      if (lane == 0) {
        const int nk = min(kKpu, kb1 - kb);
        for (int j = 0; j < nk; ++j) {
          const uint32_t s = sbase + static_cast<uint32_t>((unit * kKpu + j) * stage_bytes);
          const uint64_t ad = smem_desc_sw128(s), bd = smem_desc_sw128(s + kABytes);
#pragma unroll
          for (int k = 0; k < 4; ++k) ptx::mma_f16(tmem, ad + 2 * k, bd + 2 * k, idesc, (kb > kb0 || j > 0 || k > 0) ? 1u : 0u);
        }
        ptx::mma_commit(empty(unit));
      }
      __syncwarp();
      if (++unit == units) { unit = 0; phase ^= 1u; }
    }
    if (lane == 0) ptx::mma_commit(done);
    __syncwarp();
  }

  // ------------------------------------------------------------ epilogue
  // every MMA of this CTA has completed; a wait that runs out gets at least a second more,
  // so that nothing is in flight when shared memory and TMEM are given back
  ctl.role_bit = FGF8_DEVERR_ROLE_EPILOGUE;
  uint32_t never = 0u;
  PairWaitCtl last = ctl;
  last.abort_flag = &never;
  last.timeout_ns = ctl.timeout_ns > 1000000000ull ? ctl.timeout_ns : 1000000000ull;
  pwait(done, 0u, last);
  if (__syncthreads_or(abort_word != 0u ? 1 : 0)) {
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 200000ull) __nanosleep(1000);
  }
  __syncwarp();                                             // lanes may have left that wait apart
  ptx::tc_fence_after();
  // accumulator row r (r < 64: G, else U of weight row r - 64) of token m to part[m][r],
  // over the stages
  float* part = reinterpret_cast<float*>(smem);
  for (int c = 0; c < args.nb; c += 16) {
    uint32_t v[16];
    ptx::tmem_ld_32x32b_x16(tmem + ((warp * 32u) << 16) + static_cast<uint32_t>(c), v);
    ptx::tmem_wait_ld();
    ptx::reg_fence(v);
#pragma unroll
    for (int j = 0; j < 16; ++j) part[(c + j) * 128 + warp * 32 + lane] = __uint_as_float(v[j]);
  }
  ptx::tc_fence_before();
  cluster_sync_all();                                       // every share's sums are there
  const uint32_t part_s = sbase;
  const bool bf16 = args.bf16 != 0;
  // four weight rows of one token per thread; the CTAs of the cluster take the tokens in turn
  for (int o = static_cast<int>(threadIdx.x); ; o += kThreads) {
    const int m = (o / 16) * static_cast<int>(S) + static_cast<int>(rank), n = (o % 16) * 4;
    if (m >= args.M) break;
    float g[4] = {}, u[4] = {};
    for (uint32_t r = 0; r < S; ++r) {
      const uint32_t at = map_to_rank(part_s + static_cast<uint32_t>(m * 128 + n) * 4u, r);
      float p[4], q[4];
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(p[0]), "=f"(p[1]), "=f"(p[2]), "=f"(p[3]) : "r"(at) : "memory");
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(q[0]), "=f"(q[1]), "=f"(q[2]), "=f"(q[3]) : "r"(at + 256u) : "memory");
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] += p[e];
        u[e] += q[e];
      }
    }
    if (row0 + n < args.N) {                                // N is a multiple of 8
      const size_t at = static_cast<size_t>(m) * args.N + row0 + n;
      auto put = [&](void* base, const float (&v)[4]) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) = make_uint2(pack_2x16(v[0], v[1], bf16), pack_2x16(v[2], v[3], bf16));
      };
      if (args.keep[0] != nullptr) {
        put(args.keep[0], g);
        put(args.keep[1], u);
      }
      float h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = act::value<ACT>(g[e]) * u[e];
      put(args.out, h);
    }
  }
  cluster_sync_all();                                       // and stay until every CTA has read them
  if (warp == 1) {
    ptx::tc_fence_after();
    tc_dealloc<1>(tmem, ncols);
  }
}

}  // namespace fgf8
