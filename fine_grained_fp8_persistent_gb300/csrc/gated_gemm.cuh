// gated_gemm.cuh -- the matrix products of the gated feed-forward block and of its
// backward pass, 16-bit operands, FP32 accumulation in TMEM (tcgen05.mma kind::f16).
//
//   Forward  H = a(G) * U, G = X Wg^T, U = X Wu^T.   One accumulator tile holds the same
//            columns of G and U side by side (B = rows of Wg, then rows of Wu), so the
//            activation and the product are an epilogue on registers and neither G nor U
//            goes through memory unless the caller keeps them.  With a CTA pair
//            (cta_group::2 takes half of B's rows from each CTA) the even CTA loads Wg,
//            the odd one Wu.
//   Grad     dX = dG Wg + dU Wu: one reduction over 2 N, the first half of its K blocks
//            from (dG, Wg), the second from (dU, Wu).  Wg and Wu are [N][K] with the
//            output index k contiguous, so B is read MN-major.
//            dWg = dG^T X, dWu = dU^T X: A = dG or dU and B = X, both MN-major (the
//            reduction runs over tokens).
//            The tiles of the three outputs go through one launch, so that the last wave
//            of dX is filled with tiles of dWg and dWu.
//
// MN-major operands need no transposed copy: TMA boxes of 64 MN elements (128 bytes) x
// 64 K rows land with the 128-byte swizzle, and the instruction descriptor's transpose
// bits (15: A, 16: B) tell the MMA that the 128-byte rows run along M or N.  The
// descriptor then holds the distance between 64-element MN chunks (one box, 8192 bytes)
// as the leading offset and between groups of eight K rows (1024 bytes) as the stride.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer, warps 2-9 epilogue (two per TMEM lane
// quarter, each with half of the columns), warp 10 relay, which does the MMA issuer's
// mbarrier waiting and hands over by a named barrier (gemm_persistent.cuh says why).  A pipeline unit is two K blocks of 64.  Two
// accumulator buffers, so the epilogue of a tile overlaps the next tile's MMAs.
//
// Measured, bf16, in a burst / back to back under the power cap: 8192 x 7168 x 2048
// forward 247 / 281 us (1946 / 1712 TFLOP/s, bound by the MMA and by power), 4096 x 4096 x
// 4096 forward 139 / 161 us, backward 321 / 359 us with the slope kernel.  Sizes of one
// wave or two take 1.0 to 1.4 ns per 128-byte row that a CTA copies, whatever the tile.
#pragma once
#include "activation.cuh"
#include "gated.h"
#include "gemm_persistent.cuh"

namespace fgf8 {

enum class GatedOp : int { Forward = 0, Grad = 1 };

struct GatedGemmArgs {
  int M, N, K;
  int a_box_rows;    // rows of a K-major A box (a multiple of 8, at most 128)
  int bf16;
  int save;          // Forward: also store G and U
  // Grad: while the first `long_clusters` clusters work on their last tile of dX, the
  // others take the first `early_tiles` tiles of dWg and dWu
  int long_clusters, early_tiles;
  uint32_t* status;
  uint64_t timeout_ns;
};

// Operand and output maps.  Forward: a = X; b = Wg, Wu; d = H, G, U.
// Grad: a = dG, dU (K-major); b = Wg, Wu, X; at = dG, dU (MN-major); d = dX, dWg, dWu.
struct GatedMaps {
  CUtensorMap a[2], b[3], at[2], d[3];
};

template <GatedOp OP, int NCTA_, int BN_, int STAGES_>
struct GatedCfg {
  static constexpr int NCTA = NCTA_, BN = BN_, STAGES = STAGES_;
  static constexpr bool kFwd = OP == GatedOp::Forward;
  static constexpr bool kBT = !kFwd;                      // B MN-major
  static constexpr int BM = 128;
  static constexpr int TILE_M = BM * NCTA;
  static constexpr int OUT_N = kFwd ? BN / 2 : BN;        // output columns of a tile
  static constexpr int B_LOCAL = BN / NCTA;               // B rows (Forward) or columns held by each CTA
  static_assert(NCTA == 1 || NCTA == 2, "one CTA or a pair");
  static_assert(!kBT || B_LOCAL % 64 == 0, "MN-major B: whole 64-element boxes");
  static_assert(!kFwd || (BN / 2) % 16 == 0, "gate and up halves");
  static constexpr int KPU = 2;
  static_assert(STAGES % KPU == 0, "stages per unit");
  static constexpr int UNITS = STAGES / KPU;
  static constexpr int BOX_BYTES = 64 * 128;              // an MN-major box: 64 K rows of 128 bytes
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = B_LOCAL * 128;
  static constexpr int NACC = 2;
  static constexpr int TMEM_USED = NACC * BN;
  static constexpr int TMEM_ALLOC = TMEM_USED <= 64 ? 64 : TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
  static_assert(TMEM_USED <= 512, "TMEM");
  static constexpr int EPI_WARPS = 8;
  static constexpr int EPI_WARP0 = 2;
  static constexpr int RELAY_WARP = EPI_WARP0 + EPI_WARPS;
  static constexpr int THREADS = 32 * (RELAY_WARP + 1);
  static constexpr int HANDOFF_BAR = 1;
  static constexpr int CW = OUT_N / 2 < 32 ? OUT_N / 2 : 32;   // columns of one staged output chunk
  static constexpr int NCH = OUT_N / 2 / CW;              // chunks of one epilogue warp
  static constexpr int CHUNK_BYTES = 32 * CW * 2;         // 32 rows of one epilogue warp
  static constexpr int EPI_BUFS = 2;                      // staging buffers per epilogue warp
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = STAGES * A_BYTES;
  static constexpr int OFF_EPI = OFF_B + STAGES * B_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + EPI_WARPS * EPI_BUFS * CHUNK_BYTES;
  static constexpr int BAR_FULL = 0, BAR_EMPTY = UNITS, BAR_ACC_FULL = 2 * UNITS;
  static constexpr int BAR_ACC_EMPTY = BAR_ACC_FULL + NACC, BAR_DRAIN = BAR_ACC_EMPTY + NACC;
  static constexpr int OFF_MISC = OFF_BAR + (BAR_DRAIN + 1) * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
};

// MN-major operand tile: 64-element chunks one box apart, 8-row K groups 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr, uint32_t box_bytes) {
  uint64_t d = smem_desc_sw128(saddr);
  d &= ~(0x3FFFull << 16);
  return d | (static_cast<uint64_t>(box_bytes >> 4) << 16);
}

template <int CW>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[CW]) {
  if constexpr (CW == 32) ptx::tmem_ld_32x32b_x32(taddr, r);
  else ptx::tmem_ld_32x32b_x16(taddr, r);
}

template <GatedOp OP, int ACT, int NCTA, int BN, int STAGES>
__global__ void __launch_bounds__(GatedCfg<OP, NCTA, BN, STAGES>::THREADS, 1)
    gated_gemm(const __grid_constant__ GatedMaps tm, const GatedGemmArgs args) {
  using C = GatedCfg<OP, NCTA, BN, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = NCTA == 2 ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const uint16_t pair_mask = static_cast<uint16_t>((1u << NCTA) - 1u);
  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * i; };
  auto lbar = [&](int i) -> uint32_t { return NCTA == 2 ? map_to_rank(bar(i), 0u) : bar(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 4);

  const int C0 = static_cast<int>(blockIdx.x) / NCTA;                  // this cluster
  const int CN = static_cast<int>(gridDim.x) / NCTA;
  auto up = [](int v, int by) { return (v + by - 1) / by; };
  // Forward: H.  Grad: tiles of dX [M][K] first, then of dWg and dWu [N][K].
  const int m1 = up(args.M, C::TILE_M), n1 = up(C::kFwd ? args.N : args.K, C::OUT_N);
  const int tiles1 = m1 * n1;
  const int m2 = C::kFwd ? 0 : up(args.N, C::TILE_M), tiles2 = 2 * m2 * n1;
  const int kb1 = up(C::kFwd ? args.K : args.N, 64), kb2 = up(args.M, 64);

  // Tiles run in bands of eight tile columns: a wave of 76 tiles then reads about as many
  // rows of either operand (bands of 4 to 16 are within 2 % of each other).
  constexpr int kBand = 8;
  // Tile: output matrix (0 H or dX; 1, 2 dWg, dWu), first row of this CTA's 128, first
  // column, rows and columns of the matrix, K blocks.
  struct Pos { int mat, row, col, rows, nkb; };
  const int mine1 = C0 < tiles1 ? up(tiles1 - C0, CN) : 0;             // tiles of the first matrix
  const bool late = C0 >= args.long_clusters;
  const int others = CN - args.long_clusters;
  const int early = !C::kFwd && late && C0 - args.long_clusters < args.early_tiles ? up(args.early_tiles - (C0 - args.long_clusters), others) : 0;
  auto tile_at = [&](int i, Pos& p) -> bool {                          // the cluster's i-th tile
    int m, n;
    if (i < mine1) {
      dense_tile(C0 + i * CN, m1, n1, kBand, m, n);
      p.mat = 0;
      p.rows = args.M;
      p.nkb = C::kFwd ? kb1 : 2 * kb1;
    } else {
      if (C::kFwd) return false;
      i -= mine1;
      // then all take turns, the ones with less to do so far first
      const int turn = late ? C0 - args.long_clusters : C0 + others;
      const int t = i < early ? C0 - args.long_clusters + i * others : args.early_tiles + turn + (i - early) * CN;
      if (t >= tiles2) return false;
      dense_tile(t, 2 * m2, n1, kBand, m, n);
      p.mat = m >= m2 ? 2 : 1;
      if (p.mat == 2) m -= m2;
      p.rows = args.N;
      p.nkb = kb2;
    }
    p.row = m * C::TILE_M + static_cast<int>(rank) * C::BM;
    p.col = n * C::OUT_N;
    return true;
  };

  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tm.a[0]);
    ptx::prefetch_tmap(&tm.b[0]);
    ptx::prefetch_tmap(&tm.d[0]);
    ptx::prefetch_tmap(&tm.b[1]);
  }
  if (threadIdx.x == 0) {
    for (int u = 0; u < C::UNITS; ++u) {
      ptx::mbar_init(bar(C::BAR_FULL + u), 1);
      ptx::mbar_init(bar(C::BAR_EMPTY + u), 1);
    }
    for (int b = 0; b < C::NACC; ++b) {
      ptx::mbar_init(bar(C::BAR_ACC_FULL + b), 1);
      ptx::mbar_init(bar(C::BAR_ACC_EMPTY + b), NCTA * C::EPI_WARPS);
    }
    ptx::mbar_init(bar(C::BAR_DRAIN), 1);
    *abort_flag = 0u;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    tc_alloc<NCTA>(ptx::smem_u32(tmem_slot), C::TMEM_ALLOC);
    ptx::tc_fence_before();
  }
  // Forward: nothing above reads global memory, so it overlaps the tail of the previous
  // kernel.  No kernel here lets the next one start early.  (When the backward pass was
  // three programmatic launches, a queue of its calls at 4096 x 7168 x 2048 stopped for
  // good, outside any bounded wait.  Two changes were made together: plain launches, and
  // the convergence after lane 0's store in the epilogue, without which a split warp could
  // reach the next tcgen05.ld.  Either may have been what mattered.)
  if constexpr (C::kFwd) ptx::griddep_wait();
  __syncthreads();
  if constexpr (NCTA == 2) cluster_sync_all();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  PairWaitCtl ctl{abort_flag, NCTA == 2 ? map_to_rank(sbase + C::OFF_MISC + 4, rank ^ 1u) : 0u, args.status, args.timeout_ns, 0};
  bool aborted = false;

  if (warp == 0) {
    // ============================================================ TMA producer
    ctl.role_bit = FGF8_DEVERR_ROLE_PRODUCER;
    int unit = 0;
    uint32_t phase = 0;
    bool ok = true;
    Pos p;
    for (int i = 0; ok && tile_at(i, p); ++i) {
      const bool at = !C::kFwd && p.mat > 0;               // A MN-major
      const uint32_t tx = NCTA * ((at ? static_cast<uint32_t>(C::A_BYTES) : static_cast<uint32_t>(args.a_box_rows) * 128u) + C::B_BYTES);
      for (int kb0 = 0; kb0 < p.nkb; kb0 += C::KPU) {
        if (!pwait(bar(C::BAR_EMPTY + unit), phase ^ 1u, ctl)) { ok = false; break; }
        if (lane == 0) {
          const int nk = min(C::KPU, p.nkb - kb0);
          const uint32_t full = lbar(C::BAR_FULL + unit);
          if (leader) ptx::mbar_arrive_expect_tx(bar(C::BAR_FULL + unit), static_cast<uint32_t>(nk) * tx);
          for (int j = 0; j < nk; ++j) {
            const uint32_t sa = sbase + C::OFF_A + (unit * C::KPU + j) * C::A_BYTES;
            const uint32_t sb = sbase + C::OFF_B + (unit * C::KPU + j) * C::B_BYTES;
            int kb = kb0 + j;
            if constexpr (C::kFwd) {
              const int k = kb * 64;
              tma_load_ab<NCTA>(sa, &tm.a[0], full, k, p.row);
              if constexpr (NCTA == 2) {
                tma_load_ab<NCTA>(sb, &tm.b[rank], full, k, p.col);
              } else {
                tma_load_ab<NCTA>(sb, &tm.b[0], full, k, p.col);
                tma_load_ab<NCTA>(sb + C::B_BYTES / 2, &tm.b[1], full, k, p.col);
              }
            } else {
              const CUtensorMap* mb = &tm.b[2];
              if (at) {
                tma_load_ab<NCTA>(sa, &tm.at[p.mat - 1], full, p.row, kb * 64);
                tma_load_ab<NCTA>(sa + C::BOX_BYTES, &tm.at[p.mat - 1], full, p.row + 64, kb * 64);
              } else {
                const int term = kb >= kb1 ? 1 : 0;        // dG Wg, then dU Wu
                if (term) kb -= kb1;
                tma_load_ab<NCTA>(sa, &tm.a[term], full, kb * 64, p.row);
                mb = &tm.b[term];
              }
              const int col = p.col + static_cast<int>(rank) * C::B_LOCAL;
#pragma unroll
              for (int c = 0; c < C::B_LOCAL / 64; ++c) tma_load_ab<NCTA>(sb + c * C::BOX_BYTES, mb, full, col + 64 * c, kb * 64);
            }
          }
        }
        __syncwarp();
        if (++unit == C::UNITS) { unit = 0; phase ^= 1u; }
      }
    }
    aborted = !ok;
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    ctl.role_bit = FGF8_DEVERR_ROLE_MMA;
    if (leader) {
      int unit = 0, acc = 0;
      const uint32_t fmt = args.bf16 ? 1u : 0u;
      const uint32_t idesc0 = idesc_dense(fmt, fmt, BN, C::TILE_M) | (C::kBT ? 1u << 16 : 0u);
      const uint64_t bdesc0 = C::kBT ? smem_desc_sw128_mn(sbase + C::OFF_B, C::BOX_BYTES) : smem_desc_sw128(sbase + C::OFF_B);
      // bytes between the operands of consecutive K = 16 instructions: 32 along a K-major
      // row, or 16 K rows of 128 bytes
      constexpr uint32_t B_STEP = C::kBT ? 2048u : 32u;
      Pos p;
      for (int i = 0; tile_at(i, p); ++i) {
        const bool at = !C::kFwd && p.mat > 0;
        const uint32_t idesc = idesc0 | (at ? 1u << 15 : 0u);
        const uint64_t adesc0 = at ? smem_desc_sw128_mn(sbase + C::OFF_A, C::BOX_BYTES) : smem_desc_sw128(sbase + C::OFF_A);
        const uint32_t a_step = at ? 2048u >> 4 : 32u >> 4;
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb0 = 0; kb0 < p.nkb; kb0 += C::KPU) {
          named_bar_sync(C::HANDOFF_BAR, 64);
          ptx::tc_fence_after();
          if (lane == 0) {
            const int nk = min(C::KPU, p.nkb - kb0);
#pragma unroll
            for (int j = 0; j < C::KPU; ++j) {
              if (j < nk) {
                const uint32_t stage = static_cast<uint32_t>(unit * C::KPU + j);
                const uint64_t ad = adesc0 + stage * (C::A_BYTES >> 4), bd = bdesc0 + stage * (C::B_BYTES >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  tc_mma<NCTA, Kind::F16>(d, ad + k * a_step, bd + (k * B_STEP >> 4), idesc, 0u, 0u,
                                          (kb0 > 0 || j > 0 || k > 0) ? 1u : 0u);
              }
            }
            tc_commit_mc<NCTA>(bar(C::BAR_EMPTY + unit), pair_mask);
          }
          __syncwarp();
          if (++unit == C::UNITS) unit = 0;
        }
        if (lane == 0) tc_commit_mc<NCTA>(bar(C::BAR_ACC_FULL + acc), pair_mask);
        __syncwarp();
        acc ^= 1;
      }
      // every MMA has completed before TMEM is released (see gemm_persistent.cuh)
      if (lane == 0) tc_commit<NCTA>(bar(C::BAR_DRAIN));
      __syncwarp();
      PairWaitCtl drain = ctl;
      uint32_t zero = 0;
      drain.abort_flag = &zero;
      drain.peer_abort = 0;
      drain.timeout_ns = ctl.timeout_ns > 1000000000ull ? ctl.timeout_ns : 1000000000ull;
      if (!pwait(bar(C::BAR_DRAIN), 0u, drain)) {
        aborted = true;
        if (lane == 0) *abort_flag = 1u;
      }
    }
  } else if (warp == C::RELAY_WARP) {
    // ============================================================ relay
    ctl.role_bit = FGF8_DEVERR_ROLE_MMA;
    if (leader) {
      int unit = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      Pos p;
      for (int i = 0; tile_at(i, p); ++i) {
        if (ok) ok = pwait(bar(C::BAR_ACC_EMPTY + acc), acc_phase ^ 1u, ctl);
        for (int kb0 = 0; kb0 < p.nkb; kb0 += C::KPU) {
          if (ok) ok = pwait(bar(C::BAR_FULL + unit), phase, ctl);
          named_bar_sync(C::HANDOFF_BAR, 64);
          if (++unit == C::UNITS) { unit = 0; phase ^= 1u; }
        }
        if (++acc == C::NACC) { acc = 0; acc_phase ^= 1u; }
      }
      aborted = !ok;
    }
  } else {
    // ============================================================ epilogue
    // Each warp takes the 32 rows of its TMEM lane quarter and half of the columns, CW at a time: rounds
    // them into one of its staging buffers and lane 0 stores them by TMA (the tensor map
    // clips rows and columns past the matrix).  A buffer is rewritten only after the
    // store EPI_BUFS stores earlier has read it.
    ctl.role_bit = FGF8_DEVERR_ROLE_EPILOGUE;
    const uint32_t q = warp & 3u;
    const int half = static_cast<int>(warp - C::EPI_WARP0) >> 2;
    const bool bf16 = args.bf16 != 0;
    const uint32_t stage0 = sbase + C::OFF_EPI + (warp - C::EPI_WARP0) * static_cast<uint32_t>(C::EPI_BUFS * C::CHUNK_BYTES);
    int acc = 0;
    uint32_t acc_phase = 0, stored = 0;
    bool ok = true;
    constexpr int CW = C::CW;
    auto put = [&](const CUtensorMap* map, const float (&v)[CW], int x, int y, bool inside) {
      const uint32_t buf = stage0 + (stored % C::EPI_BUFS) * C::CHUNK_BYTES;
      if (lane == 0) ptx::bulk_wait_group_read<C::EPI_BUFS - 1>();
      __syncwarp();
#pragma unroll
      for (int j = 0; j < CW / 8; ++j)
        st_shared_v4(buf + lane * (CW * 2u) + 16u * j, pack_2x16(v[8 * j], v[8 * j + 1], bf16), pack_2x16(v[8 * j + 2], v[8 * j + 3], bf16),
                     pack_2x16(v[8 * j + 4], v[8 * j + 5], bf16), pack_2x16(v[8 * j + 6], v[8 * j + 7], bf16));
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (inside) ptx::tma_store_2d(map, buf, x, y);
        ptx::bulk_commit_group();
      }
      __syncwarp();                                       // the next TMEM load is a whole-warp instruction
      ++stored;
    };
    Pos p;
    for (int i = 0; tile_at(i, p); ++i) {
      if (!pwait(bar(C::BAR_ACC_FULL + acc), acc_phase, ctl)) { ok = false; break; }
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((q * 32u) << 16) + static_cast<uint32_t>(acc * BN);
      const int y = p.row + static_cast<int>(q) * 32;
      auto release = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lbar(C::BAR_ACC_EMPTY + acc));
      };
#pragma unroll 1
      for (int c = 0; c < C::NCH; ++c) {
        const int x = p.col + half * (C::OUT_N / 2) + CW * c;
        const uint32_t tcol = taddr + static_cast<uint32_t>(half * (C::OUT_N / 2) + CW * c);
        const bool inside = y < p.rows && x < (C::kFwd ? args.N : args.K);
        uint32_t v[CW];
        tmem_ld_cols<CW>(tcol, v);
        float f[CW];
        if constexpr (C::kFwd) {
          uint32_t w[CW];
          tmem_ld_cols<CW>(tcol + C::OUT_N, w);
          ptx::tmem_wait_ld();
          ptx::reg_fence(v);
          ptx::reg_fence(w);
          if (c == C::NCH - 1) release();
#pragma unroll
          for (int e = 0; e < CW; ++e) f[e] = act::value<ACT>(__uint_as_float(v[e])) * __uint_as_float(w[e]);
          put(&tm.d[0], f, x, y, inside);
          if (args.save) {
#pragma unroll
            for (int e = 0; e < CW; ++e) f[e] = __uint_as_float(v[e]);
            put(&tm.d[1], f, x, y, inside);
#pragma unroll
            for (int e = 0; e < CW; ++e) f[e] = __uint_as_float(w[e]);
            put(&tm.d[2], f, x, y, inside);
          }
        } else {
          ptx::tmem_wait_ld();
          ptx::reg_fence(v);
          if (c == C::NCH - 1) release();
#pragma unroll
          for (int e = 0; e < CW; ++e) f[e] = __uint_as_float(v[e]);
          put(&tm.d[p.mat], f, x, y, inside);
        }
      }
      if (++acc == C::NACC) { acc = 0; acc_phase ^= 1u; }
    }
    // every store has completed before the CTA may exit
    if (lane == 0) ptx::bulk_wait_group<0>();
    __syncwarp();
    aborted = !ok;
  }

  // ---------------------------------------------------------------- teardown
  // after an abort, loads or MMAs may still be in flight: give them time to land
  if (__syncthreads_or(aborted ? 1 : 0) || *abort_flag) {
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 200000ull) __nanosleep(1000);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (NCTA == 2) cluster_sync_all();
  if (warp == 1) {
    ptx::tc_fence_after();
    tc_dealloc<NCTA>(tmem_base, C::TMEM_ALLOC);
  }
}

}  // namespace fgf8
