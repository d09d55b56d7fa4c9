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
__device__ __forceinline__ int load_rows(const RowsArgs& a, uint32_t t, int j0, int lane) {
  return j0 + lane < a.k ? load_row(a, static_cast<long long>(t) * a.k + j0 + lane) : -1;
}

// Items (token t, part p of its row) in flat order, `step` at a time, without a division for
// each.  T is below 2^31 and a step some thousands, so t does not wrap.
struct Walk {
  uint32_t t, p;
  const uint32_t step_t, step_p, parts;
  __device__ __forceinline__ Walk(uint32_t first, uint32_t step, uint32_t n)
      : t(first / n), p(first % n), step_t(step / n), step_p(step % n), parts(n) {}
  __device__ __forceinline__ void next() {
    t += step_t;
    p += step_p;
    if (p >= parts) {
      p -= parts;
      ++t;
    }
  }
};

// ----------------------------------------------------------------- dispatch, 16 bits
// No byte passes through a register: a warp loads a piece of a token (a whole row, or an equal
// part of at most kMaxPiece bytes) into shared memory with one bulk copy, and lane j stores it
// to the row of entry j with another.  Each warp has a ring of stages of its own: a stage is
// loaded again when the stores of the item after it have been issued and its own have read
// it.  Behind the tokens, each lane looks at one row of the layout and fills it from a piece
// of zeros if no entry owns it.  8192 tokens of 7168 bf16, k = 8 of 32: 190 us, 5.9 TB/s, nine
// tenths of it writes; the same rows stored from registers take as long.
constexpr int kMaxPiece = 8192, kStages = 3, kBulkWarps = 8, kBulkThreads = 32 * kBulkWarps;

struct BulkArgs {
  RowsArgs a;
  long long row_bytes;
  int pieces, piece;              // parts of a row, and bytes of all of them but the last
  int zero_rows;                  // rows that a warp looks at together behind the tokens, up to 32
  uint64_t timeout_ns;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// Rows without an entry, from a piece of zeros in shared memory: a lane looks at one row, a
// warp at `rows` of them (up to 32; few rows are spread over all warps).
constexpr int kZeroBytes = 4096;

__device__ __forceinline__ void clear_piece(uint4* zeros) {  // before a __syncthreads
  for (int i = static_cast<int>(threadIdx.x); i < kZeroBytes / 16; i += static_cast<int>(blockDim.x)) zeros[i] = make_uint4(0u, 0u, 0u, 0u);
  ptx::fence_proxy_async_smem();
}
__device__ __forceinline__ void fill_empty_rows(const RowsArgs& a, uint8_t* out, const uint4* zeros, uint32_t rows, uint32_t first, uint32_t step) {
  const uint32_t lane = threadIdx.x & 31, M = static_cast<uint32_t>(a.M), src = ptx::smem_u32(zeros);
  const size_t row_bytes = 2 * static_cast<size_t>(a.H);
  for (uint32_t r0 = first * rows; r0 < M; r0 += step * rows)
    if (lane < rows && r0 + lane < M && ptx::ld_global(a.src + r0 + lane) < 0) {
      uint8_t* row = out + (r0 + lane) * row_bytes;
      for (size_t b = 0; b < row_bytes; b += kZeroBytes)
        bulk_store(row + b, src, static_cast<uint32_t>(row_bytes - b < kZeroBytes ? row_bytes - b : kZeroBytes));
    }
  ptx::bulk_commit_group();
}
// The number for a grid with that many warps.
inline int zero_rows(const RowsArgs& a, long long warps) {
  int rows = 32;
  while (rows > 1 && a.M / rows < 2 * warps) rows /= 2;
  return rows;
}

__global__ void __launch_bounds__(kBulkThreads) dispatch_f16_kernel(BulkArgs args, const uint8_t* __restrict__ X,
                                                                uint8_t* __restrict__ Xs) {
  extern __shared__ __align__(128) uint8_t smem[];          // [warp][stage], args.piece bytes each
  __shared__ __align__(16) uint4 zeros[kZeroBytes / 16];
  __shared__ uint64_t bars[kBulkWarps * kStages];
  __shared__ volatile uint32_t abort_word;
  const RowsArgs& a = args.a;
  const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
  const uint32_t ring = ptx::smem_u32(smem) + static_cast<uint32_t>(args.piece * warp * kStages);
  auto full = [&](int s) { return ptx::smem_u32(&bars[warp * kStages + s]); };
  if (threadIdx.x == 0) abort_word = 0u;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) ptx::mbar_init(full(s), 1);
    ptx::fence_mbar_init();
  }
  clear_piece(zeros);
  __syncthreads();
  ptx::griddep_wait();                                      // everything may come from the previous kernel
  ptx::griddep_launch_dependents();

  // neighbouring items on different SMs, so that few of them are spread over all
  const uint32_t T = static_cast<uint32_t>(a.T), first = warp * gridDim.x + blockIdx.x, step = gridDim.x * kBulkWarps;
  Walk now(first, step, static_cast<uint32_t>(args.pieces)), ahead = now;          // `ahead`: the next item to load
  auto bytes_of = [&](uint32_t p) {
    return static_cast<uint32_t>(min(static_cast<long long>(args.piece), args.row_bytes - static_cast<long long>(p) * args.piece));
  };
  auto load = [&](int s) {
    if (ahead.t < T) {
      ptx::mbar_arrive_expect_tx(full(s), bytes_of(ahead.p));
      bulk_load(ring + static_cast<uint32_t>(s * args.piece),
                X + static_cast<size_t>(ahead.t) * args.row_bytes + static_cast<size_t>(ahead.p) * args.piece, bytes_of(ahead.p), full(s));
    }
    ahead.next();
  };
  PairWaitCtl ctl{&abort_word, 0u, a.status, args.timeout_ns, FGF8_DEVERR_ROLE_PRODUCER};
  if (lane == 0)
    for (int s = 0; s < kStages - 1; ++s) load(s);
  int rows = now.t < T ? load_rows(a, now.t, 0, lane) : -1;
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  while (now.t < T) {
    const uint32_t t = now.t, p = now.p;
    const int mine = rows;
    now.next();
    if (now.t < T) rows = load_rows(a, now.t, 0, lane);
    ok = pwait(full(stage), phase, ctl);
    if (!ok) break;
    const uint32_t src = ring + static_cast<uint32_t>(stage * args.piece);
    for (int j0 = 0; j0 < a.k; j0 += 32) {
      const int row = j0 == 0 ? mine : load_rows(a, t, j0, lane);
      if (row >= 0) bulk_store(Xs + static_cast<size_t>(row) * args.row_bytes + static_cast<size_t>(p) * args.piece, src, bytes_of(p));
    }
    ptx::bulk_commit_group();
    ptx::bulk_wait_group_read<1>();                         // the item before has left its stage
    __syncwarp();
    if (lane == 0) load(stage == 0 ? kStages - 1 : stage - 1);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (ok && a.src != nullptr) fill_empty_rows(a, Xs, zeros, static_cast<uint32_t>(args.zero_rows), first, step);
  ptx::bulk_wait_group<0>();
  // after a wait that ran out, loads may still be under way into this shared memory
  if (__syncthreads_or(abort_word != 0u ? 1 : 0)) {
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 200000ull) __nanosleep(1000);
  }
}

// ----------------------------------------------------------------- dispatch, E4M3
// A warp's item is 512 elements of a token, quantized as quantize_1x128 does it (lanes
// 8 i .. 8 i + 7 hold K block i, 16 elements each), codes and scales written to its k rows;
// the next item's elements and rows are loaded before this one is stored.  8192 tokens of
// 7168, k = 8 of 32: 105 us with UE8M0 scales (5.6 TB/s), 113 with FP32 ones, four times as
// many stores of 4 bytes.
template <bool UE8M0, bool MASKED>
__global__ void __launch_bounds__(kThreads, 4) dispatch_fp8_kernel(RowsArgs a, const uint4* __restrict__ X,
                                                                uint4* __restrict__ Xq, uint32_t* __restrict__ SF) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int nkb = a.H / 128, kq = (nkb + 3) / 4;
  const int per = MASKED ? a.slots : a.M;                  // rows of one scale table
  const size_t ld = (static_cast<size_t>(per) + 3) / 4 * 4;
  const size_t table = ld * (UE8M0 ? kq : nkb);
  const uint32_t T = static_cast<uint32_t>(a.T);
  Walk w(blockIdx.x * kWarps + (threadIdx.x >> 5), gridDim.x * kWarps, static_cast<uint32_t>(kq));
  uint4 next0, next1;                                      // the next item's elements and rows
  int next_rows = -1;
  auto load = [&]() {
    if (4 * static_cast<int>(w.p) + (lane >> 3) < nkb) {
      const uint4* src = X + (static_cast<size_t>(w.t) * a.H + static_cast<size_t>(w.p) * 512 + 16 * lane) / 8;
      next0 = ptx::ld_global_v4(src);
      next1 = ptx::ld_global_v4(src + 1);
    }
    next_rows = load_rows(a, w.t, 0, lane);
  };
  if (w.t < T) load();
  while (w.t < T) {
    const uint32_t t = w.t;
    const int qw = static_cast<int>(w.p), kb = 4 * qw + (lane >> 3);
    const bool active = kb < nkb;
    const int first_rows = next_rows;
    float f0[8], f1[8];
    float amax = 0.0f;
    if (active) {
      quant::unpack8(next0, f0);
      quant::unpack8(next1, f1);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(f0[i]), fabsf(f1[i])));
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, off));
    w.next();
    if (w.t < T) load();
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
      const int rows = j0 == 0 ? first_rows : load_rows(a, t, j0, lane);
      // in the masked layout each lane finds its row's place in the scale tables, so that the
      // division is not made for every row by every lane
      unsigned long long place = 0;
      if (MASKED && rows >= 0) place = rows / per * static_cast<unsigned long long>(table) + static_cast<unsigned>(rows % per);
      __syncwarp();
      for (int j = 0; j < 32 && j0 + j < a.k; ++j) {
        const int row = __shfl_sync(kFull, rows, j);
        const unsigned long long to = MASKED ? __shfl_sync(kFull, place, j) : static_cast<unsigned long long>(row);
        if (row < 0) continue;
        if (active) st_global_v4(Xq + (static_cast<size_t>(row) * a.H + static_cast<size_t>(qw) * 512 + 16 * lane) / 16, code);
        if (scales) SF[to + at] = word;
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

// A warp's item is U * 512 bytes of a token.  A batch of B rows is in flight together, up to
// eight 16-byte loads per lane, and added in FP32 in the order of j; the next item's rows and
// weights are loaded ahead of them.  B and U go by k, and the CTAs per SM (24 or 32 warps) by
// what the registers of B U loads and 8 U sums leave: at 8192 tokens of 7168, k = 8, 32 warps
// take 167 us and 24 take 179; at 4096 columns, k = 2, U = 2 takes 34.7 us, U = 4 36.2, U = 1 41.2.
template <bool BF16, bool WEIGHTED, int B, int U>
__global__ void __launch_bounds__(kThreads, B == 4 ? 3 : 4) combine_f16_kernel(RowsArgs a, const uint4* __restrict__ Ys,
                                                               const float* __restrict__ W, uint4* __restrict__ Y) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int vecs = a.H / 8, parts = (vecs + 32 * U - 1) / (32 * U);
  auto load_weights = [&](uint32_t t, int j0) {
    return WEIGHTED && j0 + lane < a.k ? ptx::ld_global(W + static_cast<long long>(t) * a.k + j0 + lane) : 1.0f;
  };
  const uint32_t T = static_cast<uint32_t>(a.T);
  Walk next(blockIdx.x * kWarps + (threadIdx.x >> 5), gridDim.x * kWarps, static_cast<uint32_t>(parts));
  if (next.t >= T) return;
  int rows = load_rows(a, next.t, 0, lane);
  float weights = load_weights(next.t, 0);
  while (next.t < T) {
    const uint32_t t = next.t;
    const int v0 = static_cast<int>(next.p) * 32 * U + lane;
    int mine = rows;
    float by = weights;
    next.next();
    if (next.t < T) {
      rows = load_rows(a, next.t, 0, lane);
      weights = load_weights(next.t, 0);
    }
    float sum[U][8] = {};
    for (int j0 = 0; j0 < a.k; j0 += 32) {
      if (j0 > 0) {
        mine = load_rows(a, t, j0, lane);
        by = load_weights(t, j0);
      }
      const int n = min(32, a.k - j0);
      for (int j = 0; j < n; j += B) {
        uint4 y[B][U];
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int row = __shfl_sync(kFull, mine, (j + b) & 31);   // -1 past the last entry
          if (row >= 0) {
            const uint4* p = Ys + static_cast<size_t>(row) * vecs + v0;
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (v0 + 32 * u < vecs) y[b][u] = ptx::ld_global_v4(p + 32 * u);
          }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const int row = __shfl_sync(kFull, mine, (j + b) & 31);
          const float w = WEIGHTED ? __shfl_sync(kFull, by, (j + b) & 31) : 1.0f;
          if (row >= 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
              float f[8];
              unpack16<BF16>(y[b][u], f);
#pragma unroll
              for (int i = 0; i < 8; ++i) sum[u][i] = WEIGHTED ? fmaf(w, f[i], sum[u][i]) : sum[u][i] + f[i];
            }
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v0 + 32 * u < vecs) st_global_v4(Y + static_cast<size_t>(t) * vecs + v0 + 32 * u, pack16(sum[u], BF16));
  }
}

// ----------------------------------------------------------------- gradients of combine
// A CTA takes a token, with as many warps as leave each lane about four 16-byte pieces of the
// row: its threads walk the row once for every B entries, U pieces at a time, so dY is read
// from HBM once; the dot products are summed over lanes and warps in a fixed order.  Behind
// the tokens, rows without an entry are zeroed.  8192 tokens of 7168, k = 8 of 32: 318 us,
// 6.5 TB/s.
template <bool BF16, int B, int U>
__global__ void __launch_bounds__(kThreads) combine_f16_backward_kernel(RowsArgs a, const uint4* __restrict__ dY,
                                                                        const uint4* __restrict__ Ys, const float* __restrict__ W,
                                                                        uint4* __restrict__ dYs, float* __restrict__ dW, int zero_rows) {
  __shared__ float part[2][kWarps][B];
  __shared__ __align__(16) uint4 zeros[kZeroBytes / 16];
  if (a.src != nullptr) {
    clear_piece(zeros);
    __syncthreads();
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int threads = static_cast<int>(blockDim.x), warps = threads >> 5;
  const int vecs = a.H / 8;
  int turn = 0;
  for (uint32_t t = blockIdx.x; t < static_cast<uint32_t>(a.T); t += gridDim.x) {
    for (int j0 = 0; j0 < a.k; j0 += B) {
      int row[B];
      float w[B], dot[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const long long entry = static_cast<long long>(t) * a.k + j0 + b;
        row[b] = j0 + b < a.k ? load_row(a, entry) : -1;
        w[b] = row[b] >= 0 ? ptx::ld_global(W + entry) : 0.0f;
        dot[b] = 0.0f;
      }
      for (int v0 = tid; v0 < vecs; v0 += U * threads) {
        uint4 dv[U], y[U][B];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int v = v0 + u * threads;
          if (v < vecs) {
            dv[u] = ptx::ld_global_v4(dY + static_cast<size_t>(t) * vecs + v);
#pragma unroll
            for (int b = 0; b < B; ++b)
              if (row[b] >= 0) y[u][b] = ptx::ld_global_v4(Ys + static_cast<size_t>(row[b]) * vecs + v);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int v = v0 + u * threads;
          if (v < vecs) {
            float d[8];
            unpack16<BF16>(dv[u], d);
#pragma unroll
            for (int b = 0; b < B; ++b)
              if (row[b] >= 0) {
                float f[8], g[8];
                unpack16<BF16>(y[u][b], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  dot[b] = fmaf(d[i], f[i], dot[b]);
                  g[i] = w[b] * d[i];
                }
                st_global_v4(dYs + static_cast<size_t>(row[b]) * vecs + v, pack16(g, BF16));
              }
          }
        }
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot[b] += __shfl_xor_sync(kFull, dot[b], off);
        if (lane == 0) part[turn][warp][b] = dot[b];
      }
      __syncthreads();
      if (tid < B && j0 + tid < a.k) {
        float s = 0.0f;
        for (int i = 0; i < warps; ++i) s += part[turn][i][tid];
        dW[static_cast<long long>(t) * a.k + j0 + tid] = s;
      }
      turn ^= 1;                                            // the next sums need no second barrier
    }
  }
  if (a.src == nullptr) return;
  fill_empty_rows(a, reinterpret_cast<uint8_t*>(dYs), zeros, static_cast<uint32_t>(zero_rows), warp * gridDim.x + blockIdx.x, warps * gridDim.x);
  ptx::bulk_wait_group<0>();
}

// ----------------------------------------------------------------- launches
// Resident CTAs of a kernel on the current device, for a block size.
template <typename... KArgs>
int resident(void (*kernel)(KArgs...), PerDevice<int>& cache, int threads, int* ctas) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  const int* n = nullptr;
  const int r = cache.get(dev, &n, [&](int& v) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kernel, threads, 0);
    if (e != cudaSuccess || v <= 0) return set_error(4, "dispatch occupancy: %s", cudaGetErrorString(e));
    v *= device_sm_count();
    return 0;
  });
  if (r == 0) *ctas = *n;
  return r;
}

template <typename... KArgs, typename... Args>
int launch(void (*kernel)(KArgs...), long long ctas, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
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
  if (const int r = resident(kernel, cache, kThreads, &most)) return r;
  const long long ctas = (items + kWarps - 1) / kWarps;
  return launch(kernel, ctas < most ? ctas : most, kThreads, 0, stream, args...);
}

template <bool BF16, bool WEIGHTED, int B, int U>
int launch_combine(const RowsArgs& a, const void* Ys, const float* W, void* Y, cudaStream_t stream) {
  static PerDevice<int> cache;
  const long long items = static_cast<long long>(a.T) * ((a.H / 8 + 32 * U - 1) / (32 * U));
  return launch_items(combine_f16_kernel<BF16, WEIGHTED, B, U>, cache, items, stream, a, static_cast<const uint4*>(Ys), W,
                      static_cast<uint4*>(Y));
}

template <bool BF16, bool WEIGHTED>
int combine_by_k(const RowsArgs& a, const void* Ys, const float* W, void* Y, cudaStream_t stream) {
  if (a.k <= 2) return launch_combine<BF16, WEIGHTED, 2, 2>(a, Ys, W, Y, stream);
  if (a.k <= 4) return launch_combine<BF16, WEIGHTED, 4, 2>(a, Ys, W, Y, stream);
  return launch_combine<BF16, WEIGHTED, 8, 1>(a, Ys, W, Y, stream);
}

template <bool BF16, int B, int U>
int launch_backward(const RowsArgs& a, const void* dY, const void* Ys, const float* W, void* dYs, float* dW, cudaStream_t stream) {
  static PerDevice<int> cache[kWarps];
  // about four pieces per lane, in equal steps
  const int vecs = a.H / 8, want = (vecs + 127) / 128, most = want < kWarps ? want : kWarps;
  const int steps = (vecs + 32 * most - 1) / (32 * most), warps = (vecs + 32 * steps - 1) / (32 * steps);
  auto* fn = combine_f16_backward_kernel<BF16, B, U>;
  int ctas = 0;
  if (const int r = resident(fn, cache[warps - 1], 32 * warps, &ctas)) return r;
  const int zero = zero_rows(a, static_cast<long long>(ctas) * warps);
  const long long blocks = a.src != nullptr ? (a.M + static_cast<long long>(zero) * warps - 1) / (zero * warps) : 0;
  const long long work = blocks > a.T ? blocks : a.T;
  return launch(fn, work < ctas ? work : ctas, 32 * warps, 0, stream, a, static_cast<const uint4*>(dY), static_cast<const uint4*>(Ys), W,
                static_cast<uint4*>(dYs), dW, zero);
}

template <bool BF16>
int backward_by_k(const RowsArgs& a, const void* dY, const void* Ys, const float* W, void* dYs, float* dW, cudaStream_t stream) {
  if (a.k == 1) return launch_backward<BF16, 1, 4>(a, dY, Ys, W, dYs, dW, stream);
  if (a.k == 2) return launch_backward<BF16, 2, 2>(a, dY, Ys, W, dYs, dW, stream);
  if (a.k <= 4) return launch_backward<BF16, 4, 2>(a, dY, Ys, W, dYs, dW, stream);
  return launch_backward<BF16, 8, 1>(a, dY, Ys, W, dYs, dW, stream);
}

}  // namespace

int launch_dispatch_f16(const RowsArgs& a, const void* X, void* Xs, cudaStream_t stream) {
  constexpr int kRoom = 226000;                             // of 232448 bytes of shared memory, less what is static
  static PerDevice<int> ready;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  const int* set = nullptr;
  const int r = ready.get(dev, &set, [&](int& v) {
    v = kRoom;
    const cudaError_t e = cudaFuncSetAttribute(dispatch_f16_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
    return e == cudaSuccess ? 0 : set_error(4, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  });
  if (r) return r;
  BulkArgs b;
  b.a = a;
  b.timeout_ns = wait_timeout_ns();
  const long long row_bytes = 2LL * a.H, pieces = (row_bytes + kMaxPiece - 1) / kMaxPiece;
  b.row_bytes = row_bytes;
  b.pieces = static_cast<int>(pieces);
  b.piece = static_cast<int>(((row_bytes + pieces - 1) / pieces + 15) / 16 * 16);
  const int smem = b.piece * kBulkWarps * kStages;
  const long long per_sm = (kRoom + 6000) / (smem + 6000);
  const long long most = (per_sm < 4 ? per_sm : 4) * device_sm_count();
  b.zero_rows = zero_rows(a, kBulkWarps * most);
  const long long items = a.T * pieces, blocks = a.src != nullptr ? (a.M + b.zero_rows - 1LL) / b.zero_rows : 0;
  const long long work = items > blocks ? items : blocks;
  return launch(dispatch_f16_kernel, work < most ? work : most, kBulkThreads, smem, stream, b, static_cast<const uint8_t*>(X),
                static_cast<uint8_t*>(Xs));
}

int launch_dispatch_fp8(const RowsArgs& a, const void* X, void* Xq, void* SFA, int fmt, cudaStream_t stream) {
  static PerDevice<int> cache[4];
  const long long items = static_cast<long long>(a.T) * ((a.H / 128 + 3) / 4);
  const bool masked = a.slots > 0;
  auto* fn = fmt ? (masked ? dispatch_fp8_kernel<true, true> : dispatch_fp8_kernel<true, false>)
                 : (masked ? dispatch_fp8_kernel<false, true> : dispatch_fp8_kernel<false, false>);
  return launch_items(fn, cache[(fmt ? 1 : 0) + (masked ? 2 : 0)], items, stream, a,
                      static_cast<const uint4*>(X), static_cast<uint4*>(Xq), static_cast<uint32_t*>(SFA));
}

int launch_combine_f16(const RowsArgs& a, const void* Ys, const float* W, void* Y, int bf16, cudaStream_t stream) {
  if (W != nullptr) return bf16 ? combine_by_k<true, true>(a, Ys, W, Y, stream) : combine_by_k<false, true>(a, Ys, W, Y, stream);
  return bf16 ? combine_by_k<true, false>(a, Ys, W, Y, stream) : combine_by_k<false, false>(a, Ys, W, Y, stream);
}

int launch_combine_f16_backward(const RowsArgs& a, const void* dY, const void* Ys, const float* W, void* dYs, float* dW,
                                int bf16, cudaStream_t stream) {
  return bf16 ? backward_by_k<true>(a, dY, Ys, W, dYs, dW, stream) : backward_by_k<false>(a, dY, Ys, W, dYs, dW, stream);
}

}  // namespace fgf8
