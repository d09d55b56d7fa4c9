// route.cu -- places of tokens in the layouts of the grouped products: a stable counting
// sort of the tokens' group ids.
//
//   rank(i)  = #{ i' < i : id(i') = id(i) }
//   contiguous: row(i) = starts(id) + rank(i), starts = prefix sum of the counts rounded up
//   masked:     row(i) = slots id + rank(i), or none where rank(i) >= slots
//
// One launch of a few clusters, each of which counts all entries, so that they do not wait for
// one another, and places its share of them.  In a cluster a CTA takes a run of entries, each
// of its warps a run of those, so that (CTA, warp, step, lane) is the flat order and the ranks
// do not depend on timing.  A warp counts its run into its own row of a histogram in shared
// memory, the rows are summed over warps, the sums over CTAs through distributed shared memory,
// and a second walk hands out the rows of this cluster's warps: the lanes of one id are found
// by a ballot for each of its bits (__match_any_sync takes longer from some ten thousand entries
// on).  Every CTA scans the groups' counts for itself.  m_indices follows from the counts alone
// and is written in row order; src is the only scattered output.  Clusters instead of the whole
// GPU at once: the ids of 8192 tokens with 8 experts are 256 KB, and a barrier across a cluster
// is a hardware barrier, while one across the grid would be a second launch.  Bound by
// the chain of steps (ids, counts, barrier, sums, rows) and by instruction issue: 7.2 us at
// 8192 x 8 ids of 32 groups, 4 % of the dispatch that follows; one cluster for all takes 8.2.
#include <cstring>

#include "gemm_persistent.cuh"
#include "per_device.h"
#include "routed.h"

namespace fgf8 {
namespace {

constexpr int kMaxThreads = 1024, kMaxWarps = kMaxThreads / 32;
constexpr int kMaxCluster = 16;                             // where the device fits so many, else kPortableCluster
constexpr int kPortableCluster = 8;
constexpr int kAhead = 4;                                   // steps of ids that a warp loads together
constexpr int kChunk = 128;                                 // rows of the layout that a warp fills together
constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ long long ld_global_s64(const void* p) {
  long long v;
  asm volatile("ld.global.s64 %0, [%1];" : "=l"(v) : "l"(p));
  return v;
}

// Lanes of the warp with the same id (-1 .. G - 1); `bits` bits of id + 1 hold G.
__device__ __forceinline__ uint32_t same_id(int id, int bits) {
  const uint32_t key = static_cast<uint32_t>(id + 1);
  uint32_t same = kFull;
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1u;
    const uint32_t ones = __ballot_sync(kFull, one);
    same &= one ? ones : ~ones;
  }
  return same;
}

// The group of entry i, -1 for none and for what is out of range.
template <bool IDS64>
__device__ __forceinline__ int load_id(const RouteArgs& a, int i, int end, bool& bad) {
  if (i >= end) return -1;
  long long id;
  if constexpr (IDS64)
    id = ld_global_s64(static_cast<const long long*>(a.ids) + i);
  else
    id = ptx::ld_global(static_cast<const int32_t*>(a.ids) + i);
  if (id >= 0 && id < a.G) return static_cast<int>(id);
  bad |= id != -1;
  return -1;
}

// Two CTAs to an SM: in 32 registers a thread, where the next kernel's CTAs can stand beside
// them and wait.  In 64 the route of 8192 x 8 ids and the dispatch_f16 behind it take 205 us
// together, 201 in 32.
template <bool IDS64>
__global__ void __launch_bounds__(kMaxThreads, 2) route_kernel(RouteArgs a, int S) {
  extern __shared__ int32_t smem[];
  const int G = a.G;
  const int cluster = static_cast<int>(blockIdx.x) / S, clusters = static_cast<int>(gridDim.x) / S;   // S CTAs each
  const int threads = static_cast<int>(blockDim.x), W = threads >> 5;
  int32_t* hist = smem;                                     // [warp][G]
  int32_t* total = hist + W * G;                            // [G] this CTA's counts
  int32_t* first = total + G;                               // [G + 1] first row of each group
  int32_t* base = first + G + 1;                            // [G] row of this CTA's first entry of each group (masked: its rank)
  int32_t* count = base + G;                                // [G] entries with a row, over all CTAs
  __shared__ int32_t warp_sum[kMaxWarps];
  const int bits = 32 - __clz(G), top = 1 << (bits - 1);    // of G, and the highest power of two up to it
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  for (int i = tid; i < W * G; i += threads) hist[i] = 0;
  ptx::griddep_wait();                                      // ids may come from the previous kernel
  ptx::griddep_launch_dependents();
  __syncthreads();

  // this warp's run of entries, whole steps of 32
  const long long steps = (static_cast<long long>(a.n) + 31) / 32;
  const long long per = (steps + S * W - 1) / (S * W);
  const long long lo = (static_cast<long long>(rank) * W + warp) * per * 32;
  const int begin = static_cast<int>(lo < a.n ? lo : a.n);
  const int end = static_cast<int>(lo + per * 32 < a.n ? lo + per * 32 : a.n);
  int32_t* mine = hist + warp * G;
  bool bad = false;
  int id[kAhead];
  for (int i0 = begin; i0 < end; i0 += 32 * kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) id[u] = load_id<IDS64>(a, i0 + 32 * u + lane, end, bad);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (id[u] >= 0) atomicAdd(mine + id[u], 1);
  }
  if (bad) atomicOr(a.status, FGF8_DEVERR_INPUT);
  __syncthreads();

  // counts of this CTA, and each warp's offset within them: a thread per group
  if (tid < G) {
    int32_t sum = 0;
    for (int w = 0; w < W; w += 8) {
      int32_t c[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) c[u] = w + u < W ? hist[(w + u) * G + tid] : 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (w + u < W) hist[(w + u) * G + tid] = sum;
        sum += c[u];
      }
    }
    total[tid] = sum;
  }
  if (S > 1) cluster_sync_all(); else __syncthreads();
  int32_t before = 0, all = 0;                              // of group tid: entries of earlier CTAs, of all
  if (tid < G) {
    const uint32_t at = ptx::smem_u32(total + tid);
    for (int r = 0; r < S; r += kPortableCluster) {
      uint32_t c[kPortableCluster] = {};                    // in flight together
#pragma unroll
      for (int u = 0; u < kPortableCluster; ++u)
        if (r + u < S) c[u] = ld_cluster_u32(map_to_rank(at, static_cast<uint32_t>(r + u)));
#pragma unroll
      for (int u = 0; u < kPortableCluster; ++u) {
        if (r + u < rank) before += static_cast<int32_t>(c[u]);
        all += static_cast<int32_t>(c[u]);
      }
    }
  }
  if (S > 1) cluster_arrive();                              // behind this nothing remote is read
  // first rows: an exclusive prefix sum of the padded counts, one group per thread.  A padded
  // count fits the M rows; a count plus a segment need not fit 32 bits.
  const int32_t padded = a.slots > 0 ? a.slots : (all / a.align + (all % a.align != 0 ? 1 : 0)) * a.align;
  const int32_t held = a.slots > 0 && all > a.slots ? a.slots : all;
  int32_t scan = tid < G ? padded : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int32_t v = __shfl_up_sync(kFull, scan, off);
    if (lane >= off) scan += v;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  if (tid < G) {
    int32_t start = scan - padded;
    for (int w = 0; w < warp; ++w) start += warp_sum[w];
    first[tid] = start;
    if (tid == G - 1) first[G] = start + padded;
    base[tid] = a.slots > 0 ? before : start + before;
    count[tid] = held;
    if (blockIdx.x == 0) {
      a.counts[tid] = held;
      if (a.starts != nullptr) {
        a.starts[tid] = start;
        if (tid == G - 1) a.starts[G] = start + padded;
      }
    }
  }
  __syncthreads();

  // the rows of the entries that fall to this cluster
  for (int i0 = warp % clusters == cluster ? begin : end; i0 < end; i0 += 32 * kAhead) {
    bool ignored = false;
    if (per > kAhead) {                                     // else the registers still hold them
#pragma unroll
      for (int u = 0; u < kAhead; ++u) id[u] = load_id<IDS64>(a, i0 + 32 * u + lane, end, ignored);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i0 + 32 * u >= end) break;
      const int i = i0 + 32 * u + lane;
      const uint32_t same = same_id(id[u], bits), earlier = same & ((1u << lane) - 1u);
      int32_t row = -1;
      if (id[u] >= 0) row = base[id[u]] + mine[id[u]] + __popc(earlier);
      __syncwarp();
      if (id[u] >= 0 && earlier == 0) mine[id[u]] += __popc(same);
      __syncwarp();
      if (a.slots > 0 && id[u] >= 0) row = row < a.slots ? id[u] * a.slots + row : -1;
      // ids that changed since they were counted (they must not) may leave the layout
      if (row >= a.M) row = -1;
      if (i < end) {
        a.rows[i] = row;
        if (row >= 0) a.src[row] = i;
      }
    }
  }
  // m_indices, and src of the rows without an entry, in row order, kChunk rows to a warp
  const long long ctas = gridDim.x;
  for (long long r0 = (warp * ctas + blockIdx.x) * kChunk; r0 < a.M; r0 += ctas * W * kChunk) {
    int g = 0;                                              // the last group that begins at or before r0
    for (int half = top; half > 0; half >>= 1)
      if (g + half <= G && first[g + half] <= r0) g += half;
#pragma unroll
    for (int u = 0; u < kChunk / 32; ++u) {
      const int32_t row = static_cast<int32_t>(r0) + 32 * u + lane;
      if (row >= a.M) break;
      while (g < G && first[g + 1] <= row) ++g;
      const bool owned = g < G && row - first[g] < count[g];
      if (a.m_indices != nullptr) a.m_indices[row] = owned ? g : -1;
      if (!owned) a.src[row] = -1;
    }
  }
  if (S > 1) cluster_wait();                                // stay until every CTA has read the counts
}

size_t smem_bytes(int G, int warps) { return sizeof(int32_t) * (static_cast<size_t>(warps) * G + 4 * static_cast<size_t>(G) + 1); }

struct RouteLaunch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  RouteLaunch(int ctas, int clusters, int threads, size_t smem, cudaStream_t stream, bool pdl) {
    std::memset(&cfg, 0, sizeof(cfg));
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas * clusters), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
  }
};

// The largest cluster that the device fits, and how many of kMaxCluster CTAs side by side.
struct Fit {
  int ctas, clusters;
};

template <bool IDS64>
int launch(const RouteArgs& a, cudaStream_t stream) {
  auto* fn = &route_kernel<IDS64>;
  static PerDevice<Fit> fits;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  const Fit* fit = nullptr;
  const int r = fits.get(dev, &fit, [&](Fit& f) {
    const size_t smem = smem_bytes(kRouteMaxGroups, kMaxWarps);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    int clusters = 0;
    if (e == cudaSuccess) {
      RouteLaunch l(kMaxCluster, 1, kMaxThreads, smem, nullptr, false);
      e = cudaOccupancyMaxActiveClusters(&clusters, fn, &l.cfg);
    }
    if (e != cudaSuccess) return set_error(4, "route set-up: %s", cudaGetErrorString(e));
    f.ctas = clusters > 0 ? kMaxCluster : kPortableCluster;
    f.clusters = clusters;
    return 0;
  });
  if (r) return r;
  // CTAs that share the counting, and groups of them.  One CTA (sixteen times where there are more
  // rows than it fills at once), eight eight times and sixteen four times, in us: 3.3, 3.5 and 3.9
  // at 64 x 8 ids of 32 groups, 5.2, 3.7 and 4.9 at 512 x 8, 5.0 and 4.9 (the last two) at
  // 2048 x 8, 8.8 and 7.1 at 8192 x 8, 26.8 and 21.1 at 32768 x 8 of 256.  Eight times sixteen
  // CTAs are more than fit side by side: 11.7 at 8192 x 8.
  const int ctas = a.n <= 512 ? 1 : a.n <= 16384 ? kPortableCluster : fit->ctas;
  const int clusters = ctas == 1 ? (static_cast<long long>(a.n) + a.M <= 4096 ? 1 : 16) : ctas == kMaxCluster ? (fit->clusters < 4 ? fit->clusters : 4) : 8;
  // a thread for each entry of a CTA, and for each group
  const long long least = a.G > 256 ? a.G : 256, each = (static_cast<long long>(a.n) + ctas - 1) / ctas, want = each > least ? each : least;
  const int threads = want < kMaxThreads ? static_cast<int>((want + 31) / 32 * 32) : kMaxThreads;
  RouteLaunch l(ctas, clusters, threads, smem_bytes(a.G, threads / 32), stream, pdl_enabled());
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, fn, a, ctas);
  return e == cudaSuccess ? 0 : set_error(4, "route launch: %s", cudaGetErrorString(e));
}

}  // namespace

int launch_route(const RouteArgs& a, cudaStream_t stream) {
  return a.ids64 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace fgf8
