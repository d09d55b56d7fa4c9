// route.cu -- places of tokens in the layouts of the grouped products: a stable counting
// sort of the tokens' group ids.
//
//   rank(i)  = #{ i' < i : id(i') = id(i) }
//   contiguous: row(i) = starts(id) + rank(i), starts = prefix sum of the counts rounded up
//   masked:     row(i) = slots id + rank(i), or none where rank(i) >= slots
//
// One launch of one cluster.  A CTA takes a run of entries, each of its warps a run of
// those, so that (CTA, warp, step, lane) is the flat order and the ranks do not depend on
// timing.  A warp counts its run into its own row of a histogram in shared memory
// (__match_any_sync: the lanes of one id are counted by one of them, without atomics), the
// rows are summed over warps, the sums over CTAs through distributed shared memory, and a
// second walk hands out the rows.  Every CTA scans the groups' counts for itself.  One
// cluster instead of the whole GPU: the ids of 8192 tokens with 8 experts are 256 KB, and
// a barrier across a cluster is a hardware barrier, while one across the grid would be a
// second launch.
#include <cstring>

#include "gemm_persistent.cuh"
#include "per_device.h"
#include "routed.h"

namespace fgf8 {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

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

template <bool IDS64>
__global__ void __launch_bounds__(kThreads, 1) route_kernel(RouteArgs a) {
  extern __shared__ int32_t smem[];
  const int G = a.G, S = static_cast<int>(gridDim.x);       // the grid is one cluster
  int32_t* hist = smem;                                     // [warp][G]
  int32_t* total = hist + kWarps * G;                       // [G] this CTA's counts
  int32_t* first = total + G;                               // [G + 1] first row of each group
  int32_t* count = first + G + 1;                           // [G] counts over all CTAs
  __shared__ int32_t warp_sum[kWarps];
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  for (int i = tid; i < kWarps * G; i += kThreads) hist[i] = 0;
  ptx::griddep_wait();                                      // ids may come from the previous kernel
  ptx::griddep_launch_dependents();
  __syncthreads();

  // this warp's run of entries, whole steps of 32
  const long long steps = (static_cast<long long>(a.n) + 31) / 32;
  const long long per = (steps + S * kWarps - 1) / (S * kWarps);
  const long long lo = (static_cast<long long>(rank) * kWarps + warp) * per * 32;
  const int begin = static_cast<int>(lo < a.n ? lo : a.n);
  const int end = static_cast<int>(lo + per * 32 < a.n ? lo + per * 32 : a.n);
  int32_t* mine = hist + warp * G;
  bool bad = false;
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int id = load_id<IDS64>(a, i0 + lane, end, bad);
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
    if (id >= 0 && (same & ((1u << lane) - 1u)) == 0) mine[id] += __popc(same);
    __syncwarp();
  }
  if (bad) atomicOr(a.status, FGF8_DEVERR_INPUT);
  __syncthreads();

  // counts of this CTA, and each warp's offset within them
  for (int g = tid; g < G; g += kThreads) {
    int32_t sum = 0;
    for (int w = 0; w < kWarps; ++w) {
      const int32_t c = hist[w * G + g];
      hist[w * G + g] = sum;
      sum += c;
    }
    total[g] = sum;
  }
  cluster_sync_all();
  int32_t before = 0, all = 0;                              // of group tid: entries of earlier CTAs, of all
  if (tid < G) {
    const uint32_t at = ptx::smem_u32(total + tid);
    for (int r = 0; r < S; ++r) {
      const int32_t c = static_cast<int32_t>(ld_cluster_u32(map_to_rank(at, static_cast<uint32_t>(r))));
      if (r < rank) before += c;
      all += c;
    }
    count[tid] = all;
  }
  // first rows: an exclusive prefix sum of the padded counts, one group per thread
  const int32_t padded = a.slots > 0 ? 0 : (all + a.align - 1) / a.align * a.align;
  int32_t scan = padded;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int32_t v = __shfl_up_sync(0xFFFFFFFFu, scan, off);
    if (lane >= off) scan += v;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  int32_t start = scan - padded;
  for (int w = 0; w < warp; ++w) start += warp_sum[w];
  if (tid < G) first[tid] = a.slots > 0 ? tid * a.slots : start;
  if (tid == G - 1) first[G] = a.slots > 0 ? G * a.slots : start + padded;
  if (tid < G) {
    const int32_t base = a.slots > 0 ? before : start + before;
    for (int w = 0; w < kWarps; ++w) hist[w * G + tid] += base;
    if (rank == 0) {
      a.counts[tid] = a.slots > 0 && all > a.slots ? a.slots : all;
      if (a.starts != nullptr) {
        a.starts[tid] = start;
        if (tid == G - 1) a.starts[G] = start + padded;
      }
    }
  }
  __syncthreads();

  // the entries' rows
  for (int i0 = begin; i0 < end; i0 += 32) {
    bool ignored = false;
    const int i = i0 + lane, id = load_id<IDS64>(a, i, end, ignored);
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
    const uint32_t earlier = same & ((1u << lane) - 1u);
    int32_t row = -1;
    if (id >= 0) row = mine[id] + __popc(earlier);
    __syncwarp();
    if (id >= 0 && earlier == 0) mine[id] += __popc(same);
    __syncwarp();
    if (a.slots > 0 && id >= 0) row = row < a.slots ? id * a.slots + row : -1;
    if (i < end) {
      a.rows[i] = row;
      if (row >= 0) {
        a.src[row] = i;
        if (a.m_indices != nullptr) a.m_indices[row] = id;
      }
    }
  }
  // rows without an entry: behind each group's, and behind the last group
  for (int g = rank * kWarps + warp; g <= G; g += S * kWarps) {
    const int32_t stop = g < G ? first[g + 1] : a.M;
    const int32_t held = g < G ? (a.slots > 0 && count[g] > a.slots ? a.slots : count[g]) : 0;
    for (int32_t row = first[g] + held + lane; row < stop; row += 32) {
      a.src[row] = -1;
      if (a.m_indices != nullptr) a.m_indices[row] = -1;
    }
  }
  cluster_sync_all();                                       // stay until every CTA has read the counts
}

constexpr int kMaxCluster = 8;

template <bool IDS64>
int launch(const RouteArgs& a, cudaStream_t stream) {
  auto* fn = &route_kernel<IDS64>;
  const size_t smem = sizeof(int32_t) * (static_cast<size_t>(kWarps + 3) * a.G + 1);
  static PerDevice<int> ready;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return set_error(2, "device id %d", dev);
  const int* set = nullptr;
  const int r = ready.get(dev, &set, [&](int& v) {
    v = static_cast<int>(sizeof(int32_t)) * ((kWarps + 3) * kRouteMaxGroups + 1);
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v);
    return e == cudaSuccess ? 0 : set_error(4, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  });
  if (r) return r;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[2];
  // one CTA walks up to four steps per warp alone; past that a cluster shares them
  const unsigned ctas = a.n <= 4 * kThreads ? 1u : static_cast<unsigned>(kMaxCluster);
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, a);
  return e == cudaSuccess ? 0 : set_error(4, "route launch: %s", cudaGetErrorString(e));
}

}  // namespace

int launch_route(const RouteArgs& a, cudaStream_t stream) {
  return a.ids64 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace fgf8
