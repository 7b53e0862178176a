// Tokens sorted by expert: the stable counting sort of the T*K slots into
// groups whose starts are multiples of a caller-chosen alignment.
//
// A slot's row is the group's start + the number of equal ids before it. The
// slots are cut into consecutive ranges, one per warp; a warp walks its range
// 32 slots at a time and a ballot for each bit of the id finds the equal ids
// inside a step (the match instruction does the same, but slowly where the ids
// differ: 65,536 slots over 256 experts took 23 us with it).
// Pass 1 counts per warp and expert and leaves each slot's rank in its warp's
// range in inv; the counts are summed over the warps of a CTA and, through
// distributed shared memory, over the CTAs of a cluster; pass 2 adds the
// group's start and the counts before the warp. No data atomics: the result is exact and
// the same on every run.
//
// Bound by latency, not bandwidth (65,536 slots are 0.3 MB in, 0.6 MB out): the
// cluster keeps the counts of large batches on chip and the sort at one
// launch. Measured with cold caches: 32 slots over 256 experts 6.4 us, 65,536
// 12.7 us (8 CTAs: 16.5), 131,072 over 512 20 us (8 CTAs: 30).
#include <cooperative_groups.h>

#include <atomic>

#include "block_internal.cuh"
#include "../ptx.cuh"

namespace cg = cooperative_groups;

namespace bsmoe {

namespace {

constexpr int kSortWarps = 32;  // at most, of a CTA
constexpr int kSortThreads = kSortWarps * 32;
constexpr int kSortAhead = 8;  // steps whose ids are loaded together
constexpr int kSortWide = 16384;   // from this many slots on the cluster has 16 CTAs, else 8
constexpr int kSortOneCta = 1024;  // up to this many slots one CTA sorts alone

// The lanes of `active` with this lane's key (of `bits` bits).
__device__ __forceinline__ unsigned equal_keys(unsigned active, int key, int bits) {
  unsigned peers = active;
#pragma unroll
  for (int b = 0; b < 10; ++b) {  // 512 experts and the skipped ones
    if (b >= bits) break;
    const bool one = (key >> b) & 1;
    const unsigned ones = __ballot_sync(active, one);
    peers &= one ? ones : ~ones;
  }
  return peers;
}

// The ids of the next steps, loaded together: a step is shorter than a load.
__device__ __forceinline__ void load_ids(int (&id)[kSortAhead], const int32_t* __restrict__ idx, int s, int end) {
#pragma unroll
  for (int j = 0; j < kSortAhead; ++j) id[j] = s + 32 * j < end ? __ldg(idx + s + 32 * j) : 0;
}

// Exclusive scan of one value per thread.
__device__ __forceinline__ int excl_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const int c = lane < warps ? warp_sums[lane] : 0;
  *total = __reduce_add_sync(0xffffffffu, c);
  return __reduce_add_sync(0xffffffffu, lane < warp ? c : 0) + x - v;
}

__global__ void __launch_bounds__(kSortThreads, 1)
sort_kernel(const int32_t* __restrict__ idx, SortPlan p, int range, int count_warps, int cluster_size) {
  extern __shared__ int smem[];
  const int stride = p.E + 1, bits = 32 - __clz(p.E);
  int* hist = smem;                          // [count_warps][E + 1]
  int* total = smem + count_warps * stride;  // [E + 1] of this CTA
  int* start = total + stride;               // [E + 1] first row of each group
  int* base_row = start + stride;            // [E + 1] first row of this CTA's slots of each group
  __shared__ int warp_sums[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_size > 1 ? static_cast<int>(blockIdx.x) : 0;
  const int block_warps = blockDim.x >> 5, gwarp = rank * block_warps + warp;
  pdl_wait();
  pdl_launch_dependents();
  for (int i = tid; i < count_warps * stride; i += blockDim.x) hist[i] = 0;
  // the status word reflects the latest sort; ids are checked in pass 2,
  // after the barriers below
  if (rank == 0 && tid == 0) *p.status = 0u;
  __syncthreads();

  // (warps behind count_warps have no slots)
  const int beg = warp < count_warps ? min(p.S, (rank * count_warps + warp) * range) : p.S, end = min(p.S, beg + range);
  int* h = hist + warp * stride;
  for (int base = beg; base < end; base += 32 * kSortAhead) {
    int id[kSortAhead];
    load_ids(id, idx, base + lane, end);
#pragma unroll
    for (int j = 0; j < kSortAhead; ++j) {
      if (base + 32 * j >= end) break;
      const int s = base + 32 * j + lane;
      const unsigned active = __ballot_sync(0xffffffffu, s < end);
      if (s < end) {
        const int key = (id[j] >= 0 && id[j] < p.E) ? id[j] : p.E;
        const unsigned peers = equal_keys(active, key, bits);
        p.inv[s] = h[key] + __popc(peers & ((1u << lane) - 1u));
        __syncwarp(active);
        if (lane == __ffs(peers) - 1) h[key] += __popc(peers);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  // per expert: the counts of earlier warps, in place, and the CTA's total
  if (tid < stride) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < count_warps; ++w) {
      const int c = hist[w * stride + tid];
      hist[w * stride + tid] = run;
      run += c;
    }
    total[tid] = run;
  }
  int before = 0, count = 0;  // of expert tid: in earlier CTAs, in all
  if (cluster_size > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (tid < stride) {
#pragma unroll 8
      for (int r = 0; r < cluster_size; ++r) {
        const int c = cluster.map_shared_rank(total, r)[tid];
        before += r < rank ? c : 0;
        count += c;
      }
    }
    cluster.sync();  // no CTA leaves while its totals are read
  } else if (tid < stride) {
    count = total[tid];
  }
  const int padded = tid < p.E ? (count + p.align - 1) / p.align * p.align : 0;
  int used;
  const int first = excl_scan(padded, warp_sums, &used);
  if (tid < stride) {
    start[tid] = tid < p.E ? first : used;
    if (rank == 0) {
      if (tid < p.E) p.counts[tid] = count;
      p.offsets[tid] = tid < p.E ? first : used;
    }
  }
  if (tid < stride) {
    total[tid] = count;
    base_row[tid] = first + before;
  }
  __syncthreads();
  // rows of no slot: behind each group, and behind the last one
  const int warps = cluster_size * block_warps;
  for (int e = gwarp; e < p.E; e += warps)
    for (int r = start[e] + total[e] + lane; r < start[e + 1]; r += 32) p.row_slot[r] = -1;
  for (int r = used + gwarp * 32 + lane; r < p.M; r += warps * 32) p.row_slot[r] = -1;

  for (int base = beg + lane; base < end; base += 32 * kSortAhead) {
    int id[kSortAhead], rank_in_warp[kSortAhead];
    load_ids(id, idx, base, end);
#pragma unroll
    for (int j = 0; j < kSortAhead; ++j) rank_in_warp[j] = base + 32 * j < end ? p.inv[base + 32 * j] : 0;
#pragma unroll
    for (int j = 0; j < kSortAhead; ++j) {
      const int s = base + 32 * j;
      if (s >= end) break;
      const int e = id[j];
      if (e >= 0 && e < p.E) {
        const int row = base_row[e] + h[e] + rank_in_warp[j];
        p.inv[s] = row;
        p.row_slot[row] = s;
      } else {
        p.inv[s] = -1;
        if (e != -1) atomicOr(p.status, MOE_DEV_BAD_EXPERT_ID);
      }
    }
  }
}

}  // namespace

bool sort_layout(int T, int E, int K, int row_align, moe_sort_layout* out) {
  if (T < 0 || E < 1 || E > kMaxExperts || K < 1 || K > kMaxTopK || row_align < 1 || row_align > kMaxRowAlign)
    return false;
  const long long S = static_cast<long long>(T) * K;
  if (S > (1ll << 26)) return false;
  const long long M = (S + std::min<long long>(E, S) * (row_align - 1)) / row_align * row_align;
  size_t off = 0;
  auto take = [&](size_t ints) {
    const size_t o = off;
    off = align_up(off + 4 * ints, 256);
    return o;
  };
  out->status = take(1);
  out->counts = take(E);
  out->offsets = take(E + 1);
  out->inv = take(S);
  out->row_slot = take(M);
  out->total_bytes = off;
  out->row_capacity = static_cast<int32_t>(M);
  return true;
}

namespace {

constexpr size_t kSortMaxSmem = sizeof(int) * (kSortWarps + 3) * (kMaxExperts + 1);

// Whether the current device runs clusters of 16 CTAs (they need a GPC with that
// many SMs): asked once a device. That the kernel may have them is a limit of the
// kernel there and is set in every call, as the one on shared memory is.
bool wide_clusters_fit() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // 0: not asked yet, 1: yes, -1: no
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices ||
      cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      allow_smem(sort_kernel, kSortMaxSmem, kSortMaxSmem) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (const int answer = known[dev].load(std::memory_order_relaxed)) return answer > 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = 16;
  cfg.blockDim = kSortThreads;
  cfg.dynamicSmemBytes = kSortMaxSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 16;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, sort_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  known[dev].store(clusters > 0 ? 1 : -1, std::memory_order_relaxed);
  return clusters > 0;
}

}  // namespace

cudaError_t launch_sort(const int32_t* topk_idx, const SortPlan& p, cudaStream_t st) {
  // one CTA with a warp per 32 slots (and a thread per expert); a cluster of
  // full CTAs for large batches
  const int cluster = p.S <= kSortOneCta ? 1 : p.S >= kSortWide && wide_clusters_fit() ? 16 : 8;
  const int count_warps = cluster > 1 ? kSortWarps : std::max(1, std::min(kSortWarps, ceil_div(p.S, 32)));
  const int range = ceil_div(ceil_div(p.S, cluster * count_warps), 32) * 32;
  const int threads = std::max(count_warps, ceil_div(p.E + 1, 32)) * 32;
  const size_t smem = sizeof(int) * (count_warps + 3) * (p.E + 1);
  if (smem > 48 * 1024) {
    const cudaError_t e = allow_smem(sort_kernel, smem, kSortMaxSmem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = cluster;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sort_kernel, topk_idx, p, range, count_warps, cluster);
}

}  // namespace bsmoe
