// Tokens sorted by expert: the stable counting sort of the T*K slots into
// groups whose starts are multiples of a caller-chosen alignment.
//
// A slot's row is the group's start + the number of equal ids before it. The
// slots are cut into consecutive ranges, one per warp; a warp walks its range
// 32 slots at a time and __match_any_sync finds the equal ids inside a step.
// Pass 1 counts per warp and expert; the counts are summed over the warps of
// a CTA and, through distributed shared memory, over the CTAs of a cluster;
// pass 2 walks again and places. No data atomics: the result is exact and
// the same on every run.
//
// Bound by latency, not bandwidth (262,144 slots are 1 MB in, 1 MB out): the
// cluster keeps the counts of large batches on chip and the sort at one
// launch.
#include <cooperative_groups.h>

#include "block_internal.cuh"
#include "../ptx.cuh"

namespace cg = cooperative_groups;

namespace bsmoe {

namespace {

constexpr int kSortWarps = 32;
constexpr int kSortThreads = kSortWarps * 32;
constexpr int kSortCluster = 8;
constexpr int kSortOneCta = 4096;  // up to this many slots one CTA sorts alone

// Exclusive scan of one value per thread (1024 threads).
__device__ __forceinline__ int excl_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    const int c = warp_sums[w];
    before += w < warp ? c : 0;
    all += c;
  }
  *total = all;
  return before + x - v;
}

__global__ void __launch_bounds__(kSortThreads, 1)
sort_kernel(const int32_t* __restrict__ idx, SortPlan p, int range, int cluster_size) {
  extern __shared__ int smem[];
  const int stride = p.E + 1;
  int* hist = smem;                          // [warps][E + 1]
  int* total = smem + kSortWarps * stride;   // [E + 1] of this CTA
  int* start = total + stride;               // [E + 1] first row of each group
  int* base_row = start + stride;            // [E + 1] first row of this CTA's slots of each group
  __shared__ int warp_sums[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_size > 1 ? static_cast<int>(blockIdx.x) : 0;
  const int gwarp = rank * kSortWarps + warp;
  pdl_wait();
  pdl_launch_dependents();
  for (int i = tid; i < kSortWarps * stride; i += kSortThreads) hist[i] = 0;
  // the status word reflects the latest sort; ids are checked in pass 2,
  // after the barriers below
  if (rank == 0 && tid == 0) *p.status = 0u;
  __syncthreads();

  const int beg = min(p.S, gwarp * range), end = min(p.S, beg + range);
  int* h = hist + warp * stride;
  for (int base = beg; base < end; base += 32) {
    const int s = base + lane;
    const unsigned active = __ballot_sync(0xffffffffu, s < end);
    if (s < end) {
      const int v = __ldg(idx + s);
      const int key = (v >= 0 && v < p.E) ? v : p.E;
      const unsigned peers = __match_any_sync(active, key);
      if (lane == __ffs(peers) - 1) h[key] += __popc(peers);
    }
    __syncwarp();
  }
  __syncthreads();
  // per expert: the counts of earlier warps, in place, and the CTA's total
  if (tid < stride) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
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
#pragma unroll
      for (int r = 0; r < kSortCluster; ++r) {
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
  const int warps = cluster_size * kSortWarps;
  for (int e = gwarp; e < p.E; e += warps)
    for (int r = start[e] + total[e] + lane; r < start[e + 1]; r += 32) p.row_slot[r] = -1;
  for (int r = used + gwarp * 32 + lane; r < p.M; r += warps * 32) p.row_slot[r] = -1;

  for (int base = beg; base < end; base += 32) {
    const int s = base + lane;
    const unsigned active = __ballot_sync(0xffffffffu, s < end);
    if (s < end) {
      const int v = __ldg(idx + s);
      const bool valid = v >= 0 && v < p.E;
      const int key = valid ? v : p.E;
      const unsigned peers = __match_any_sync(active, key);
      const int row = h[key] + __popc(peers & ((1u << lane) - 1u)) + base_row[key];
      __syncwarp(active);
      if (lane == __ffs(peers) - 1) h[key] += __popc(peers);
      p.inv[s] = valid ? row : -1;
      if (valid) p.row_slot[row] = s;
      else if (v != -1) atomicOr(p.status, MOE_DEV_BAD_EXPERT_ID);
    }
    __syncwarp();
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

cudaError_t launch_sort(const int32_t* topk_idx, const SortPlan& p, cudaStream_t st) {
  const int cluster = p.S <= kSortOneCta ? 1 : kSortCluster;
  const int warps = cluster * kSortWarps;
  const int range = ceil_div(ceil_div(p.S, warps), 32) * 32;
  const size_t smem = sizeof(int) * (kSortWarps + 3) * (p.E + 1);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = cluster;
  cfg.blockDim = kSortThreads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sort_kernel, topk_idx, p, range, cluster);
}

}  // namespace bsmoe
