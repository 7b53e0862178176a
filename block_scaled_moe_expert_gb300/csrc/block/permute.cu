// Rows by expert and back (see sort.cu for the order).
//
//   place:  rows[inv[t, k]] = w[t, k] x[t], zeros elsewhere: the way to the
//           experts, and with the output's gradient as x the gradient of the
//           way back, which also wants <x[t], rows[inv[t, k]]>;
//   gather: out[t] = sum_k w[t, k] rows[inv[t, k]]: the way back, and the
//           gradient of the way to the experts (again with the dots).
//
// Both walk tokens, not rows: a token's own row is read (or written) once and
// its K rows move once each, so the traffic is the floor; walking rows would
// read each token's row up to K times, and its K visits lie too far apart in
// expert order for the L2 to keep it. Bound by DRAM bandwidth. Sums over k
// run in ascending k in fp32, without atomics, and round once.
#include "block_internal.cuh"
#include "../ptx.cuh"

namespace bsmoe {

namespace {

constexpr int kPermThreads = 256;
constexpr int kPermWarps = kPermThreads / 32;
constexpr int kKGroup = 8;    // rows of a token in flight together
constexpr int kZeroRows = 32;  // rows that a zero-fill block looks after

// Sums v[0..7] over the block; valid in thread 0..7 as the return value.
__device__ __forceinline__ float block_sum8(const float (&v)[kKGroup], float (*s)[kPermWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();  // the previous use of s
#pragma unroll
  for (int j = 0; j < kKGroup; ++j) {
    const float t = warp_sum(v[j]);
    if (lane == 0) s[j][warp] = t;
  }
  __syncthreads();
  float r = 0.f;
  if (threadIdx.x < kKGroup)
    for (int w = 0; w < kPermWarps; ++w) r += s[threadIdx.x][w];
  return r;
}

// grid (T + ceil(M / 32), column splits); the last blocks zero the rows that
// belong to no slot.
template <typename T, int V, bool W, bool DOTS>
__global__ void __launch_bounds__(kPermThreads)
place_kernel(PlaceArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int H = a.H, K = a.p.K;
  T* rows = static_cast<T*>(a.rows);
  const int c0 = (blockIdx.y * kPermThreads + threadIdx.x) * V, cstep = gridDim.y * kPermThreads * V;
  if (blockIdx.x >= a.p.T) {
    const int r0 = (blockIdx.x - a.p.T) * kZeroRows;
    Pack<T, V> z;
#pragma unroll
    for (int i = 0; i < V; ++i) z.e[i] = from_f32<T>(0.f);
    for (int r = r0; r < min(r0 + kZeroRows, a.p.M); ++r) {
      if (a.p.row_slot[r] >= 0) continue;
      T* dst = rows + static_cast<size_t>(r) * H;
      for (int c = c0; c < H; c += cstep) store_pack(dst + c, z);
    }
    return;
  }
  const size_t t = blockIdx.x;
  __shared__ int s_row[kMaxTopK];
  __shared__ float s_w[kMaxTopK];
  __shared__ float s_sum[kKGroup][kPermWarps];
  if (threadIdx.x < K) {
    s_row[threadIdx.x] = a.p.inv[t * K + threadIdx.x];
    s_w[threadIdx.x] = W ? a.w[t * K + threadIdx.x] : 1.f;
  }
  __syncthreads();
  const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
  const T* other = static_cast<const T*>(a.other);
  for (int k0 = 0; k0 < K; k0 += kKGroup) {
    float dot[kKGroup] = {};
    for (int c = c0; c < H; c += cstep) {
      const Pack<T, V> xp = load_pack<V>(x + c);
      float xf[V];
      if (W || DOTS) unpack(xp, xf);
      Pack<T, V> op[kKGroup];
      if (DOTS) {
#pragma unroll
        for (int j = 0; j < kKGroup; ++j)
          if (k0 + j < K && s_row[k0 + j] >= 0)
            op[j] = load_pack<V>(other + static_cast<size_t>(s_row[k0 + j]) * a.ld_other + c);
      }
#pragma unroll
      for (int j = 0; j < kKGroup; ++j) {
        if (k0 + j >= K || s_row[k0 + j] < 0) continue;
        T* dst = rows + static_cast<size_t>(s_row[k0 + j]) * H + c;
        if (W) {
          float o[V];
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] = s_w[k0 + j] * xf[i];
          store_pack(dst, pack<T, V>(o));
        } else {
          store_pack(dst, xp);
        }
        if (DOTS) {
          float of[V];
          unpack(op[j], of);
#pragma unroll
          for (int i = 0; i < V; ++i) dot[j] = fmaf(xf[i], of[i], dot[j]);
        }
      }
    }
    if (DOTS) {
      const float d = block_sum8(dot, s_sum);
      if (threadIdx.x < kKGroup && k0 + threadIdx.x < K) a.dots[t * K + k0 + threadIdx.x] = d;
    }
  }
}

// grid (T, column splits)
template <typename T, int V, bool W, bool DOTS>
__global__ void __launch_bounds__(kPermThreads)
gather_kernel(GatherArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int H = a.H, K = a.p.K;
  const size_t t = blockIdx.x;
  __shared__ int s_row[kMaxTopK];
  __shared__ float s_w[kMaxTopK];
  __shared__ float s_sum[kKGroup][kPermWarps];
  if (threadIdx.x < K) {
    s_row[threadIdx.x] = a.p.inv[t * K + threadIdx.x];
    s_w[threadIdx.x] = W ? a.w[t * K + threadIdx.x] : 1.f;
  }
  __syncthreads();
  const T* rows = static_cast<const T*>(a.rows);
  const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
  T* out = static_cast<T*>(a.out) + t * H;
  const int c0 = (blockIdx.y * kPermThreads + threadIdx.x) * V, cstep = gridDim.y * kPermThreads * V;
  // the columns of a block: all of them with dots (one block per token then)
  float dots[DOTS ? kMaxTopK : 1] = {};
  for (int c = c0; c < H; c += cstep) {
    float acc[V] = {};
    float xf[V];
    if (DOTS) unpack(load_pack<V>(x + c), xf);
#pragma unroll
    for (int k0 = 0; k0 < kMaxTopK; k0 += kKGroup) {
      if (k0 >= K) break;
      Pack<T, V> rp[kKGroup];
#pragma unroll
      for (int j = 0; j < kKGroup; ++j)
        if (k0 + j < K && s_row[k0 + j] >= 0)
          rp[j] = load_pack<V>(rows + static_cast<size_t>(s_row[k0 + j]) * a.ld_rows + c);
#pragma unroll
      for (int j = 0; j < kKGroup; ++j) {
        if (k0 + j >= K || s_row[k0 + j] < 0) continue;
        float rf[V];
        unpack(rp[j], rf);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          acc[i] = W ? fmaf(s_w[k0 + j], rf[i], acc[i]) : acc[i] + rf[i];
          if (DOTS) dots[k0 + j] = fmaf(xf[i], rf[i], dots[k0 + j]);
        }
      }
    }
    store_pack(out + c, pack<T, V>(acc));
  }
  if (DOTS) {
#pragma unroll
    for (int k0 = 0; k0 < kMaxTopK; k0 += kKGroup) {
      if (k0 >= K) break;
      float v[kKGroup];
#pragma unroll
      for (int j = 0; j < kKGroup; ++j) v[j] = dots[DOTS ? k0 + j : 0];
      const float d = block_sum8(v, s_sum);
      if (threadIdx.x < kKGroup && k0 + threadIdx.x < K) a.dots[t * K + k0 + threadIdx.x] = d;
    }
  }
}

// Column splits of a token's row: more blocks where the tokens alone do not
// fill the GPU (a handful of tokens at decode).
int column_splits(int T, int H, int V) {
  const int full = ceil_div(H, kPermThreads * V);
  return T >= 512 ? 1 : full;
}

template <typename T>
bool vec_ok(int H, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
  if (H % kVec<T>) return false;
  for (const void* p : ptrs)
    if (!aligned16(p)) return false;
  for (int64_t l : lds)
    if (l % kVec<T>) return false;
  return true;
}

template <typename T, int V>
cudaError_t place(const PlaceArgs& a, cudaStream_t st) {
  const int zero_blocks = ceil_div(a.p.M, kZeroRows);
  const bool dots = a.dots != nullptr;
  const dim3 grid(a.p.T + zero_blocks, dots ? 1 : column_splits(a.p.T, a.H, V));
  auto* k = a.w == nullptr ? place_kernel<T, V, false, false>
            : dots         ? place_kernel<T, V, true, true>
                           : place_kernel<T, V, true, false>;
  return launch_kernel(true, k, grid, kPermThreads, 0, st, a);
}

template <typename T, int V>
cudaError_t gather(const GatherArgs& a, cudaStream_t st) {
  const bool dots = a.dots != nullptr;
  const dim3 grid(a.p.T, dots ? 1 : column_splits(a.p.T, a.H, V));
  auto* k = a.w == nullptr ? gather_kernel<T, V, false, false>
            : dots         ? gather_kernel<T, V, true, true>
                           : gather_kernel<T, V, true, false>;
  return launch_kernel(true, k, grid, kPermThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_place(int dtype, const PlaceArgs& a, cudaStream_t st) {
  return with_dtype(dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    return vec_ok<T>(a.H, {a.x, a.other, a.rows}, {a.ld_x, a.ld_other}) ? place<T, kVec<T>>(a, st)
                                                                        : place<T, 1>(a, st);
  });
}

cudaError_t launch_gather(int dtype, const GatherArgs& a, cudaStream_t st) {
  return with_dtype(dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    return vec_ok<T>(a.H, {a.rows, a.x, a.out}, {a.ld_rows, a.ld_x}) ? gather<T, kVec<T>>(a, st)
                                                                     : gather<T, 1>(a, st);
  });
}

}  // namespace bsmoe
