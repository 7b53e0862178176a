// Shared by the norms' forward and gradient kernels: row sums, gates,
// weights of either type.
#pragma once
#include "block_internal.cuh"
#include "../ptx.cuh"

namespace bsmoe {

// N sums over the threads of a row: a warp (WARP) or the whole block, with
// one barrier. A scratch s may be written again once every thread has passed
// a later barrier: callers use one per sum of a row and alternate by row.
template <int N, bool WARP>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*s)[32]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (WARP) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i][warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? s[i][lane] : 0.f);
}

__device__ __forceinline__ float gate_value(int act, float v) {
  if (act == MOE_GATE_SIGMOID) return 1.f / (1.f + expf(-v));
  if (act == MOE_GATE_TANH) return tanhf(v);
  return v;
}
// d act / d gate from the activation's value.
__device__ __forceinline__ float gate_slope(int act, float g) {
  if (act == MOE_GATE_SIGMOID) return g * (1.f - g);
  if (act == MOE_GATE_TANH) return 1.f - g * g;
  return 1.f;
}

// w_offset + weight (1 without a weight) of columns c..c+V-1.
template <typename T, int V>
__device__ __forceinline__ void load_weight(const void* w, int w_f32, float offset, int c, float (&f)[V]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 1.f;
  } else if (w_f32 && sizeof(T) != 4) {
    constexpr int V4 = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < V; i += V4) {
      const Pack<float, V4> p = load_pack<V4>(static_cast<const float*>(w) + c + i);
#pragma unroll
      for (int j = 0; j < V4; ++j) f[i + j] = p.e[j] + offset;
    }
  } else {
    unpack(load_pack<V>(static_cast<const T*>(w) + c), f);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] += offset;
  }
}

// Every operand allows 16-byte accesses (null pointers and unused strides of
// 0 pass).
template <typename T>
bool rows_vectorize(int H, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
  if (H % kVec<T>) return false;
  for (const void* p : ptrs)
    if (!aligned16(p)) return false;
  for (const int64_t l : lds)
    if (l % kVec<T>) return false;
  return true;
}

}  // namespace bsmoe
