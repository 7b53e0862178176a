// Shared by the norms' forward and gradient kernels: the rows' way into
// registers, row sums, gates, weights of either type.
#pragma once
#include "../ptx.cuh"
#include "block_internal.cuh"

namespace bsmoe {

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Thread j of a row owns the packs j, j + threads, ... (CH of them) of every
// row that its block (or warp) walks. With STAGES > 0 its packs of the next
// STAGES - 1 rows are on their way into its own slots of shared memory while
// it works on one: nobody else reads them, so there is no barrier in the
// queue. Packs that asynchronous copies cannot carry (V = 1), or rows too
// long for shared memory, are read from global memory where they are used
// (STAGES = 0), a second time from the L1.
template <typename T, int V, int CH, int ARRAYS, int STAGES>
struct RowQueue {
  const T* src[ARRAYS];  // null: absent
  int64_t ld[ARRAYS];
  int H, threads, j;
  int64_t row, step, last;  // rows row, row + step, ... below last
  // STAGES > 0: [STAGES][arrays present][CH][threads], at this thread
  Pack<T, V>* ring;
  int64_t put_row;
  int stage_packs, put_at, get_at;
  int array_at[ARRAYS];

  __device__ __forceinline__ int column(int i) const { return (i * threads + j) * V; }

  __device__ __forceinline__ void put() {
    if (put_row < last) {
#pragma unroll
      for (int a = 0; a < ARRAYS; ++a) {
        if (src[a] == nullptr) continue;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int c = column(i);
          if (c < H) cp_async16(ring + put_at + array_at[a] + i * threads, src[a] + put_row * ld[a] + c);
        }
      }
    }
    put_row += step;
    cp_async_commit();
    put_at = put_at + stage_packs == STAGES * stage_packs ? 0 : put_at + stage_packs;
  }

  __device__ __forceinline__ void start(int64_t first, int64_t step_, int64_t last_, void* smem) {
    step = step_;
    last = last_;
    row = first - step;
    if constexpr (STAGES > 0) {
      put_row = first;
      int present = 0;
#pragma unroll
      for (int a = 0; a < ARRAYS; ++a) {
        array_at[a] = present * CH * threads;
        present += src[a] != nullptr;
      }
      stage_packs = present * CH * threads;
      // (a warp's row has its own ring)
      ring = static_cast<Pack<T, V>*>(smem) + (threadIdx.x / threads) * (STAGES * stage_packs) + j;
      put_at = 0;
      get_at = -stage_packs;
#pragma unroll
      for (int s = 0; s < STAGES - 1; ++s) put();
    }
  }

  // Moves on to the next row.
  __device__ __forceinline__ void next() {
    row += step;
    if constexpr (STAGES > 0) {
      put();
      cp_async_wait<STAGES - 1>();
      get_at = get_at + stage_packs == STAGES * stage_packs ? 0 : get_at + stage_packs;
    }
  }

  // Pack i of an array that is present, of the row.
  __device__ __forceinline__ Pack<T, V> at(int a, int i) const {
    if constexpr (STAGES > 0) return ring[get_at + array_at[a] + i * threads];
    else return load_pack<V>(src[a] + row * ld[a] + column(i));
  }
};

// N sums over the threads of a row: a warp (WARP) or the whole block, with
// one barrier. A scratch s (32 floats a value, zero behind the last warp) may
// be written again once every thread has passed a later barrier: callers use
// one per sum of a row and alternate by row.
template <int N, bool WARP>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*s)[32]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (WARP) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i][warp] = v[i];
  }
  __syncthreads();
  const int quads = (blockDim.x + 127) >> 7;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < quads; ++q) {
      const float4 p = *reinterpret_cast<const float4*>(&s[i][4 * q]);
      t.x += p.x;
      t.y += p.y;
      t.z += p.z;
      t.w += p.w;
    }
    v[i] = (t.x + t.y) + (t.z + t.w);
  }
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

// Times the channel gate's activation.
template <typename T, int V>
__device__ __forceinline__ void times_channel_gate(const NormArgs& a, int c, float (&f)[V]) {
  float g[V];
  unpack(load_pack<V>(static_cast<const T*>(a.gate) + c), g);
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] *= gate_value(a.gate_act, g[i]);
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

// Shared memory of an SM that the blocks' rows in flight share.
constexpr int kQueueSmem = 220 * 1024;

}  // namespace bsmoe
