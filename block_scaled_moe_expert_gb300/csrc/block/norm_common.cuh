// Shared by the norms' forward and gradient kernels: the rows' way into
// registers, row sums, gates, weights of either type.
#pragma once
#include "../ptx.cuh"
#include "block_internal.cuh"

namespace bsmoe {

// An asynchronous copy of only the first `bytes` of 16 bytes (the rest become zero).
__device__ __forceinline__ void cp_async16_part(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

// Bytes of an array's stage for rows of any alignment: whole 16-byte chunks.
__host__ __device__ constexpr int loose_row_bytes(int H, int size) { return (H * size + 15 + 15) / 16 * 16; }

// Thread j of a row owns the packs j, j + threads, ... (CH of them) of every
// row that its block (or warp) walks, and with STAGES > 0 the next rows are on
// their way into shared memory while it works on one.
//   Packs (V > 1): each thread copies its own packs into its own slots, which
// nobody else reads, so there is no barrier in the queue.
//   Packs of shifted rows (SHIFT): rows of a width that is no multiple of a pack
// start anywhere in a 16-byte chunk, but contiguous rows of one width and type
// all start at the same place of theirs, and rows a multiple of 8 apart start
// alike. The packs are then the aligned chunks: `shift` elements of the first
// belong to the row in front, the last is cut at the row's end, and their
// values outside the row count as zero.
//   Rows of any width and alignment (V = 1): the block copies the aligned
// 16-byte chunks that hold the row, whatever they hold beside it (in front of
// the row that is memory of the same allocation, which starts at a multiple of
// 256 bytes; the last chunk is cut at the row's end), and the elements are read
// where they lie in them; one barrier a row.
//   STAGES = 0: rows that are too long for shared memory are read from global
// memory where they are used, a second time from the L1.
// THREADS: of a row, where the kernel is compiled for their number (an
// element's place is then a constant away from the thread's), else 0.
template <typename T, int V, int CH, int ARRAYS, int STAGES, int THREADS, bool SHIFT>
struct RowQueue {
  static constexpr bool kLoose = V == 1 && STAGES > 0;
  const T* src[ARRAYS];  // null: absent; else, once started, where the row to fetch starts (for this thread)
  int64_t ld[ARRAYS];    // once started, the way to the block's next row
  int H, j;
  int shift = 0;         // see SHIFT
  int put_left;          // rows still to fetch
  // STAGES > 0, in bytes: [STAGES][arrays present][a row]
  uint8_t* ring;
  int stage_bytes, put_at, get_at;
  int array_at[ARRAYS];
  int phase[ARRAYS], phase_step[ARRAYS];  // loose rows: where in its first chunk the row in work starts

  __device__ __forceinline__ int threads() const { return THREADS > 0 ? THREADS : static_cast<int>(blockDim.x); }
  // Pack i's place in the row's chunks, its first column, whether the row has it, whether it has all of it.
  __device__ __forceinline__ int place(int i) const { return (i * threads() + j) * V; }
  __device__ __forceinline__ int column(int i) const { return SHIFT ? place(i) - shift : place(i); }
  __device__ __forceinline__ bool in(int i) const { return column(i) < H; }
  __device__ __forceinline__ bool whole(int i) const { return !SHIFT || (column(i) >= 0 && column(i) + V <= H); }

  __device__ __forceinline__ void put() {
    if (put_left > 0) {
      --put_left;
#pragma unroll
      for (int a = 0; a < ARRAYS; ++a) {
        if (src[a] == nullptr) continue;
        uint8_t* dst = ring + put_at + array_at[a];
        if constexpr (kLoose) {
          const int skip = static_cast<int>(reinterpret_cast<uintptr_t>(src[a]) & 15);
          const uint8_t* p = reinterpret_cast<const uint8_t*>(src[a]) - skip;
          const int bytes = skip + H * static_cast<int>(sizeof(T));
          for (int at = j * 16; at < bytes; at += threads() * 16) cp_async16_part(dst + at, p + at, min(16, bytes - at));
        } else {
#pragma unroll
          for (int i = 0; i < CH; ++i)
            if (in(i)) {
              if constexpr (SHIFT)
                cp_async16_part(dst + i * threads() * 16, src[a] + i * threads() * V,
                                min(16, (H - column(i)) * static_cast<int>(sizeof(T))));
              else cp_async16(dst + i * threads() * 16, src[a] + i * threads() * V);
            }
        }
        src[a] += ld[a];
      }
    }
    cp_async_commit();
    put_at = put_at + stage_bytes == STAGES * stage_bytes ? 0 : put_at + stage_bytes;
  }

  // Where the rows first, first + step, ... of a contiguous array start in their first chunk.
  __device__ __forceinline__ void set_shift(const void* array, int64_t first) {
    if constexpr (SHIFT)
      shift = static_cast<int>((reinterpret_cast<uintptr_t>(array) + first * H * sizeof(T)) & 15) / static_cast<int>(sizeof(T));
  }

  // Rows first, first + step, ... (n of them).
  __device__ __forceinline__ void start(int64_t first, int64_t step, int n, void* smem) {
    put_left = n;
#pragma unroll
    for (int a = 0; a < ARRAYS; ++a) {
      if (src[a] != nullptr) src[a] += (STAGES > 0 ? first : first - step) * ld[a] + (kLoose ? 0 : j * V) - shift;
      ld[a] *= step;
    }
    if constexpr (STAGES > 0) {
      const int row_bytes = kLoose ? loose_row_bytes(H, sizeof(T)) : CH * threads() * 16;
      int present = 0;
#pragma unroll
      for (int a = 0; a < ARRAYS; ++a) {
        array_at[a] = present * row_bytes;
        present += src[a] != nullptr;
        if constexpr (kLoose) {
          phase_step[a] = static_cast<int>((ld[a] * static_cast<int64_t>(sizeof(T))) & 15);
          phase[a] = static_cast<int>(reinterpret_cast<uintptr_t>(src[a]) & 15) - phase_step[a];
        }
      }
      stage_bytes = present * row_bytes;
      // (a warp's row has its own ring)
      ring = static_cast<uint8_t*>(smem) + (threadIdx.x / threads()) * (STAGES * stage_bytes) + (kLoose ? 0 : j * 16);
      put_at = 0;
      get_at = -stage_bytes;
#pragma unroll
      for (int s = 0; s < STAGES - 1; ++s) put();
    }
  }

  // Moves on to the next row.
  __device__ __forceinline__ void next() {
    if constexpr (kLoose) {
      cp_async_wait<STAGES - 2>();
      __syncthreads();  // the row is here, and nobody reads the one before, whose place the next fetch takes
      put();
#pragma unroll
      for (int a = 0; a < ARRAYS; ++a) phase[a] = (phase[a] + phase_step[a]) & 15;
    } else if constexpr (STAGES > 0) {
      put();
      cp_async_wait<STAGES - 1>();
    } else {
#pragma unroll
      for (int a = 0; a < ARRAYS; ++a)
        if (src[a] != nullptr) src[a] += ld[a];
    }
    if constexpr (STAGES > 0) get_at = get_at + stage_bytes == STAGES * stage_bytes ? 0 : get_at + stage_bytes;
  }

  // Pack i of an array that is present, of the row.
  __device__ __forceinline__ Pack<T, V> at(int a, int i) const {
    if constexpr (kLoose)
      return *reinterpret_cast<const Pack<T, V>*>(ring + get_at + array_at[a] + phase[a] + column(i) * sizeof(T));
    else if constexpr (STAGES > 0) return *reinterpret_cast<const Pack<T, V>*>(ring + get_at + array_at[a] + i * threads() * 16);
    else return load_pack<V>(src[a] + i * threads() * V);
  }
};

// Shared memory of a queue's rows of one block.
template <typename T, int V, int CH, int STAGES>
size_t queue_smem(int H, int arrays, int threads) {
  if (STAGES == 0) return 0;
  return static_cast<size_t>(STAGES) * arrays * (V == 1 ? loose_row_bytes(H, sizeof(T)) : CH * threads * 16);
}

// N sums over the threads of a row: a warp (WARP) or the whole block, with
// one barrier. A scratch s may be written again once every thread has passed
// a later barrier: callers use one per sum of a row and alternate by row.
template <int N, bool WARP>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*s)[32]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (WARP) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i][warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = warp_sum(lane < warps ? s[i][lane] : 0.f);
  }
}

// P sums (1, 2, 4 or 8) over the threads of a row at the price of about two: in
// the first steps the lanes halve the values between them, so that a lane ends
// with one value's sum over its warp; one barrier. s: [P][16] floats of the
// block, zero behind its last warp, used again two rows on at the earliest (see
// row_sum).
template <int P, bool WARP>
__device__ __forceinline__ void row_sums(float (&v)[P], float* s) {
  const int lane = threadIdx.x & 31;
  constexpr int kLanes = 32 / P;  // that share a value
  int o = 16;
#pragma unroll
  for (int half = P / 2; half > 0; half /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float t = v[0];
#pragma unroll
  for (int x = kLanes / 2; x > 0; x /= 2) t += __shfl_xor_sync(0xffffffffu, t, x);
  if (!WARP) {
    if (lane % kLanes == 0) s[lane / kLanes * 16 + (threadIdx.x >> 5)] = t;
    __syncthreads();
    constexpr int kEach = P >= 2 ? 16 / kLanes > 0 ? 16 / kLanes : 1 : 1;
    t = 0.f;
    if (lane % kLanes < 16 / kEach) {
      const Pack<float, kEach> p = load_pack<kEach>(s + lane / kLanes * 16 + lane % kLanes * kEach);
#pragma unroll
      for (int i = 0; i < kEach; ++i) t += p.e[i];
    }
#pragma unroll
    for (int x = kLanes / 2; x > 0; x /= 2) t += __shfl_xor_sync(0xffffffffu, t, x);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) v[i] = __shfl_sync(0xffffffffu, t, i * kLanes);
}

// V fp32 values of a pack, in pairs where there are pairs.
template <int V>
struct Values {
  float v[V];
  __device__ __forceinline__ float2 pair(int i) const { return make_float2(v[i], v[i + 1]); }
  __device__ __forceinline__ void set(int i, float2 p) {
    v[i] = p.x;
    v[i + 1] = p.y;
  }
};
template <int V>
__device__ __forceinline__ Values<V> operator*(const Values<V>& a, const Values<V>& b) {
  Values<V> d;
  if constexpr (V == 1) {
    d.v[0] = a.v[0] * b.v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) d.set(i, mul2(a.pair(i), b.pair(i)));
  }
  return d;
}
template <int V>
__device__ __forceinline__ Values<V> operator*(const Values<V>& a, float s) {
  Values<V> b;
#pragma unroll
  for (int i = 0; i < V; ++i) b.v[i] = s;
  return a * b;
}
template <int V>
__device__ __forceinline__ Values<V> fma(const Values<V>& a, const Values<V>& b, const Values<V>& c) {
  Values<V> d;
  if constexpr (V == 1) {
    d.v[0] = fmaf(a.v[0], b.v[0], c.v[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) d.set(i, fma2(a.pair(i), b.pair(i), c.pair(i)));
  }
  return d;
}
template <int V>
__device__ __forceinline__ Values<V> fma(const Values<V>& a, float s, const Values<V>& c) {
  Values<V> b;
#pragma unroll
  for (int i = 0; i < V; ++i) b.v[i] = s;
  return fma(a, b, c);
}
// A sum of products as two strands.
template <int V>
__device__ __forceinline__ void add_dot(float2& sum, const Values<V>& a, const Values<V>& b) {
  if constexpr (V == 1) {
    sum.x = fmaf(a.v[0], b.v[0], sum.x);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) sum = fma2(a.pair(i), b.pair(i), sum);
  }
}
template <int V>
__device__ __forceinline__ Values<V> zeros() {
  Values<V> z;
#pragma unroll
  for (int i = 0; i < V; ++i) z.v[i] = 0.f;
  return z;
}
template <typename T, int V>
__device__ __forceinline__ Values<V> values(const Pack<T, V>& p) {
  Values<V> f;
  unpack(p, f.v);
  return f;
}

__device__ __forceinline__ float gate_value(int act, float v) {
  if (act == MOE_GATE_SIGMOID) return 1.f / (1.f + expf(-v));
  if (act == MOE_GATE_TANH) return tanhf(v);
  return v;
}
// Values of a pack that the row has, zero outside it.
template <typename Q>
__device__ __forceinline__ auto row_values(const Q& rows, int a, int i) {
  auto f = values(rows.at(a, i));
  if (!rows.whole(i)) {
#pragma unroll
    for (int e = 0; e < static_cast<int>(sizeof(f.v) / sizeof(float)); ++e)
      f.v[e] = rows.column(i) + e >= 0 && rows.column(i) + e < rows.H ? f.v[e] : 0.f;
  }
  return f;
}
// Stores what the row has of pack i; out: this thread's first pack.
template <typename Q, typename T, int V>
__device__ __forceinline__ void store_values(const Q& rows, T* out, int i, const Values<V>& f) {
  out += i * rows.threads() * V;
  if (rows.whole(i)) {
    store_pack(out, pack<T, V>(f.v));
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (rows.column(i) + e >= 0 && rows.column(i) + e < rows.H) out[e] = from_f32<T>(f.v[e]);
  }
}

// w_offset + weight (1 without a weight) of columns c..c+V-1.
template <typename T, int V>
__device__ __forceinline__ Values<V> load_weight(const void* w, int w_f32, float offset, int c) {
  Values<V> f;
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) f.v[i] = 1.f;
  } else if (w_f32 && sizeof(T) != 4) {
    constexpr int V4 = V < 4 ? V : 4;
#pragma unroll
    for (int i = 0; i < V; i += V4) {
      const Pack<float, V4> p = load_pack<V4>(static_cast<const float*>(w) + c + i);
#pragma unroll
      for (int j = 0; j < V4; ++j) f.v[i + j] = p.e[j] + offset;
    }
  } else {
    f = values(load_pack<V>(static_cast<const T*>(w) + c));
#pragma unroll
    for (int i = 0; i < V; ++i) f.v[i] += offset;
  }
  return f;
}

// The gate's activation, V values of it.
template <int V>
__device__ __forceinline__ Values<V> gate_values(int act, Values<V> g) {
  if (act != MOE_GATE_LINEAR) {
#pragma unroll
    for (int i = 0; i < V; ++i) g.v[i] = gate_value(act, g.v[i]);
  }
  return g;
}
// And its slope. 1 - g and 1 - g^2 have no bits left where the activation g has
// come near 1 (sigmoid: 6 % off at 16, 0 from 17), so the slopes come from an
// exponential: e / (1 + e)^2 with e = e^-|v|, and e (1 + |g|)^2 with e = e^(-2 |v|).
template <int V>
struct Gate {
  Values<V> value, slope;
};
template <int V>
__device__ __forceinline__ Gate<V> gate_with_slope(int act, const Values<V>& v) {
  Gate<V> g;
  if (act == MOE_GATE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float e = expf(-fabsf(v.v[i])), d = 1.f / (1.f + e);
      g.value.v[i] = v.v[i] < 0.f ? e * d : d;
      g.slope.v[i] = e * d * d;
    }
  } else if (act == MOE_GATE_TANH) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float t = tanhf(v.v[i]), s = 1.f + fabsf(t);
      g.value.v[i] = t;
      g.slope.v[i] = expf(-2.f * fabsf(v.v[i])) * (s * s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      g.value.v[i] = v.v[i];
      g.slope.v[i] = 1.f;
    }
  }
  return g;
}
__device__ __forceinline__ Gate<1> gate_with_slope(int act, float v) {
  Values<1> one;
  one.v[0] = v;
  return gate_with_slope(act, one);
}
template <typename T, int V>
__device__ __forceinline__ Values<V> channel_gate(const NormArgs& a, int c) {
  return gate_values(a.gate_act, values(load_pack<V>(static_cast<const T*>(a.gate) + c)));
}

// A factor of the columns of a pack: V at a time, or one by one where the
// pack may reach beyond the row (zero there).
template <bool SHIFT, int V, typename Wide, typename One>
__device__ __forceinline__ Values<V> column_factor(int c, int H, const Wide& wide, const One& one) {
  if constexpr (!SHIFT) {
    return wide(c);
  } else {
    Values<V> f;
#pragma unroll
    for (int e = 0; e < V; ++e) f.v[e] = c + e >= 0 && c + e < H ? one(c + e) : 0.f;
    return f;
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

// The operands [T, H] start at the same place of a 16-byte chunk in every row
// (see SHIFT; null pointers pass, and the width for an absent one's stride).
template <typename T>
bool rows_shift_alike(int n, int H, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
  int phase = -1;
  for (const void* p : ptrs) {
    if (p == nullptr) continue;
    const int at = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    if (phase >= 0 && at != phase) return false;
    phase = at;
  }
  for (const int64_t l : lds)
    if (n > 1 && ((l - H) * static_cast<int64_t>(sizeof(T))) % 16) return false;
  return true;
}

// Blocks that walk more than one row each take rows a multiple of 8 apart.
inline int shifted_grid(int grid, int rows) { return grid < rows ? std::min(rows, std::max(8, grid / 8 * 8)) : grid; }

// Shared memory of an SM that the blocks' rows in flight share.
constexpr int kQueueSmem = 220 * 1024;

}  // namespace bsmoe
