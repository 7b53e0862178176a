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
//
// Measured (bf16, of 6.8 TB/s for a plain copy): place, 8192 tokens of 7168
// columns, K = 8, into 128-row groups 230 us, 6.6 TB/s (nearly all of it
// writes); gather with weights, 8192 of 2880, K = 4 40 us, 5.8 TB/s; place with
// dots, 4096 of 4096, K = 2 27 us, 6.2 TB/s; gather with dots of unaligned fp32
// rows, 3001 of 1001, K = 5 23 us, 3.4 TB/s: there each lane's loads are 4 bytes
// and the 64 registers hold 16 of them. Registers are held to four blocks an
// SM: with more packs in flight a lane and fewer warps the gather of 2880
// columns took 59 us, with six blocks (and spills) 108.
#include "block_internal.cuh"
#include "../ptx.cuh"

namespace bsmoe {

namespace {

constexpr int kPermThreads = 256;
constexpr int kPermWarps = kPermThreads / 32;
constexpr int kPermBlocks = 4;  // blocks per SM that the registers are held to
// Packs of rows that a lane has in flight.
template <int V>
constexpr int kPacks = V == 1 ? 16 : 4;

// A block holds kPermWarps / wpt tokens; the wpt warps of a token take turns
// along its columns. A lane has KB experts of the token by U
// packs of columns in flight.
struct Where {
  int64_t t;
  int warp_in_token, token_in_block;
};
__device__ __forceinline__ Where locate(int wpt) {
  const int warp = threadIdx.x >> 5;
  return {static_cast<int64_t>(blockIdx.x) * (kPermWarps / wpt) + warp / wpt, warp % wpt, warp / wpt};
}

// The row of slot (t, lane), -1 where it has none. A plan that does not belong
// to the call moves nothing out of the rows' range.
__device__ __forceinline__ int slot_row(const SortPlan& p, int64_t t, int lane) {
  const int row = p.inv[t * p.K + lane];
  return static_cast<unsigned>(row) < static_cast<unsigned>(p.M) ? row : -1;
}

// Sums the dots of KT rows over the warps of a token and stores them.
template <int KT>
__device__ __forceinline__ void store_dots(float (&dot)[KT], const Where& at, int wpt, bool live, float* dots, int K,
                                           int k0, float (*s)[KT]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < KT; ++j) dot[j] = warp_sum(dot[j]);
  if (wpt > 1) {
    __syncthreads();
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < KT; ++j) s[warp][j] = dot[j];
    }
    __syncthreads();
    if (at.warp_in_token == 0) {
#pragma unroll
      for (int j = 0; j < KT; ++j)
        for (int w = 1; w < wpt; ++w) dot[j] += s[warp + w][j];
    }
  }
  if (live && at.warp_in_token == 0) {
    float mine = 0.f;
#pragma unroll
    for (int j = 0; j < KT; ++j) mine = lane == j ? dot[j] : mine;
    if (lane < KT && k0 + lane < K) dots[at.t * K + k0 + lane] = mine;
  }
}

// rows null: the dots alone. grid ceil(T / tokens a block) + zero blocks: the
// last blocks zero the rows that belong to no slot, 32 rows a warp.
template <typename T, int V, int KB, int U, bool W, bool DOTS>
__global__ void __launch_bounds__(kPermThreads, kPermBlocks) place_kernel(PlaceArgs a, int wpt, int token_blocks) {
  __shared__ float s_dot[kPermWarps][KB];
  pdl_wait();
  pdl_launch_dependents();
  const int H = a.H, K = a.p.K, lane = threadIdx.x & 31;
  T* rows = static_cast<T*>(a.rows);
  if (static_cast<int>(blockIdx.x) >= token_blocks) {
    const int r0 = (static_cast<int>(blockIdx.x) - token_blocks) * kPermWarps * 4 + (threadIdx.x >> 5) * 4;
    Pack<T, V> z;
#pragma unroll
    for (int i = 0; i < V; ++i) z.e[i] = from_f32<T>(0.f);
    for (int r = r0; r < min(r0 + 4, a.p.M); ++r) {
      if (a.p.row_slot[r] >= 0) continue;
      T* dst = rows + static_cast<size_t>(r) * H;
      for (int c = lane * V; c < H; c += 32 * V) store_pack(dst + c, z);
    }
    return;
  }
  const Where at = locate(wpt);
  const bool live = at.t < a.p.T;
  int my_row = -1;
  float my_w = 0.f;
  if (live && lane < K) {
    my_row = slot_row(a.p, at.t, lane);
    if (W) my_w = a.w[at.t * K + lane];
  }
  const T* x = static_cast<const T*>(a.x) + at.t * a.ld_x;
  const T* other = static_cast<const T*>(a.other);
  for (int k0 = 0; k0 < K; k0 += KB) {
    int row[KB];
    float w[KB], dot[KB] = {};
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      row[j] = __shfl_sync(0xffffffffu, my_row, k0 + j);
      if (k0 + j >= K) row[j] = -1;
      w[j] = W ? __shfl_sync(0xffffffffu, my_w, k0 + j) : 1.f;
    }
    const int first = (at.warp_in_token * 32 * U + lane) * V, step = wpt * 32 * U * V;
    for (int c = live ? first : H; c < H; c += step) {
      Pack<T, V> xp[U], op[U][KB];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int cu = c + u * 32 * V;
        if (cu >= H) continue;
        xp[u] = load_pack<V>(x + cu);
        if (DOTS) {
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (row[j] >= 0) op[u][j] = load_pack<V>(other + static_cast<int64_t>(row[j]) * a.ld_other + cu);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int cu = c + u * 32 * V;
        if (cu >= H) continue;
        float xf[V];
        if (W || DOTS) unpack(xp[u], xf);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          if (row[j] < 0) continue;
          if (!DOTS || rows != nullptr) {
            T* dst = rows + static_cast<int64_t>(row[j]) * H + cu;
            if (W) {
              float o[V];
#pragma unroll
              for (int i = 0; i < V; ++i) o[i] = w[j] * xf[i];
              store_pack(dst, pack<T, V>(o));
            } else {
              store_pack(dst, xp[u]);
            }
          }
          if (DOTS) {
            float of[V];
            unpack(op[u][j], of);
#pragma unroll
            for (int i = 0; i < V; ++i) dot[j] = fmaf(xf[i], of[i], dot[j]);
          }
        }
      }
    }
    if (DOTS) store_dots<KB>(dot, at, wpt, live, a.dots, K, k0, s_dot);
  }
}

// With DOTS, K <= KT (the dots ride along with the one pass over the rows);
// without, KT = KB and any K.
template <typename T, int V, int KT, int KB, int U, bool W, bool DOTS>
__global__ void __launch_bounds__(kPermThreads, kPermBlocks) gather_kernel(GatherArgs a, int wpt) {
  __shared__ float s_dot[kPermWarps][KT];
  pdl_wait();
  pdl_launch_dependents();
  const int H = a.H, K = a.p.K, lane = threadIdx.x & 31;
  const Where at = locate(wpt);
  const bool live = at.t < a.p.T;
  int my_row = -1;
  float my_w = 0.f;
  if (live && lane < K) {
    my_row = slot_row(a.p, at.t, lane);
    if (W) my_w = a.w[at.t * K + lane];
  }
  const T* rows = static_cast<const T*>(a.rows);
  const T* x = static_cast<const T*>(a.x) + at.t * a.ld_x;
  T* out = static_cast<T*>(a.out) + at.t * H;
  float dot[KT] = {};
  const int first = at.warp_in_token * 32 * U * V, step = wpt * 32 * U * V;
  // (all lanes of a warp take the same number of steps: the shuffles need them)
  for (int c0 = live ? first : H; c0 < H; c0 += step) {
    const int c = c0 + lane * V;
    float acc[U][V] = {}, xf[U][V];
    auto add = [&](int k0, float* d) {  // KB experts from k0 on
      int row[KB];
      float w[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        row[j] = __shfl_sync(0xffffffffu, my_row, k0 + j);
        if (k0 + j >= K) row[j] = -1;
        w[j] = W ? __shfl_sync(0xffffffffu, my_w, k0 + j) : 1.f;
      }
      Pack<T, V> rp[U][KB];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int cu = c + u * 32 * V;
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (row[j] >= 0 && cu < H) rp[u][j] = load_pack<V>(rows + static_cast<int64_t>(row[j]) * a.ld_rows + cu);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c + u * 32 * V >= H) continue;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          if (row[j] < 0) continue;
          float rf[V];
          unpack(rp[u][j], rf);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            acc[u][i] = W ? fmaf(w[j], rf[i], acc[u][i]) : acc[u][i] + rf[i];
            if (DOTS) d[j] = fmaf(xf[u][i], rf[i], d[j]);
          }
        }
      }
    };
    if constexpr (DOTS) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c + u * 32 * V < H) unpack(load_pack<V>(x + c + u * 32 * V), xf[u]);
#pragma unroll
      for (int k0 = 0; k0 < KT; k0 += KB)
        if (k0 < K) add(k0, dot + k0);
    } else {
      for (int k0 = 0; k0 < K; k0 += KB) add(k0, nullptr);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int cu = c + u * 32 * V;
      if (cu < H) store_pack(out + cu, pack<T, V>(acc[u]));
    }
  }
  if (DOTS) store_dots<KT>(dot, at, wpt, live, a.dots, K, 0, s_dot);
}

// Warps per token: one where the tokens alone give every SM a few rounds of
// warps, more (up to a block) for fewer tokens, as far as the row has work for
// them. The dots' join over a token's warps costs more than a shorter tail
// gives, so with dots one round is enough. Measured, one round against four:
// 4096 tokens of 4096 bf16 columns, K = 2, gradient of unpermute 26.5 us against
// 32.1, of permute 24.9 against 28.6; without dots 8192 of 7168, K = 8, permute
// 190 against 170. (It is not so for all: 4096 of 4096, K = 2, without dots 15.1
// against 17.9, and 8192 of 7168, K = 8, gradient of unpermute 330 against 309.)
int warps_per_token(int T, int H, int V, bool dots) {
  const int64_t enough = 152 * (dots ? 32 : 128);
  int wpt = 1;
  while (wpt < kPermWarps && static_cast<int64_t>(T) * wpt < enough && H > wpt * 32 * V) wpt *= 2;
  return wpt;
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

template <typename T, int V, int KB, int U, bool W, bool DOTS>
cudaError_t place(const PlaceArgs& a, cudaStream_t st) {
  const int wpt = warps_per_token(a.p.T, a.H, V, DOTS);
  const int token_blocks = ceil_div(a.p.T, kPermWarps / wpt);
  const int zero_blocks = a.rows != nullptr ? ceil_div(a.p.M, kPermWarps * 4) : 0;
  return launch_kernel(true, place_kernel<T, V, KB, U, W, DOTS>, token_blocks + zero_blocks, kPermThreads, 0, st, a,
                       wpt, token_blocks);
}

template <typename T, int V, int KT>
cudaError_t gather(const GatherArgs& a, cudaStream_t st) {
  constexpr int KB = KT < 4 ? KT : 4, U = kPacks<V> / KB;
  const int wpt = warps_per_token(a.p.T, a.H, V, a.dots != nullptr);
  auto* k = a.w == nullptr        ? gather_kernel<T, V, KB, KB, U, false, false>
            : a.dots != nullptr ? gather_kernel<T, V, KT, KB, U, true, true>
                                : gather_kernel<T, V, KB, KB, U, true, false>;
  return launch_kernel(true, k, ceil_div(a.p.T, kPermWarps / wpt), kPermThreads, 0, st, a, wpt);
}

// Without dots only the token's own row is loaded: all its experts at a time.
template <typename T, int V>
cudaError_t place_k(const PlaceArgs& a, cudaStream_t st) {
  if (a.dots != nullptr)
    return a.p.K <= 2 ? place<T, V, 2, kPacks<V> / 2, true, true>(a, st)
                      : place<T, V, 4, kPacks<V> / 4, true, true>(a, st);
  if (a.w != nullptr) return place<T, V, 8, kPacks<V>, true, false>(a, st);
  return place<T, V, 8, kPacks<V>, false, false>(a, st);
}

template <typename T, int V>
cudaError_t gather_k(const GatherArgs& a, cudaStream_t st) {
  if (a.dots != nullptr && a.p.K > 8) {
    // the sums and the dots of many experts do not fit one pass's registers
    GatherArgs sums = a;
    sums.dots = nullptr;
    const cudaError_t e = gather<T, V, 4>(sums, st);
    if (e != cudaSuccess) return e;
    return place_k<T, V>({a.x, a.ld_x, a.rows, a.ld_rows, a.w, nullptr, a.dots, a.H, a.p}, st);
  }
  if (a.p.K <= 2) return gather<T, V, 2>(a, st);
  if (a.p.K <= 4 || a.dots == nullptr) return gather<T, V, 4>(a, st);
  return gather<T, V, 8>(a, st);
}

}  // namespace

cudaError_t launch_place(int dtype, const PlaceArgs& a, cudaStream_t st) {
  return with_dtype(dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    return vec_ok<T>(a.H, {a.x, a.other, a.rows}, {a.ld_x, a.ld_other}) ? place_k<T, kVec<T>>(a, st)
                                                                        : place_k<T, 1>(a, st);
  });
}

cudaError_t launch_gather(int dtype, const GatherArgs& a, cudaStream_t st) {
  return with_dtype(dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    return vec_ok<T>(a.H, {a.rows, a.x, a.out}, {a.ld_rows, a.ld_x}) ? gather_k<T, kVec<T>>(a, st)
                                                                     : gather_k<T, 1>(a, st);
  });
}

}  // namespace bsmoe
