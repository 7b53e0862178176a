// Norms before and after a block:
//   N(v; w) = v rsqrt(mean(v^2) + eps) (w + offset)
//   norm_before: y = N(x; w)
//   norm_after:  r = beta x + alpha g z, z = N(h; w) or h, g = act(gate),
//                and y = N(r; w_next) for the next block.
//
// One pass: a row lives in registers between its sums, so x and h are read
// once, r and y written once, and the sum over r^2 needs no second look at r.
// Bound by DRAM bandwidth (by latency for a few tokens). A block walks many
// rows with the next ones on their way (RowQueue), and keeps its columns'
// factors alpha w g and w_next in registers. Sums in fp32 by a fixed tree.
#include "norm_common.cuh"

namespace bsmoe {

namespace {

enum { kX = 0, kH = 1, kGate = 2 };

// One row per warp (WARP) or per block.
template <typename T, int V, int CH, int STAGES, bool AFTER, bool NEXT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : 1024) norm_kernel(NormArgs a) {
  constexpr int ARRAYS = AFTER ? 3 : 1;
  constexpr bool CACHED = CH * V <= 8;  // the columns' factors stay in registers
  extern __shared__ __align__(16) uint8_t s_ring[];
  __shared__ __align__(16) float s_sum[2][2][1][32];  // by the row's parity: a row's sums do not wait for the row before
  RowQueue<T, V, CH, ARRAYS, STAGES> rows;
  rows.H = a.H;
  rows.threads = WARP ? 32 : blockDim.x;
  rows.j = WARP ? threadIdx.x & 31 : threadIdx.x;
  rows.src[kX] = static_cast<const T*>(a.x);
  rows.ld[kX] = a.ld_x;
  if constexpr (AFTER) {
    rows.src[kH] = static_cast<const T*>(a.h);
    rows.ld[kH] = a.ld_h;
    rows.src[kGate] = a.gate_kind == MOE_GATE_ELEMENT ? static_cast<const T*>(a.gate) : nullptr;
    rows.ld[kGate] = a.ld_gate;
  }
  if (!WARP)
    for (int i = threadIdx.x; i < 128; i += blockDim.x) (&s_sum[0][0][0][0])[i] = 0.f;
  pdl_wait();
  pdl_launch_dependents();
  const int per_block = WARP ? blockDim.x / 32 : 1;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * per_block + (WARP ? threadIdx.x >> 5 : 0);
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
  rows.start(first, step, a.T, s_ring);

  auto factor = [&](int c, float (&f)[V]) {  // alpha w g of the columns
    load_weight<T, V>(a.norm ? a.weight : nullptr, a.weight_f32, a.w_offset, c, f);
    if (a.gate_kind == MOE_GATE_CHANNEL) times_channel_gate<T, V>(a, c, f);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] *= a.alpha;
  };
  float wa[CH][V], wn[CH][V];
  if (CACHED) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = rows.column(i);
      if (c >= a.H) continue;
      if (AFTER) factor(c, wa[i]);
      if (NEXT) load_weight<T, V>(a.next_weight, a.weight_f32, a.w_offset, c, wn[i]);
    }
  }
  const float inv_h = 1.f / static_cast<float>(a.H);
  if (!WARP) __syncthreads();  // s_sum is zero
  int parity = 0;
  for (int64_t t = first; t < a.T; t += step, parity ^= 1) {
    rows.next();
    float r[CH][V];
    if constexpr (AFTER) {
      float scale = 1.f;
      if (a.norm) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if (rows.column(i) >= a.H) continue;
          float hf[V];
          unpack(rows.at(kH, i), hf);
#pragma unroll
          for (int e = 0; e < V; ++e) ss[0] = fmaf(hf[e], hf[e], ss[0]);
        }
        row_sum<1, WARP>(ss, s_sum[parity][0]);
        scale = rsqrtf(ss[0] * inv_h + a.eps);
      }
      if (a.gate_kind == MOE_GATE_TOKEN)
        scale *= gate_value(a.gate_act, to_f32(static_cast<const T*>(a.gate)[t * a.ld_gate]));
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = rows.column(i);
        if (c >= a.H) continue;
        if (!CACHED) factor(c, wa[i]);
        float hf[V], xf[V];
        unpack(rows.at(kH, i), hf);
        unpack(rows.at(kX, i), xf);
        if (a.gate_kind == MOE_GATE_ELEMENT) {
          float g[V];
          unpack(rows.at(kGate, i), g);
#pragma unroll
          for (int e = 0; e < V; ++e) hf[e] *= gate_value(a.gate_act, g[e]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) r[i][e] = fmaf(hf[e] * scale, wa[i][e], a.beta * xf[e]);
        store_pack(static_cast<T*>(a.r) + t * a.H + c, pack<T, V>(r[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i) unpack(rows.at(kX, i), r[i]);
    }
    if constexpr (NEXT) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (rows.column(i) >= a.H) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) ss[0] = fmaf(r[i][e], r[i][e], ss[0]);
      }
      row_sum<1, WARP>(ss, s_sum[parity][1]);
      const float scale = rsqrtf(ss[0] * inv_h + a.next_eps);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = rows.column(i);
        if (c >= a.H) continue;
        if (!CACHED) load_weight<T, V>(a.next_weight, a.weight_f32, a.w_offset, c, wn[i]);
        float y[V];
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = r[i][e] * scale * wn[i][e];
        store_pack(static_cast<T*>(a.y) + t * a.H + c, pack<T, V>(y));
      }
    }
  }
}

template <typename T, int V, int CH, int STAGES, bool WARP>
cudaError_t run(const NormArgs& a, int threads, int num_sms, cudaStream_t st) {
  auto* k = a.h == nullptr ? norm_kernel<T, V, CH, STAGES, false, true, WARP>
            : a.next       ? norm_kernel<T, V, CH, STAGES, true, true, WARP>
                           : norm_kernel<T, V, CH, STAGES, true, false, WARP>;
  const int arrays = a.h == nullptr ? 1 : a.gate_kind == MOE_GATE_ELEMENT ? 3 : 2;
  const size_t smem = static_cast<size_t>(STAGES) * arrays * CH * threads * sizeof(Pack<T, V>);
  // 1024 threads an SM (64 registers each), fewer blocks where their rows in
  // flight would not fit
  int blocks = std::max(1, 1024 / threads);
  if (smem > 0) blocks = std::max(1, std::min<int>(blocks, kQueueSmem / smem));
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int grid = std::min(ceil_div(a.T, WARP ? threads / 32 : 1), blocks * num_sms);
  return launch_kernel(true, k, grid, threads, smem, st, a);
}

}  // namespace

cudaError_t launch_norm(int dtype, const NormArgs& a, int num_sms, cudaStream_t st) {
  return with_dtype(dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    const bool vec = rows_vectorize<T>(
        a.H, {a.x, a.h, a.weight, a.next_weight, a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate, a.r, a.y},
        {a.ld_x, a.ld_h, a.gate_kind == MOE_GATE_ELEMENT ? a.ld_gate : 0});
    constexpr int V = kVec<T>;
    const int packs = vec ? a.H / V : a.H;
    auto threads = [&](int ch) { return ceil_div(ceil_div(packs, ch), 32) * 32; };
    if (!vec) {
      if (packs <= 4096) return run<T, 1, 4, 0, false>(a, threads(4), num_sms, st);
      if (packs <= 8192) return run<T, 1, 8, 0, false>(a, threads(8), num_sms, st);
      return run<T, 1, 16, 0, false>(a, threads(16), num_sms, st);
    }
    if (packs <= 32) return run<T, V, 1, 4, true>(a, 128, num_sms, st);
    if (packs <= 64) return run<T, V, 2, 4, true>(a, 128, num_sms, st);
    // as many stages as three arrays' rows fit into shared memory
    if (packs <= 1024) return run<T, V, 1, 4, false>(a, threads(1), num_sms, st);
    if (packs <= 2048) return run<T, V, 2, 2, false>(a, threads(2), num_sms, st);
    if constexpr (sizeof(T) == 4) return run<T, V, 4, 0, false>(a, threads(4), num_sms, st);
    return cudaErrorInvalidValue;  // 16-bit rows have at most 2048 packs
  });
}

}  // namespace bsmoe
