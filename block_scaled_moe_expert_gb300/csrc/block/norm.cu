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
//
// Measured (bf16): norm_after with channel gate and next norm, 8192 rows of
// 7168 columns, 75 us, 6.3 TB/s, 92% of a plain copy's rate; of 2001 columns 28
// us, 4.7 TB/s. One thread a pack (896 a row) and one block an SM: with two
// packs a thread the factors do not fit into the registers and the same rows
// took 200 us. Instructions count: packed fp32 pairs and one conversion
// instruction a pair took 110 us to 80.
#include "norm_common.cuh"

namespace bsmoe {

namespace {

enum { kX = 0, kH = 1, kGate = 2 };

// One row per warp (WARP) or per block. ELEMENT: a gate
// by element.
template <typename T, int V, int CH, int STAGES, int THREADS, bool AFTER, bool NEXT, bool ELEMENT, bool WARP, bool SHIFT>
__global__ void __launch_bounds__(WARP ? 128 : THREADS > 0 ? THREADS : CH * V <= 16 ? 1024 : 512,
                  WARP ? 8 : THREADS > 0 && CH <= 16 ? 1024 / (THREADS + !THREADS) : 1)
    norm_kernel(NormArgs a) {
  constexpr int ARRAYS = AFTER ? ELEMENT ? 3 : 2 : 1;
  // the columns' factors stay in registers, or for many columns of loose rows
  // (each a branch on the weights' type to load) in shared memory behind the
  // ring, each thread its own
  constexpr bool CACHED = CH * V <= 8, SHARED = !CACHED && V == 1 && STAGES > 0;
  extern __shared__ __align__(16) uint8_t s_ring[];
  __shared__ float s_sum[2][2][1][32];  // by the row's parity: a row's sums do not wait for the row before
  RowQueue<T, V, CH, ARRAYS, STAGES, WARP ? 32 : THREADS, SHIFT> rows;
  rows.H = a.H;
  rows.j = WARP ? threadIdx.x & 31 : threadIdx.x;
  rows.src[kX] = static_cast<const T*>(a.x);
  rows.ld[kX] = a.ld_x;
  if constexpr (AFTER) {
    rows.src[kH] = static_cast<const T*>(a.h);
    rows.ld[kH] = a.ld_h;
    if constexpr (ELEMENT) {
      rows.src[kGate] = static_cast<const T*>(a.gate);
      rows.ld[kGate] = a.ld_gate;
    }
  }
  pdl_wait();
  pdl_launch_dependents();
  const int per_block = WARP ? blockDim.x / 32 : 1;
  const int first = blockIdx.x * per_block + (WARP ? threadIdx.x >> 5 : 0), step = gridDim.x * per_block;
  const int n = first < a.T ? (a.T - 1 - first) / step + 1 : 0;
  rows.set_shift(AFTER ? a.r : a.y, first);
  rows.start(first, step, n, s_ring);

  auto factor = [&](int c) {  // alpha w g of the columns
    return column_factor<SHIFT, V>(
        c, a.H,
        [&](int at) {
          Values<V> f = load_weight<T, V>(a.norm ? a.weight : nullptr, a.weight_f32, a.w_offset, at);
          if (a.gate_kind == MOE_GATE_CHANNEL) f = f * channel_gate<T, V>(a, at);
          return f * a.alpha;
        },
        [&](int at) {
          const float w = load_weight<T, 1>(a.norm ? a.weight : nullptr, a.weight_f32, a.w_offset, at).v[0];
          return a.alpha * (a.gate_kind == MOE_GATE_CHANNEL ? w * channel_gate<T, 1>(a, at).v[0] : w);
        });
  };
  auto next_factor = [&](int c) {
    return column_factor<SHIFT, V>(
        c, a.H, [&](int at) { return load_weight<T, V>(a.next_weight, a.weight_f32, a.w_offset, at); },
        [&](int at) { return load_weight<T, 1>(a.next_weight, a.weight_f32, a.w_offset, at).v[0]; });
  };
  Values<V> wa[CACHED ? CH : 1], wn[CACHED ? CH : 1];
  Values<V>* s_factor = reinterpret_cast<Values<V>*>(s_ring + (SHARED ? STAGES * rows.stage_bytes : 0)) + rows.j;
  if (CACHED || SHARED) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = rows.column(i);
      if (!rows.in(i)) continue;
      if constexpr (CACHED) {
        if (AFTER) wa[i] = factor(c);
        if (NEXT) wn[i] = next_factor(c);
      } else {
        if (AFTER) s_factor[i * rows.threads()] = factor(c);
        if (NEXT) s_factor[(CH + i) * rows.threads()] = next_factor(c);
      }
    }
  }
  auto factor_of = [&](int i, int c) {
    if constexpr (CACHED) return wa[i];
    else if constexpr (SHARED) return s_factor[i * rows.threads()];
    else return factor(c);
  };
  auto next_factor_of = [&](int i, int c) {
    if constexpr (CACHED) return wn[i];
    else if constexpr (SHARED) return s_factor[(CH + i) * rows.threads()];
    else return next_factor(c);
  };
  const float inv_h = 1.f / static_cast<float>(a.H);
  const int64_t out_step = static_cast<int64_t>(step) * a.H;
  T* r_out = static_cast<T*>(a.r) + static_cast<int64_t>(first) * a.H + rows.j * V - rows.shift;
  T* y_out = static_cast<T*>(a.y) + static_cast<int64_t>(first) * a.H + rows.j * V - rows.shift;
  const T* token_gate = static_cast<const T*>(a.gate) + first * a.ld_gate;
  for (int k = 0; k < n; ++k, r_out += out_step, y_out += out_step) {
    rows.next();
    Values<V> r[CH];
    if constexpr (AFTER) {
      float scale = 1.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) r[i] = rows.in(i) ? row_values(rows, kH, i) : zeros<V>();
      if (a.norm) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < CH; ++i) add_dot(ss, r[i], r[i]);
        float sum[1] = {ss.x + ss.y};
        row_sum<1, WARP>(sum, s_sum[k & 1][0]);
        scale = rsqrtf(sum[0] * inv_h + a.eps);
      }
      if (a.gate_kind == MOE_GATE_TOKEN) {
        scale *= gate_value(a.gate_act, to_f32(*token_gate));
        token_gate += step * a.ld_gate;
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = rows.column(i);
        if (!rows.in(i)) continue;
        Values<V> x = row_values(rows, kX, i);
        if (a.beta != 1.f) x = x * a.beta;
        if constexpr (ELEMENT) r[i] = r[i] * gate_values(a.gate_act, row_values(rows, kGate, i));
        r[i] = fma(r[i] * scale, factor_of(i, c), x);
        store_values(rows, r_out, i, r[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i) r[i] = rows.in(i) ? row_values(rows, kX, i) : zeros<V>();
    }
    if constexpr (NEXT) {
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < CH; ++i) add_dot(ss, r[i], r[i]);
      float sum[1] = {ss.x + ss.y};
      row_sum<1, WARP>(sum, s_sum[k & 1][1]);
      const float scale = rsqrtf(sum[0] * inv_h + a.next_eps);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = rows.column(i);
        if (!rows.in(i)) continue;
        store_values(rows, y_out, i, r[i] * scale * next_factor_of(i, c));
      }
    }
  }
}

template <typename T, int V, int CH, int STAGES, bool WARP, int THREADS = 0, bool SHIFT = false>
cudaError_t run(const NormArgs& a, int threads, int num_sms, cudaStream_t st) {
  const bool element = a.gate_kind == MOE_GATE_ELEMENT;
  auto* k = a.h == nullptr ? norm_kernel<T, V, CH, STAGES, THREADS, false, true, false, WARP, SHIFT>
            : a.next       ? (element ? norm_kernel<T, V, CH, STAGES, THREADS, true, true, true, WARP, SHIFT>
                                      : norm_kernel<T, V, CH, STAGES, THREADS, true, true, false, WARP, SHIFT>)
                           : (element ? norm_kernel<T, V, CH, STAGES, THREADS, true, false, true, WARP, SHIFT>
                                      : norm_kernel<T, V, CH, STAGES, THREADS, true, false, false, WARP, SHIFT>);
  const int arrays = a.h == nullptr ? 1 : element ? 3 : 2;
  size_t smem = queue_smem<T, V, CH, STAGES>(a.H, arrays, threads);
  if (V == 1 && STAGES > 0 && CH > 8) smem += sizeof(float) * 2 * CH * threads;
  // 1024 threads an SM (512 with many columns a thread), fewer blocks where
  // their rows in flight would not fit
  int blocks = std::max(1, (CH * V <= 16 ? 1024 : 512) / threads);
  if (smem > 0) blocks = std::max(1, std::min<int>(blocks, kQueueSmem / smem));
  if (smem > 40 * 1024) {
    const cudaError_t e = allow_smem(k, smem);
    if (e != cudaSuccess) return e;
  }
  const int rows = ceil_div(a.T, WARP ? threads / 32 : 1);
  int grid = std::min(rows, blocks * num_sms);
  if (SHIFT) grid = shifted_grid(grid, rows);
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
    const bool shift =
        !vec && rows_shift_alike<T>(a.T, a.H, {a.x, a.h, a.gate_kind == MOE_GATE_ELEMENT ? a.gate : nullptr, a.r, a.y},
                                    {a.ld_x, a.h != nullptr ? a.ld_h : a.H, a.gate_kind == MOE_GATE_ELEMENT ? a.ld_gate : a.H});
    // (the last packs of a shifted row reach at most V - 1 elements beyond it)
    const int packs = vec ? a.H / V : shift ? ceil_div(a.H + V - 1, V) : a.H;
    auto threads = [&](int ch) { return ceil_div(ceil_div(packs, ch), 32) * 32; };
    if (shift && packs <= 1024) return run<T, V, 1, 4, false, 0, true>(a, threads(1), num_sms, st);
    if constexpr (sizeof(T) == 4)
      if (shift && packs <= 2048) return run<T, V, 2, 2, false, 0, true>(a, threads(2), num_sms, st);
    if (!vec) {
      if (a.H <= 1024) return run<T, 1, 4, 3, false, 256>(a, 256, num_sms, st);
      if (a.H <= 2048) return run<T, 1, 8, 3, false, 256>(a, 256, num_sms, st);
      if (a.H <= 4096) return run<T, 1, 16, 3, false, 256>(a, 256, num_sms, st);
      if (a.H > 8192) return run<T, 1, 32, 0, false, 512>(a, 512, num_sms, st);
      // three arrays' rows of 8192 fp32 columns do not fit into shared memory
      if constexpr (sizeof(T) == 4) return run<T, 1, 16, 0, false, 512>(a, 512, num_sms, st);
      else return run<T, 1, 16, 2, false, 512>(a, 512, num_sms, st);
    }
    if (packs <= 32) return run<T, V, 1, 4, true>(a, 128, num_sms, st);
    if (packs <= 64) return run<T, V, 2, 4, true>(a, 128, num_sms, st);
    // as many stages as three arrays' rows fit into shared memory
    if (packs <= 1024) return run<T, V, 1, 4, false>(a, threads(1), num_sms, st);
    if (packs <= 2048) return run<T, V, 2, 2, false>(a, threads(2), num_sms, st);
    if constexpr (sizeof(T) == 4) return run<T, V, 8, 0, false>(a, threads(8), num_sms, st);
    return cudaErrorInvalidValue;  // 16-bit rows have at most 2048 packs
  });
}

}  // namespace bsmoe
