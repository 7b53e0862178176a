// Gradients of the norms around a block (formulas in norm.cu). With
// G = dr + N'(r)^T dy, u = w gate G:
//   N'(v)^T d = inv (w d) - v inv^3 sum(v w d) / H,  inv = rsqrt(mean v^2 + eps)
//   dx = beta G,  dh = alpha (inv u - h inv^3 sum(h u) / H)
//   d_weight = sum_t alpha gate G h inv,  d_next_weight = sum_t dy r inv_r,
//   d_gate = act' alpha z G, summed over the axes that the gate lacks.
//
// One pass over the rows: every input is read once and every output written
// once; the row statistics are computed again from rows that are loaded
// anyway, so the forward saves nothing. A block walks many rows with the next
// ones on their way (RowQueue) and keeps two column sums of its rows in
// registers: sum_t gate inv G h, from which the weight's gradient (times
// alpha g) and the channel gate's (times alpha act' w) both follow, and the
// next weight's. A second small kernel adds the blocks' sums in block order,
// so the same call gives the same bits. A row needs one barrier: G is linear in
// dr, w dy and r, so the sums that dh needs are taken for the three apart,
// beside the sums that G needs,
//   sum h w g G = sum h w g dr + inv_r sum h w g (w' dy) - back sum h w g r.
//
// Measured: norm_after's gradient with token gate and next norm, 8192 rows of
// 4096 bf16 columns, 85 us with the column sums, 4.7 TB/s (a plain copy: 6.8).
// What is left is the latency of its two passes with 16 warps an SM: the column
// sums and the row leave no registers for more. Three stages of rows instead of
// two: one block an SM fits, 133 us. Half as many columns a thread: 121 us.
#include "norm_common.cuh"

namespace bsmoe {

namespace {

enum { kDr = 0, kDy = 1, kR = 2, kH = 3, kGate = 4 };
enum { kSumBlock = 0, kSumNext = 1 };

__device__ __forceinline__ bool wants(const NormBackwardArgs& b, int which) {
  if (which == kSumBlock) return b.d_weight != nullptr || b.f.gate_kind == MOE_GATE_CHANNEL;
  return b.d_next_weight != nullptr;
}
__device__ __forceinline__ float* partial_row(const NormBackwardArgs& b, int which, int part) {
  return b.partials + (static_cast<size_t>(which) * kNormParts + part) * b.f.H;
}

// One row per warp (WARP) or per block. ELEMENT: a gate by element.
template <typename T, int V, int CH, int STAGES, int THREADS, bool AFTER, bool NEXT, bool ELEMENT, bool WARP, bool SHIFT>
__global__ void __launch_bounds__(WARP ? 256 : THREADS > 0 ? THREADS : 512, WARP ? 2 : THREADS == 256 ? CH <= 8 ? 4 : 3 : 1)
    norm_backward_kernel(NormBackwardArgs b) {
  constexpr int ARRAYS = AFTER ? ELEMENT ? 5 : 4 : 3;
  // the columns' factors stand in shared memory behind the ring (each thread
  // its own): beside the column sums they would not fit into the registers
  constexpr bool CACHED = STAGES > 0 && !WARP;
  extern __shared__ __align__(16) uint8_t s_ring[];
  constexpr int SUMS = AFTER ? NEXT ? 8 : 2 : 2;
  __shared__ __align__(16) float s_sum[2][SUMS * 16];  // by the row's parity
  const NormArgs& a = b.f;
  RowQueue<T, V, CH, ARRAYS, STAGES, WARP ? 32 : THREADS, SHIFT> rows;
  rows.H = a.H;
  rows.j = WARP ? threadIdx.x & 31 : threadIdx.x;
  rows.src[kDr] = static_cast<const T*>(b.dr);
  rows.src[kDy] = NEXT ? static_cast<const T*>(b.dy) : nullptr;
  rows.src[kR] = NEXT ? static_cast<const T*>(a.r) : nullptr;
  rows.ld[kDr] = b.ld_dr;
  rows.ld[kDy] = b.ld_dy;
  rows.ld[kR] = b.ld_r;
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
  const int warp = threadIdx.x >> 5;
  const int per_block = WARP ? blockDim.x / 32 : 1;
  const int first = blockIdx.x * per_block + (WARP ? warp : 0), step = gridDim.x * per_block;
  const int n = first < a.T ? (a.T - 1 - first) / step + 1 : 0;
  rows.set_shift(AFTER ? b.dh : b.dx, first);
  rows.start(first, step, n, s_ring);

  auto factor = [&](int which, int c) {  // w times the channel gate, or the next w
    const void* weight = which == kSumNext ? a.next_weight : a.norm ? a.weight : nullptr;
    const bool gated = which == kSumBlock && a.gate_kind == MOE_GATE_CHANNEL;
    return column_factor<SHIFT, V>(
        c, a.H,
        [&](int at) {
          const Values<V> f = load_weight<T, V>(weight, a.weight_f32, a.w_offset, at);
          return gated ? f * channel_gate<T, V>(a, at) : f;
        },
        [&](int at) {
          const float f = load_weight<T, 1>(weight, a.weight_f32, a.w_offset, at).v[0];
          return gated ? f * channel_gate<T, 1>(a, at).v[0] : f;
        });
  };
  constexpr int F = V > 1 ? 4 : 1;  // floats of a factor that move together
  using FactorPack = Pack<float, F>;
  FactorPack* s_factor = reinterpret_cast<FactorPack*>(s_ring + static_cast<size_t>(STAGES) * rows.stage_bytes) + rows.j;
  auto factor_at = [&](int which, int i, int v) -> FactorPack& {
    return s_factor[((which * CH + i) * (V / F) + v / F) * rows.threads()];
  };
  auto get_factor = [&](int which, int i, int c) {
    if constexpr (CACHED) {
      Values<V> f;
#pragma unroll
      for (int v = 0; v < V; v += F) {
        const FactorPack q = factor_at(which, i, v);
#pragma unroll
        for (int e = 0; e < F; ++e) f.v[v + e] = q.e[e];
      }
      return f;
    } else {
      return factor(which, c);
    }
  };
  if constexpr (CACHED) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = rows.column(i);
      if (!rows.in(i)) continue;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        if (which == kSumBlock ? !AFTER : !NEXT) continue;
        const Values<V> f = factor(which, c);
#pragma unroll
        for (int v = 0; v < V; v += F) {
          FactorPack q;
#pragma unroll
          for (int e = 0; e < F; ++e) q.e[e] = f.v[v + e];
          factor_at(which, i, v) = q;
        }
      }
    }
  }
  if (!WARP) {
    for (int i = threadIdx.x; i < 2 * SUMS * 16; i += blockDim.x) (&s_sum[0][0])[i] = 0.f;
    __syncthreads();
  }
  const float inv_h = 1.f / static_cast<float>(a.H);
  Values<V> sums[2][CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) sums[0][i] = sums[1][i] = zeros<V>();
  const int64_t out_step = static_cast<int64_t>(step) * a.H, out_first = static_cast<int64_t>(first) * a.H + rows.j * V - rows.shift;
  T* dx_out = b.dx != nullptr ? static_cast<T*>(b.dx) + out_first : nullptr;
  T* dh_out = static_cast<T*>(b.dh) + out_first;
  T* dg_out = static_cast<T*>(b.d_gate) + (ELEMENT ? out_first : first);
  const T* token_gate = static_cast<const T*>(a.gate) + first * a.ld_gate;
  const bool has_dr = b.dr != nullptr;
  for (int k = 0; k < n; ++k) {
    rows.next();
    float2 rr = make_float2(0.f, 0.f), rd = rr, hh = rr, h_dr = rr, h_dy = rr, h_r = rr;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = rows.column(i);
      if (!rows.in(i)) continue;
      Values<V> r, d;
      if constexpr (NEXT) {
        r = row_values(rows, kR, i);
        d = get_factor(kSumNext, i, c) * row_values(rows, kDy, i);
        add_dot(rr, r, r);
        add_dot(rd, r, d);
      }
      if constexpr (AFTER) {
        const Values<V> h = row_values(rows, kH, i);
        Values<V> u = h * get_factor(kSumBlock, i, c);
        if constexpr (ELEMENT) u = u * gate_values(a.gate_act, row_values(rows, kGate, i));
        add_dot(hh, h, h);
        if (has_dr) add_dot(h_dr, u, row_values(rows, kDr, i));
        if constexpr (NEXT) {
          add_dot(h_dy, u, d);
          add_dot(h_r, u, r);
        }
      }
    }
    float inv_r = 0.f, back_r = 0.f, inv = 1.f, back = 0.f, h_G = 0.f;
    if constexpr (AFTER && NEXT) {
      float v[8] = {rr.x + rr.y, rd.x + rd.y, hh.x + hh.y, h_dr.x + h_dr.y, h_dy.x + h_dy.y, h_r.x + h_r.y, 0.f, 0.f};
      row_sums<8, WARP>(v, s_sum[k & 1]);
      inv_r = rsqrtf(v[0] * inv_h + a.next_eps);
      back_r = inv_r * inv_r * (inv_r * (v[1] * inv_h));
      inv = rsqrtf(v[2] * inv_h + a.eps);
      h_G = fmaf(-back_r, v[5], fmaf(inv_r, v[4], v[3]));
    } else if constexpr (NEXT) {
      float v[2] = {rr.x + rr.y, rd.x + rd.y};
      row_sums<2, WARP>(v, s_sum[k & 1]);
      inv_r = rsqrtf(v[0] * inv_h + a.next_eps);
      back_r = inv_r * inv_r * (inv_r * (v[1] * inv_h));
    } else {
      float v[2] = {hh.x + hh.y, h_dr.x + h_dr.y};
      row_sums<2, WARP>(v, s_sum[k & 1]);
      inv = rsqrtf(v[0] * inv_h + a.eps);
      h_G = v[1];
    }
    float gt = 1.f;
    if constexpr (AFTER) {
      if (!a.norm) inv = 1.f;
      else back = inv * inv * (inv * (h_G * inv_h));
      if (a.gate_kind == MOE_GATE_TOKEN) {
        const float logit = to_f32(*token_gate);
        gt = gate_value(a.gate_act, logit);
        token_gate += step * a.ld_gate;
        if (rows.j == 0)
          *dg_out = from_f32<T>(gate_with_slope(a.gate_act, logit).slope.v[0] * (a.alpha * (inv * h_G)));
      }
    }
    const float scale = a.alpha * gt;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = rows.column(i);
      if (!rows.in(i)) continue;
      Values<V> G = has_dr ? row_values(rows, kDr, i) : zeros<V>();
      if constexpr (NEXT) {
        const Values<V> r = row_values(rows, kR, i), d = row_values(rows, kDy, i) * inv_r;
        G = fma(r, -back_r, fma(d, get_factor(kSumNext, i, c), G));
        sums[kSumNext][i] = fma(d, r, sums[kSumNext][i]);
      }
      if (dx_out != nullptr)
        store_values(rows, dx_out, i, a.beta != 1.f ? G * a.beta : G);
      if constexpr (AFTER) {
        const Values<V> h = row_values(rows, kH, i), w = get_factor(kSumBlock, i, c);
        if constexpr (ELEMENT) {  // its gradient takes the G without it
          const Gate<V> g = gate_with_slope(a.gate_act, row_values(rows, kGate, i));
          store_values(rows, dg_out, i, G * (h * (a.alpha * inv)) * w * g.slope);
          G = G * g.value;
        }
        sums[kSumBlock][i] = fma(G * (gt * inv), h, sums[kSumBlock][i]);
        store_values(rows, dh_out, i, fma(h, -scale * back, w * (G * (scale * inv))));
      }
    }
    if (dx_out != nullptr) dx_out += out_step;
    dh_out += out_step;
    dg_out += ELEMENT ? out_step : step;
  }

  float* s_cols = reinterpret_cast<float*>(s_ring);  // WARP: the join of the block's warps, after the rows
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (!wants(b, which)) continue;
    float* part = partial_row(b, which, blockIdx.x);
    if (WARP) {  // the warps of the block in turn
      for (int w = 0; w < per_block; ++w) {
        __syncthreads();
        if (warp != w) continue;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int c = rows.column(i);
          if (!rows.in(i)) continue;
#pragma unroll
          for (int e = 0; e < V; ++e) s_cols[c + e] = (w > 0 ? s_cols[c + e] : 0.f) + sums[which][i].v[e];
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.H; c += blockDim.x) part[c] = s_cols[c];
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = rows.column(i);
        if (!rows.in(i)) continue;
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (!SHIFT || (c + e >= 0 && c + e < a.H)) part[c + e] = sums[which][i].v[e];
      }
    }
  }
}

// Any width and alignment: rows are read again for each use, the column sums
// stand in shared memory (each thread its own columns).
template <typename T>
__global__ void __launch_bounds__(1024) norm_backward_general_kernel(NormBackwardArgs b) {
  extern __shared__ float s_cols[];  // [sums wanted][H]
  __shared__ float s_sum[2][2][2][32];
  pdl_wait();
  pdl_launch_dependents();
  const NormArgs& a = b.f;
  const bool after = a.h != nullptr, next = a.next != 0;
  const float inv_h = 1.f / static_cast<float>(a.H);
  float* s_acc[2];
  {
    int n = 0;
    for (int which = 0; which < 2; ++which) {
      s_acc[which] = s_cols + static_cast<size_t>(n) * a.H;
      n += wants(b, which);
    }
  }
  for (int which = 0; which < 2; ++which)
    if (wants(b, which))
      for (int c = threadIdx.x; c < a.H; c += blockDim.x) s_acc[which][c] = 0.f;
  const bool column_gate = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_ELEMENT;
  int parity = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 1) {
    const T* dr = static_cast<const T*>(b.dr) + t * b.ld_dr;
    const T* dy = static_cast<const T*>(b.dy) + t * b.ld_dy;
    const T* r = static_cast<const T*>(a.r) + t * b.ld_r;
    const T* h = static_cast<const T*>(a.h) + t * a.ld_h;
    const T* gate = static_cast<const T*>(a.gate) + (a.gate_kind == MOE_GATE_CHANNEL ? 0 : t * a.ld_gate);
    auto weight_at = [&](const void* w, int c) {
      return load_weight<T, 1>(w, a.weight_f32, a.w_offset, c).v[0];
    };
    float next_inv = 0.f, next_back = 0.f;
    if (next) {
      float ss[2] = {0.f, 0.f};
      for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
        const float rf = to_f32(r[c]);
        ss[0] = fmaf(rf, rf, ss[0]);
        ss[1] = fmaf(rf, weight_at(a.next_weight, c) * to_f32(dy[c]), ss[1]);
      }
      row_sum<2, false>(ss, s_sum[parity][0]);
      next_inv = rsqrtf(ss[0] * inv_h + a.next_eps);
      next_back = next_inv * next_inv * (next_inv * (ss[1] * inv_h));
    }
    auto G_at = [&](int c) {
      float g = b.dr != nullptr ? to_f32(dr[c]) : 0.f;
      if (next) g += next_inv * (weight_at(a.next_weight, c) * to_f32(dy[c])) - to_f32(r[c]) * next_back;
      return g;
    };
    if (next && b.d_next_weight != nullptr)
      for (int c = threadIdx.x; c < a.H; c += blockDim.x)
        s_acc[kSumNext][c] = fmaf(to_f32(dy[c]), to_f32(r[c]) * next_inv, s_acc[kSumNext][c]);
    if (b.dx != nullptr)
      for (int c = threadIdx.x; c < a.H; c += blockDim.x)
        static_cast<T*>(b.dx)[t * a.H + c] = from_f32<T>(a.beta * G_at(c));
    if (!after) continue;
    float gt = 1.f, gt_slope = 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN) {
      const Gate<1> g = gate_with_slope(a.gate_act, to_f32(gate[0]));
      gt = g.value.v[0];
      gt_slope = g.slope.v[0];
    }
    float inv = 1.f, back = 0.f;
    if (a.norm || a.gate_kind == MOE_GATE_TOKEN) {
      float ss[2] = {0.f, 0.f};
      for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
        const float hf = to_f32(h[c]);
        float w = weight_at(a.norm ? a.weight : nullptr, c);
        if (column_gate) w *= gate_value(a.gate_act, to_f32(gate[c]));
        ss[0] = fmaf(hf, hf, ss[0]);
        ss[1] = fmaf(hf, w * G_at(c), ss[1]);
      }
      row_sum<2, false>(ss, s_sum[parity][1]);
      if (a.norm) {
        inv = rsqrtf(ss[0] * inv_h + a.eps);
        back = inv * inv * (inv * (ss[1] * inv_h));
      }
      if (a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0)
        static_cast<T*>(b.d_gate)[t] = from_f32<T>(gt_slope * (a.alpha * (inv * ss[1])));
    }
    const float scale = a.alpha * gt;
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
      const float hf = to_f32(h[c]), w = weight_at(a.norm ? a.weight : nullptr, c), G = G_at(c);
      float g = 1.f;
      if (column_gate) {
        const Gate<1> gs = gate_with_slope(a.gate_act, to_f32(gate[c]));
        g = gs.value.v[0];
        if (a.gate_kind == MOE_GATE_ELEMENT)
          static_cast<T*>(b.d_gate)[t * a.H + c] = from_f32<T>(gs.slope.v[0] * (a.alpha * G * (hf * inv * w)));
      }
      const float gG = scale * (g * G);
      if (wants(b, kSumBlock))
        s_acc[kSumBlock][c] =
            fmaf(gt * inv * (a.gate_kind == MOE_GATE_ELEMENT ? g : 1.f) * G, hf, s_acc[kSumBlock][c]);
      static_cast<T*>(b.dh)[t * a.H + c] = from_f32<T>(inv * (w * gG) - scale * (hf * back));
    }
  }
  for (int which = 0; which < 2; ++which)
    if (wants(b, which))
      for (int c = threadIdx.x; c < a.H; c += blockDim.x) partial_row(b, which, blockIdx.x)[c] = s_acc[which][c];
}

// Column sums over the blocks' parts, in part order within each of 32 strands
// that are then added in order, and the gradients that follow from them. grid
// (columns / 32, 2).
template <typename T>
__global__ void __launch_bounds__(1024) column_sum_kernel(NormBackwardArgs b, int parts) {
  __shared__ float s[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const NormArgs& a = b.f;
  const int which = blockIdx.y;
  if (!wants(b, which)) return;
  const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f, part[(kNormParts + 31) / 32];  // loaded together: one load's latency
#pragma unroll
  for (int i = 0; i < (kNormParts + 31) / 32; ++i) {
    const int p = strand + 32 * i;
    part[i] = p < parts && c < a.H ? partial_row(b, which, p)[c] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < (kNormParts + 31) / 32; ++i) v += part[i];
  s[strand][lane] = v;
  __syncthreads();
  if (strand != 0 || c >= a.H) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) v += s[i][lane];
  auto store_weight = [&](void* out, float d) {
    if (a.weight_f32) static_cast<float*>(out)[c] = d;
    else static_cast<T*>(out)[c] = from_f32<T>(d);
  };
  if (which == kSumNext) {
    store_weight(b.d_next_weight, v);
    return;
  }
  v *= a.alpha;
  float gate = 1.f;
  if (a.gate_kind == MOE_GATE_CHANNEL) {
    const float w = load_weight<T, 1>(a.norm ? a.weight : nullptr, a.weight_f32, a.w_offset, c).v[0];
    const Gate<1> g = gate_with_slope(a.gate_act, to_f32(static_cast<const T*>(a.gate)[c]));
    gate = g.value.v[0];
    static_cast<T*>(b.d_gate)[c] = from_f32<T>(g.slope.v[0] * w * v);
  }
  if (b.d_weight != nullptr) store_weight(b.d_weight, gate * v);
}

template <typename T, int V, int CH, int STAGES, bool WARP, int THREADS = 0, bool SHIFT = false>
cudaError_t run(const NormBackwardArgs& b, int threads, int num_sms, cudaStream_t st, int* parts) {
  const NormArgs& a = b.f;
  const bool element = a.gate_kind == MOE_GATE_ELEMENT;
  auto* k = a.h == nullptr ? norm_backward_kernel<T, V, CH, STAGES, THREADS, false, true, false, WARP, SHIFT>
            : a.next       ? (element ? norm_backward_kernel<T, V, CH, STAGES, THREADS, true, true, true, WARP, SHIFT>
                                      : norm_backward_kernel<T, V, CH, STAGES, THREADS, true, true, false, WARP, SHIFT>)
                           : (element ? norm_backward_kernel<T, V, CH, STAGES, THREADS, true, false, true, WARP, SHIFT>
                                      : norm_backward_kernel<T, V, CH, STAGES, THREADS, true, false, false, WARP, SHIFT>);
  const int arrays = (b.dr != nullptr) + 2 * (a.next != 0) + (a.h != nullptr) + element;
  size_t smem = queue_smem<T, V, CH, STAGES>(a.H, arrays, threads);
  if (WARP) smem = std::max(smem, sizeof(float) * a.H);
  else if (STAGES > 0) smem += sizeof(float) * 2 * CH * V * threads;
  int blocks = std::max(1, (THREADS == 256 ? CH <= 8 ? 1024 : 768 : 512) / threads);
  if (smem > 0) blocks = std::max(1, std::min<int>(blocks, kQueueSmem / smem));
  if (smem > 40 * 1024) {
    const cudaError_t e = allow_smem(k, smem);
    if (e != cudaSuccess) return e;
  }
  const int rows = ceil_div(a.T, WARP ? threads / 32 : 1);
  *parts = std::min(std::min(rows, blocks * num_sms), kNormParts);
  if (SHIFT) *parts = shifted_grid(*parts, rows);
  return launch_kernel(true, k, *parts, threads, smem, st, b);
}

template <typename T>
cudaError_t run_general(const NormBackwardArgs& b, int num_sms, cudaStream_t st, int* parts) {
  const bool block = b.d_weight != nullptr || b.f.gate_kind == MOE_GATE_CHANNEL;
  const size_t smem = sizeof(float) * (block + (b.d_next_weight != nullptr)) * b.f.H;
  if (smem > 40 * 1024) {
    const cudaError_t e = allow_smem(norm_backward_general_kernel<T>, smem);
    if (e != cudaSuccess) return e;
  }
  *parts = std::min(std::min(b.f.T, num_sms), kNormParts);
  return launch_kernel(true, norm_backward_general_kernel<T>, *parts, 1024, smem, st, b);
}

}  // namespace

cudaError_t launch_norm_backward(int dtype, const NormBackwardArgs& b, int num_sms, cudaStream_t st) {
  return with_dtype(dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    constexpr int V = kVec<T>;
    const NormArgs& a = b.f;
    const bool vec = rows_vectorize<T>(a.H,
                                       {b.dr, b.dy, a.h, a.r, a.weight, a.next_weight,
                                        a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate, b.dx, b.dh,
                                        a.gate_kind == MOE_GATE_ELEMENT ? b.d_gate : nullptr},
                                       {b.ld_dr, b.ld_dy, a.ld_h, b.ld_r,
                                        a.gate_kind == MOE_GATE_ELEMENT ? a.ld_gate : 0});
    const bool shift =
        !vec && rows_shift_alike<T>(a.T, a.H,
                                    {b.dr, b.dy, a.h, a.next ? a.r : nullptr, b.dx, b.dh,
                                     a.gate_kind == MOE_GATE_ELEMENT ? a.gate : nullptr,
                                     a.gate_kind == MOE_GATE_ELEMENT ? b.d_gate : nullptr},
                                    {b.dr != nullptr ? b.ld_dr : a.H, a.next ? b.ld_dy : a.H,
                                     a.h != nullptr ? a.ld_h : a.H, a.next ? b.ld_r : a.H,
                                     a.gate_kind == MOE_GATE_ELEMENT ? a.ld_gate : a.H});
    // (the last packs of a shifted row reach at most V - 1 elements beyond it)
    const int packs = vec ? a.H / V : shift ? ceil_div(a.H + V - 1, V) : a.H;
    auto threads = [&](int ch) { return ceil_div(ceil_div(packs, ch), 32) * 32; };
    int parts = 0;
    cudaError_t e = cudaSuccess;
    if (a.T == 0) {
    } else if (shift && packs <= 256) {
      e = run<T, V, 1, 2, false, 0, true>(b, threads(1), num_sms, st, &parts);
    } else if (shift && packs <= 1024) {
      e = run<T, V, 2, 2, false, 0, true>(b, threads(2), num_sms, st, &parts);
    } else if (vec && packs <= 32) {
      e = run<T, V, 1, 2, true>(b, 256, num_sms, st, &parts);
    } else if (vec && packs <= 64) {
      e = run<T, V, 2, 2, true>(b, 256, num_sms, st, &parts);
    } else if (vec && packs <= 256) {
      e = run<T, V, 1, 2, false>(b, threads(1), num_sms, st, &parts);
    } else if (vec && packs <= 1024) {
      e = run<T, V, 2, 2, false>(b, threads(2), num_sms, st, &parts);
    } else if (!vec && a.H <= 1024) {
      e = run<T, 1, 4, 2, false, 256>(b, 256, num_sms, st, &parts);
    } else if (!vec && a.H <= 2048) {
      e = run<T, 1, 8, 2, false, 256>(b, 256, num_sms, st, &parts);
    } else if (!vec && a.H <= 4096) {
      e = run<T, 1, 16, 2, false, 256>(b, 256, num_sms, st, &parts);
    } else if (!vec && a.H <= 8192) {
      e = run<T, 1, 16, 0, false, 512>(b, 512, num_sms, st, &parts);
    } else if (vec && packs <= 2048 && sizeof(T) == 4) {
      if constexpr (sizeof(T) == 4) e = run<T, V, 4, 0, false>(b, threads(4), num_sms, st, &parts);
    } else {
      e = run_general<T>(b, num_sms, st, &parts);
    }
    if (e != cudaSuccess) return e;
    if (b.d_weight == nullptr && b.d_next_weight == nullptr && a.gate_kind != MOE_GATE_CHANNEL) return e;
    return launch_kernel(true, column_sum_kernel<T>, dim3(ceil_div(a.H, 32), 2), 1024, 0, st, b, parts);
  });
}

}  // namespace bsmoe
