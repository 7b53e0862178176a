// Gradients of the norms around a block (formulas in norm.cu). With
// G = dr + N'(r)^T dy, u = w gate G:
//   N'(v)^T d = inv (w d) - v inv^3 sum(v w d) / H,  inv = rsqrt(mean v^2 + eps)
//   dx = beta G,  dh = alpha (inv u - h inv^3 sum(h u) / H)
//   d_weight = sum_t alpha gate G h inv,  d_next_weight = sum_t dy r inv_r,
//   d_gate = act' alpha z G, summed over the axes that the gate lacks.
//
// One pass over the rows: every input is read once and every output written
// once; the row statistics are computed again from rows that are loaded
// anyway, so the forward saves nothing. A block walks many rows and keeps the
// column sums (weights, channel gate) of its rows; a second small kernel adds
// the blocks' sums in block order, so the same call gives the same bits.
// Bound by DRAM bandwidth.
#include "norm_common.cuh"

namespace bsmoe {

namespace {

enum { kSumWeight = 0, kSumNext = 1, kSumGate = 2 };

__device__ __forceinline__ bool wants(const NormBackwardArgs& b, int which) {
  if (which == kSumWeight) return b.d_weight != nullptr;
  if (which == kSumNext) return b.d_next_weight != nullptr;
  return b.f.gate_kind == MOE_GATE_CHANNEL;
}
__device__ __forceinline__ float* partial_row(const NormBackwardArgs& b, int which, int part) {
  return b.partials + (static_cast<size_t>(which) * kNormParts + part) * b.f.H;
}

template <typename T, int V, int CH, bool WARP>
__global__ void __launch_bounds__(512) norm_backward_kernel(NormBackwardArgs b) {
  extern __shared__ float s_cols[];            // WARP: [H], the join of the block's warps
  __shared__ float s_sum[2][2][2][32];
  pdl_wait();
  pdl_launch_dependents();
  const NormArgs& a = b.f;
  const int tpr = WARP ? 32 : blockDim.x;
  const int j = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int warp = threadIdx.x >> 5;
  const int per_block = WARP ? blockDim.x / 32 : 1;
  const bool after = a.h != nullptr, next = a.next != 0;
  const float inv_h = 1.f / static_cast<float>(a.H);
  float sums[3][CH][V] = {};
  int parity = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per_block + (WARP ? warp : 0); t < a.T;
       t += static_cast<int64_t>(gridDim.x) * per_block, parity ^= 1) {
    Pack<T, V> drp[CH], dyp[CH], rp[CH], hp[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * tpr + j) * V;
      if (c >= a.H) continue;
      if (b.dr != nullptr) drp[i] = load_pack<V>(static_cast<const T*>(b.dr) + t * b.ld_dr + c);
      if (next) {
        dyp[i] = load_pack<V>(static_cast<const T*>(b.dy) + t * b.ld_dy + c);
        rp[i] = load_pack<V>(static_cast<const T*>(a.r) + t * b.ld_r + c);
      }
      if (after) hp[i] = load_pack<V>(static_cast<const T*>(a.h) + t * a.ld_h + c);
    }
    float G[CH][V];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (b.dr != nullptr && (i * tpr + j) * V < a.H) {
        unpack(drp[i], G[i]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) G[i][e] = 0.f;
      }
    }
    if (next) {
      float ss[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = (i * tpr + j) * V;
        if (c >= a.H) continue;
        float w[V], rf[V], dy[V];
        load_weight<T, V>(a.next_weight, a.weight_f32, a.w_offset, c, w);
        unpack(rp[i], rf);
        unpack(dyp[i], dy);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          ss[0] = fmaf(rf[e], rf[e], ss[0]);
          ss[1] = fmaf(rf[e], w[e] * dy[e], ss[1]);
        }
      }
      row_sum<2, WARP>(ss, s_sum[parity][0]);
      const float inv = rsqrtf(ss[0] * inv_h + a.next_eps);
      const float back = inv * inv * (inv * (ss[1] * inv_h));
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = (i * tpr + j) * V;
        if (c >= a.H) continue;
        float w[V], rf[V], dy[V];
        load_weight<T, V>(a.next_weight, a.weight_f32, a.w_offset, c, w);
        unpack(rp[i], rf);
        unpack(dyp[i], dy);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          G[i][e] += inv * (w[e] * dy[e]) - rf[e] * back;
          sums[kSumNext][i][e] = fmaf(dy[e], rf[e] * inv, sums[kSumNext][i][e]);
        }
      }
    }
    if (b.dx != nullptr) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = (i * tpr + j) * V;
        if (c >= a.H) continue;
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = a.beta * G[i][e];
        store_pack(static_cast<T*>(b.dx) + t * a.H + c, pack<T, V>(o));
      }
    }
    if (!after) continue;
    // u = w gate G in place of G where the norm is applied; gates by column
    // are read again for their gradient
    const bool column_gate = a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_ELEMENT;
    const T* gate_row =
        static_cast<const T*>(a.gate) + (a.gate_kind == MOE_GATE_CHANNEL ? 0 : t * a.ld_gate);
    float gt = 1.f, gt_slope = 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN) {
      gt = gate_value(a.gate_act, to_f32(gate_row[0]));
      gt_slope = gate_slope(a.gate_act, gt);
    }
    float inv = 1.f, back = 0.f;
    if (a.norm || a.gate_kind == MOE_GATE_TOKEN) {
      float ss[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = (i * tpr + j) * V;
        if (c >= a.H) continue;
        float w[V], hf[V];
        load_weight<T, V>(a.norm ? a.weight : nullptr, a.weight_f32, a.w_offset, c, w);
        unpack(hp[i], hf);
        if (column_gate) {
          float g[V];
          unpack(load_pack<V>(gate_row + c), g);
#pragma unroll
          for (int e = 0; e < V; ++e) w[e] *= gate_value(a.gate_act, g[e]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          ss[0] = fmaf(hf[e], hf[e], ss[0]);
          ss[1] = fmaf(hf[e], w[e] * G[i][e], ss[1]);
        }
      }
      row_sum<2, WARP>(ss, s_sum[parity][1]);
      if (a.norm) {
        inv = rsqrtf(ss[0] * inv_h + a.eps);
        back = inv * inv * (inv * (ss[1] * inv_h));
      }
      if (a.gate_kind == MOE_GATE_TOKEN && j == 0)
        static_cast<T*>(b.d_gate)[t] = from_f32<T>(gt_slope * (a.alpha * (inv * ss[1])));
    }
    const float scale = a.alpha * gt;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * tpr + j) * V;
      if (c >= a.H) continue;
      float w[V], hf[V], g[V], o[V];
      load_weight<T, V>(a.norm ? a.weight : nullptr, a.weight_f32, a.w_offset, c, w);
      unpack(hp[i], hf);
      if (column_gate) {
        unpack(load_pack<V>(gate_row + c), g);
        float dg[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          g[e] = gate_value(a.gate_act, g[e]);
          dg[e] = gate_slope(a.gate_act, g[e]) * (a.alpha * G[i][e] * (hf[e] * inv * w[e]));
        }
        if (a.gate_kind == MOE_GATE_ELEMENT) {
          store_pack(static_cast<T*>(b.d_gate) + t * a.H + c, pack<T, V>(dg));
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) sums[kSumGate][i][e] += dg[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = 1.f;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float gG = scale * (g[e] * G[i][e]);
        o[e] = inv * (w[e] * gG) - scale * (hf[e] * back);
        sums[kSumWeight][i][e] = fmaf(gG, hf[e] * inv, sums[kSumWeight][i][e]);
      }
      store_pack(static_cast<T*>(b.dh) + t * a.H + c, pack<T, V>(o));
    }
  }

#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (!wants(b, which)) continue;
    float* part = partial_row(b, which, blockIdx.x);
    if (WARP) {  // the warps of the block in turn
      for (int w = 0; w < per_block; ++w) {
        __syncthreads();
        if (warp != w) continue;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int c = (i * tpr + j) * V;
          if (c >= a.H) continue;
#pragma unroll
          for (int e = 0; e < V; ++e) s_cols[c + e] = (w > 0 ? s_cols[c + e] : 0.f) + sums[which][i][e];
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.H; c += blockDim.x) part[c] = s_cols[c];
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = (i * tpr + j) * V;
        if (c >= a.H) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) part[c + e] = sums[which][i][e];
      }
    }
  }
}

// Any width and alignment: rows are read again for each use, the column sums
// stand in shared memory (each thread its own columns).
template <typename T>
__global__ void __launch_bounds__(1024) norm_backward_general_kernel(NormBackwardArgs b) {
  extern __shared__ float s_cols[];  // [3][H]
  __shared__ float s_sum[2][2][2][32];
  pdl_wait();
  pdl_launch_dependents();
  const NormArgs& a = b.f;
  const bool after = a.h != nullptr, next = a.next != 0;
  const float inv_h = 1.f / static_cast<float>(a.H);
  float* s_acc[3];
  {
    int n = 0;
    for (int which = 0; which < 3; ++which) {
      s_acc[which] = s_cols + static_cast<size_t>(n) * a.H;
      n += wants(b, which);
    }
  }
  for (int which = 0; which < 3; ++which)
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
      float f[1];
      load_weight<T, 1>(w, a.weight_f32, a.w_offset, c, f);
      return f[0];
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
      gt = gate_value(a.gate_act, to_f32(gate[0]));
      gt_slope = gate_slope(a.gate_act, gt);
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
        g = gate_value(a.gate_act, to_f32(gate[c]));
        const float dg = gate_slope(a.gate_act, g) * (a.alpha * G * (hf * inv * w));
        if (a.gate_kind == MOE_GATE_ELEMENT) static_cast<T*>(b.d_gate)[t * a.H + c] = from_f32<T>(dg);
        else s_acc[kSumGate][c] += dg;
      }
      const float gG = scale * (g * G);
      if (b.d_weight != nullptr) s_acc[kSumWeight][c] = fmaf(gG, hf * inv, s_acc[kSumWeight][c]);
      static_cast<T*>(b.dh)[t * a.H + c] = from_f32<T>(inv * (w * gG) - scale * (hf * back));
    }
  }
  for (int which = 0; which < 3; ++which)
    if (wants(b, which))
      for (int c = threadIdx.x; c < a.H; c += blockDim.x) partial_row(b, which, blockIdx.x)[c] = s_acc[which][c];
}

// Column sums over the blocks' parts, in part order within each of 8 strands
// that are then added in order. grid (columns / 32, 3).
template <typename T>
__global__ void __launch_bounds__(256) column_sum_kernel(NormBackwardArgs b, int parts) {
  __shared__ float s[8][32];
  pdl_wait();
  pdl_launch_dependents();
  const int which = blockIdx.y;
  if (!wants(b, which)) return;
  const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < b.f.H)
    for (int p = strand; p < parts; p += 8) v += partial_row(b, which, p)[c];
  s[strand][lane] = v;
  __syncthreads();
  if (strand != 0 || c >= b.f.H) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) v += s[i][lane];
  void* out = which == kSumWeight ? b.d_weight : which == kSumNext ? b.d_next_weight : b.d_gate;
  if (which != kSumGate && b.f.weight_f32) static_cast<float*>(out)[c] = v;
  else static_cast<T*>(out)[c] = from_f32<T>(v);
}

template <typename T, int CH, bool WARP>
cudaError_t run(const NormBackwardArgs& b, int grid, int threads, cudaStream_t st) {
  return launch_kernel(true, norm_backward_kernel<T, kVec<T>, CH, WARP>, grid, threads,
                       WARP ? sizeof(float) * b.f.H : 0, st, b);
}

}  // namespace

cudaError_t launch_norm_backward(int dtype, const NormBackwardArgs& b, int num_sms, cudaStream_t st) {
  return with_dtype(dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    const NormArgs& a = b.f;
    const bool vec = rows_vectorize<T>(a.H,
                                       {b.dr, b.dy, a.h, a.r, a.weight, a.next_weight,
                                        a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate, b.dx, b.dh,
                                        a.gate_kind == MOE_GATE_ELEMENT ? b.d_gate : nullptr},
                                       {b.ld_dr, b.ld_dy, a.ld_h, b.ld_r,
                                        a.gate_kind == MOE_GATE_ELEMENT ? a.ld_gate : 0});
    const int packs = a.H / kVec<T>;
    const int most = std::min(kNormParts, 2 * num_sms);
    int parts = 0;
    cudaError_t e = cudaSuccess;
    if (a.T == 0) {
    } else if (vec && packs <= 64) {
      parts = std::min(ceil_div(a.T, 8), most);
      e = run<T, 2, true>(b, parts, 256, st);
    } else if (vec && packs <= 1024) {
      parts = std::min(a.T, most);
      const int threads = ceil_div(packs <= 512 ? packs : ceil_div(packs, 2), 32) * 32;
      e = packs <= 512 ? run<T, 1, false>(b, parts, threads, st) : run<T, 2, false>(b, parts, threads, st);
    } else {
      parts = std::min(a.T, std::min(num_sms, kNormParts));
      const int arrays = (b.d_weight != nullptr) + (b.d_next_weight != nullptr) + (a.gate_kind == MOE_GATE_CHANNEL);
      const size_t smem = sizeof(float) * arrays * a.H;
      if (smem > 48 * 1024)
        e = cudaFuncSetAttribute(norm_backward_general_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem));
      if (e == cudaSuccess)
        e = launch_kernel(true, norm_backward_general_kernel<T>, parts, 1024, smem, st, b);
    }
    if (e != cudaSuccess) return e;
    if (b.d_weight == nullptr && b.d_next_weight == nullptr && a.gate_kind != MOE_GATE_CHANNEL) return e;
    return launch_kernel(true, column_sum_kernel<T>, dim3(ceil_div(a.H, 32), 3), 256, 0, st, b, parts);
  });
}

}  // namespace bsmoe
