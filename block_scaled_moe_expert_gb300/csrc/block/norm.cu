// Norms before and after a block:
//   N(v; w) = v rsqrt(mean(v^2) + eps) (w + offset)
//   norm_before: y = N(x; w)
//   norm_after:  r = beta x + alpha g z, z = N(h; w) or h, g = act(gate),
//                and y = N(r; w_next) for the next block.
//
// One pass: a row lives in registers between its sums, so x and h are read
// once, r and y written once, and the sum over r^2 needs no second look at r.
// Bound by DRAM bandwidth (by latency for a few tokens). Sums in fp32 by a
// fixed tree.
#include "norm_common.cuh"

namespace bsmoe {

namespace {

// One row per warp (WARP) or per block; thread j of a row owns the packs
// j, j + threads, ... (CH of them).
template <typename T, int V, int CH, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : CH == 4 && sizeof(T) == 2 ? 512 : 1024) norm_kernel(NormArgs a) {
  __shared__ float s_sum[2][2][1][32];  // by the row's parity: a row's sums do not wait for the row before
  pdl_wait();
  pdl_launch_dependents();
  const int tpr = WARP ? 32 : blockDim.x;
  const int j = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int per_block = WARP ? blockDim.x / 32 : 1;
  const bool after = a.h != nullptr;
  const float inv_h = 1.f / static_cast<float>(a.H);
  int parity = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per_block + (WARP ? threadIdx.x >> 5 : 0); t < a.T;
       t += static_cast<int64_t>(gridDim.x) * per_block, parity ^= 1) {
    Pack<T, V> xp[CH], hp[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * tpr + j) * V;
      if (c < a.H) {
        if (after) hp[i] = load_pack<V>(static_cast<const T*>(a.h) + t * a.ld_h + c);
        xp[i] = load_pack<V>(static_cast<const T*>(a.x) + t * a.ld_x + c);
      }
    }
    float r[CH][V];
    if (after) {
      float scale = 1.f;
      if (a.norm) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          if ((i * tpr + j) * V >= a.H) continue;
          float hf[V];
          unpack(hp[i], hf);
#pragma unroll
          for (int e = 0; e < V; ++e) ss[0] = fmaf(hf[e], hf[e], ss[0]);
        }
        row_sum<1, WARP>(ss, s_sum[parity][0]);
        scale = rsqrtf(ss[0] * inv_h + a.eps);
      }
      float token_gate = 1.f;
      if (a.gate_kind == MOE_GATE_TOKEN)
        token_gate = gate_value(a.gate_act, to_f32(static_cast<const T*>(a.gate)[t * a.ld_gate]));
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = (i * tpr + j) * V;
        if (c >= a.H) continue;
        float z[V], xf[V];
        unpack(hp[i], z);
        unpack(xp[i], xf);
        if (a.norm) {
          float w[V];
          load_weight<T, V>(a.weight, a.weight_f32, a.w_offset, c, w);
#pragma unroll
          for (int e = 0; e < V; ++e) z[e] = z[e] * scale * w[e];
        }
        if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_ELEMENT) {
          float g[V];
          const int64_t row = a.gate_kind == MOE_GATE_ELEMENT ? t * a.ld_gate : 0;
          unpack(load_pack<V>(static_cast<const T*>(a.gate) + row + c), g);
#pragma unroll
          for (int e = 0; e < V; ++e) z[e] *= gate_value(a.gate_act, g[e]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) r[i][e] = fmaf(a.beta, xf[e], a.alpha * (token_gate * z[e]));
        store_pack(static_cast<T*>(a.r) + t * a.H + c, pack<T, V>(r[i]));
      }
      if (!a.next) continue;
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i) unpack(xp[i], r[i]);
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if ((i * tpr + j) * V >= a.H) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) ss[0] = fmaf(r[i][e], r[i][e], ss[0]);
    }
    row_sum<1, WARP>(ss, s_sum[parity][1]);
    const float scale = rsqrtf(ss[0] * inv_h + a.next_eps);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * tpr + j) * V;
      if (c >= a.H) continue;
      float w[V], y[V];
      load_weight<T, V>(a.next_weight, a.weight_f32, a.w_offset, c, w);
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = r[i][e] * scale * w[e];
      store_pack(static_cast<T*>(a.y) + t * a.H + c, pack<T, V>(y));
    }
  }
}

// Any width and alignment: the row is read again for each use (from the L2).
template <typename T>
__global__ void __launch_bounds__(1024) norm_general_kernel(NormArgs a) {
  __shared__ float s_sum[2][2][1][32];  // by the row's parity: a row's sums do not wait for the row before
  pdl_wait();
  pdl_launch_dependents();
  const bool after = a.h != nullptr;
  const float inv_h = 1.f / static_cast<float>(a.H);
  int parity = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 1) {
    const T* x = static_cast<const T*>(a.x) + t * a.ld_x;
    const T* h = static_cast<const T*>(a.h) + t * a.ld_h;
    float scale = 1.f;
    if (after && a.norm) {
      float ss[1] = {0.f};
      for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
        const float v = to_f32(h[c]);
        ss[0] = fmaf(v, v, ss[0]);
      }
      row_sum<1, false>(ss, s_sum[parity][0]);
      scale = rsqrtf(ss[0] * inv_h + a.eps);
    }
    const T* gate = static_cast<const T*>(a.gate);
    if (a.gate_kind == MOE_GATE_ELEMENT || a.gate_kind == MOE_GATE_TOKEN) gate += t * a.ld_gate;
    auto r_at = [&](int c) {
      const float xv = to_f32(x[c]);
      if (!after) return xv;
      float z = to_f32(h[c]);
      if (a.norm) {
        float w[1];
        load_weight<T, 1>(a.weight, a.weight_f32, a.w_offset, c, w);
        z = z * scale * w[0];
      }
      if (a.gate_kind != MOE_GATE_NONE)
        z *= gate_value(a.gate_act, to_f32(gate[a.gate_kind == MOE_GATE_TOKEN ? 0 : c]));
      return fmaf(a.beta, xv, a.alpha * z);
    };
    float ss[1] = {0.f};
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
      const float v = r_at(c);
      ss[0] = fmaf(v, v, ss[0]);
      if (after) static_cast<T*>(a.r)[t * a.H + c] = from_f32<T>(v);
    }
    if (a.next) {
      row_sum<1, false>(ss, s_sum[parity][1]);
      const float ns = rsqrtf(ss[0] * inv_h + a.next_eps);
      for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
        float w[1];
        load_weight<T, 1>(a.next_weight, a.weight_f32, a.w_offset, c, w);
        static_cast<T*>(a.y)[t * a.H + c] = from_f32<T>(r_at(c) * ns * w[0]);
      }
    }
  }
}

template <typename T, int CH, bool WARP>
cudaError_t run(const NormArgs& a, int grid, int threads, cudaStream_t st) {
  return launch_kernel(true, norm_kernel<T, kVec<T>, CH, WARP>, grid, threads, 0, st, a);
}

}  // namespace

cudaError_t launch_norm(int dtype, const NormArgs& a, int num_sms, cudaStream_t st) {
  return with_dtype(dtype, [&](auto* tag) {
    using T = std::remove_pointer_t<decltype(tag)>;
    const bool vec = rows_vectorize<T>(
        a.H, {a.x, a.h, a.weight, a.next_weight, a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate, a.r, a.y},
        {a.ld_x, a.ld_h, a.gate_kind == MOE_GATE_ELEMENT ? a.ld_gate : 0});
    const int packs = a.H / kVec<T>;
    if (!vec || packs > 4096)
      return launch_kernel(true, norm_general_kernel<T>, std::min(a.T, 2 * num_sms), 1024, 0, st, a);
    if (packs <= 64) return run<T, 2, true>(a, std::min(ceil_div(a.T, 4), 16 * num_sms), 128, st);
    // few rows: more threads a row; many rows: more packs a thread
    const int ch = a.T <= num_sms ? ceil_div(packs, 1024) : packs <= 256 ? 1 : packs <= 1024 ? 2 : 4;
    const int threads = ceil_div(ceil_div(packs, ch), 32) * 32;
    const int grid = std::min(a.T, num_sms * std::max(1, 2048 / threads));
    if (ch == 1) return run<T, 1, false>(a, grid, threads, st);
    if (ch == 2) return run<T, 2, false>(a, grid, threads, st);
    return run<T, 4, false>(a, grid, threads, st);
  });
}

}  // namespace bsmoe
