// Routing (router_forward.cuh): the mean scores' last sum, and the gradient.
//
// The gradient reads a token's logits once where every expert has a part (mean scores, or
// softmax weights that are not renormalised) and only the chosen ones' otherwise; it
// writes a row of d_logits, the chosen experts' elements last. Bound like the forward:
// 65536 x 256 fp32, K = 8: 36 us, with mean scores 45; 16384 x 128 bf16, K = 4, with mean
// scores 6.4 (8.9 MB).
#include "router_common.cuh"

namespace bsmoe {

namespace {

// mean[e] = sum of the blocks' columns / T: 8 columns a block, 32 rows at a time,
// added up in a fixed order.
__global__ void __launch_bounds__(256) route_mean_kernel(const float* __restrict__ partials, int blocks, int E, float T,
                                                         float* __restrict__ mean) {
  constexpr int U = (kRouteParts + 31) / 32;
  __shared__ float part[8][33];
  const int c = threadIdx.x % 8, r = threadIdx.x / 8, e = blockIdx.x * 8 + c;
  pdl_wait();
  pdl_launch_dependents();
  float v[U], sum = 0.f;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int b = r + 32 * i;
    v[i] = b < blocks && e < E ? partials[static_cast<size_t>(b) * E + e] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < U; ++i) sum += v[i];
  part[c][r] = sum;
  __syncthreads();
  const int w = threadIdx.x / 32, col = blockIdx.x * 8 + w;
  const float total = warp_sum(part[w][threadIdx.x % 32]);
  if (threadIdx.x % 32 == 0 && col < E) mean[col] = T > 0.f ? total / T : 0.f;
}

template <int P, typename T>
__device__ __forceinline__ void store_as(void* base, int64_t at, int n, bool vec, const float (&x)[P]) {
  T* p = static_cast<T*>(base) + at;
  constexpr int W = sizeof(T) * P >= 16 ? 16 / sizeof(T) : P;
  if (vec && n == P) {
#pragma unroll
    for (int i = 0; i < P; i += W) {
      float f[W];
#pragma unroll
      for (int j = 0; j < W; ++j) f[j] = x[i + j];
      store_pack(p + i, pack<T>(f));
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i < n) p[i] = from_f32<T>(x[i]);
  }
}

// With s the scores, w' the chosen ones over their sum S and v = scale dw:
//   renormalised: ds_k = (v_k - <v, w'>) / S, else ds_k = v_k; 0 for the rest;
//   softmax: dx = s (ds - <ds, s>), which for renormalised weights is
//            w' (v - <v, w'>) at the chosen and 0 elsewhere;
//   sigmoid: dx = s (1 - s) ds;
//   mean, p = s / sum(s), h = dmean / T: dx += p (h - <h, p>) (sigmoid: times 1 - s).
template <int P, int L, bool SIGMOID>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(Shape s, const float* __restrict__ dw,
                                                                       const float* __restrict__ dmean,
                                                                       const void* __restrict__ logits,
                                                                       const int32_t* __restrict__ idx, bool vec_out,
                                                                       void* __restrict__ dx) {
  constexpr int kTokens = kRouteThreads / L;
  const int lane = threadIdx.x & 31, sub = lane % L;
  const Span sp = span_of(s, sub);
  const bool dense = dmean != nullptr || (!SIGMOID && !s.renorm);
  const float inv_T = 1.f / static_cast<float>(s.T);
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens; t0 < s.T; t0 += static_cast<int64_t>(gridDim.x) * kTokens) {
    const int64_t t = t0 + threadIdx.x / L;
    const bool valid = t < s.T;
    const int64_t tr = valid ? t : s.T - 1;
    float x[P], d[P];
    if (dense) load_logits<P>(s, logits, tr, sp, x);
    // lane k: the k-th choice
    int e = -1;
    float v = 0.f, xk = neg_inf();
    if (sub < s.K) {
      e = idx[tr * s.K + sub];
      if (e < 0 || e >= s.E) e = -1;
      if (e >= 0) {
        v = dw[tr * s.K + sub] * s.scale;
        xk = logit_at(s, logits, tr * s.ld + e);
      }
    }
    float most = neg_inf(), sum = 0.f;
    if (dense) {
#pragma unroll
      for (int i = 0; i < P; ++i) most = fmaxf(most, x[i]);
      most = lane_max<L>(most);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (!SIGMOID || most < -60.f) d[i] = x[i] == neg_inf() ? 0.f : exp_fast(x[i] - most);
        else d[i] = sigmoid_fast(x[i]);
        sum += d[i];
      }
      sum = lane_sum<L>(sum);
    }
    const float inv = sum != 0.f ? rcp_fast(sum) : 0.f;
    // the chosen experts' part: dx += add at expert e
    float add = 0.f, all = 0.f;  // all: <ds, s>, taken off every expert (softmax without renormalisation)
    if (s.renorm) {
      const float top = lane_max<L>(e >= 0 ? xk : neg_inf());
      const float sc = e >= 0 ? ratio_score<SIGMOID>(xk, top) : 0.f;
      const float S = lane_sum<L>(sc);
      const float wn = S != 0.f ? sc / S : 0.f;
      const float inner = lane_sum<L>(e >= 0 ? v * wn : 0.f);
      add = e >= 0 ? wn * (v - inner) : 0.f;
      if (SIGMOID) {
        float a, b;
        sigmoid_pair(xk, &a, &b);
        add *= b;
      }
    } else if (SIGMOID) {
      float a, b;
      sigmoid_pair(xk, &a, &b);
      add = e >= 0 ? v * a * b : 0.f;
    } else {
      const float sc = e >= 0 && most > neg_inf() ? expf(xk - most) * inv : 0.f;
      add = e >= 0 ? v * sc : 0.f;
      all = lane_sum<L>(add);
    }
    // the experts that are not chosen: their part of the mean's gradient and of `all`
    float inner = 0.f;
    if (dense) {
      float h[P];
      if (dmean != nullptr) {
        load_as<P, float>(dmean, sp.e0, sp.n, s.vec_bias, h);
#pragma unroll
        for (int i = 0; i < P; ++i) inner += i < sp.n ? d[i] * h[i] : 0.f;
        inner = lane_sum<L>(inner) * inv;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float g = dmean != nullptr ? (h[i] - inner) * inv_T - all : -all;
        d[i] *= inv * g;
        if (SIGMOID) d[i] *= sigmoid_fast(-x[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) d[i] = 0.f;
    }
    // the chosen: an expert's first slot adds up all of its slots
    float sum_k = 0.f;
    bool first_k = e >= 0;
    for (int k = 0; k < s.K; ++k) {
      const int ek = __shfl_sync(kFull, e, lane - sub + k);
      const float ak = __shfl_sync(kFull, add, lane - sub + k);
      sum_k += ek == e ? ak : 0.f;
      if (ek == e && k < sub) first_k = false;
    }
    if (dense && first_k) {
      float p = !SIGMOID || most < -60.f ? exp_fast(xk - most) : sigmoid_fast(xk);
      p *= inv * ((dmean != nullptr ? (__ldg(dmean + e) - inner) * inv_T : 0.f) - all);
      if (SIGMOID) p *= sigmoid_fast(-xk);
      sum_k += xk == neg_inf() ? 0.f : p;
    }
    const int64_t at = t * s.E;
    if (valid) {
      if (s.dtype == MOE_BF16) store_as<P, __nv_bfloat16>(dx, at + sp.e0, sp.n, vec_out, d);
      else if (s.dtype == MOE_FP16) store_as<P, __half>(dx, at + sp.e0, sp.n, vec_out, d);
      else store_as<P, float>(dx, at + sp.e0, sp.n, vec_out, d);
    }
    __syncwarp();  // the chosen experts' stores come after those of their lanes
    if (valid && first_k) {
      if (s.dtype == MOE_BF16) static_cast<__nv_bfloat16*>(dx)[at + e] = from_f32<__nv_bfloat16>(sum_k);
      else if (s.dtype == MOE_FP16) static_cast<__half*>(dx)[at + e] = from_f32<__half>(sum_k);
      else static_cast<float*>(dx)[at + e] = sum_k;
    }
  }
}

}  // namespace

cudaError_t launch_route_tokens(int dtype, const RouteArgs& a, int num_sms, cudaStream_t st) {
  if (a.T > 0) {
    const cudaError_t e = a.sigmoid ? launch_route_sigmoid(dtype, a, num_sms, st) : launch_route_softmax(dtype, a, num_sms, st);
    if (e != cudaSuccess) return e;
  }
  if (a.mean == nullptr) return cudaSuccess;
  const int blocks = route_blocks(a, split_of(a.E, a.K, a.G), kRouteParts);
  if (blocks == 1) return cudaSuccess;  // written by the block itself
  return launch_kernel(true, route_mean_kernel, ceil_div(a.E, 8), 256, 0, st, static_cast<const float*>(a.partials),
                       blocks, a.E, static_cast<float>(a.T), a.mean);
}

cudaError_t launch_route_tokens_backward(int dtype, const RouteArgs& a, const float* dw, const float* dmean, void* dx,
                                         int num_sms, cudaStream_t st) {
  const Split sp = split_of(a.E, a.K, 1);
  Shape s = shape_of(dtype, a, a.logits, a.ld, sp);
  s.vec_bias = s.vec_bias && aligned16(dmean);  // dmean is read as a bias is
  const bool vec_out = shape_of(dtype, a, dx, a.E, sp).vec;
  return with_split(sp, [&](auto P, auto L) {
    constexpr int p = decltype(P)::value, l = decltype(L)::value;
    const int blocks = route_blocks(a, sp, 16 * num_sms);
    return launch_kernel(blocks >= num_sms, a.sigmoid ? route_backward_kernel<p, l, true> : route_backward_kernel<p, l, false>,
                         blocks, kRouteThreads, 0, st, s, dw, dmean, a.logits,
                         static_cast<const int32_t*>(a.idx), vec_out, dx);
  });
}

}  // namespace bsmoe
