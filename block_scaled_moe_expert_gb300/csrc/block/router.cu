// The router's choice of experts (moe_route_tokens) and its gradient.
//
// A token's E logits are held by L lanes of a warp, P consecutive ones each, so
// that 32 / L tokens share a warp and the reductions over a token's experts are
// log2(L) shuffles. With groups a token has the whole warp and each group a run of
// lanes of its own, whatever the group's size. The K best are taken one after the
// other (largest of the lanes' largest, lowest lane first: lanes hold ascending
// indices, so ties go to the lowest index); lane k keeps the k-th.
//
// The choice is that of the exact scores, not of their fp32 values. Without a bias
// the order is that of the logits and needs no scores. With a bias, or where groups
// are ranked by sums of scores, keys are computed in fp32 first; where two
// neighbours of the result are nearer than the keys' error bound and do not come
// from the same inputs, the warp chooses again with keys in 64 bits. For keys
// spread like a router's that is about one token in a thousand.
//
// Bounds: the logits are read once, 2 or 4 bytes for some 10 instructions a logit and
// 30 a choice: instruction issue for large batches, launch latency for small ones.
#include "block_internal.cuh"

namespace bsmoe {

namespace {

constexpr int kRouteThreads = 128;
constexpr unsigned kFull = 0xffffffffu;

struct Shape {
  int T, E, K, dtype, G, top_groups, group_max, sigmoid, renorm;
  int64_t ld;
  float scale;
  bool vec;  // a lane's logits are whole 16-byte (or, below that, whole power-of-two) loads
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

template <int L, typename V>
__device__ __forceinline__ V lane_max(V v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <int L, typename V>
__device__ __forceinline__ V lane_sum(V v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Where a lane's logits start and how many it has.
struct Span {
  int e0, n;
};
template <int P, int L>
__device__ __forceinline__ Span span_of(const Shape& s, int sub) {
  if (s.G == 1) {
    const int e0 = min(sub * P, s.E);
    return {e0, min(P, s.E - e0)};
  }
  // G <= 32: lanes a group: the largest power of two that fits
  const int lpg = 1 << (31 - __clz(32 / s.G));
  const int size = s.E / s.G, per = (size + lpg - 1) / lpg;
  const int g = sub / lpg;
  if (g >= s.G) return {s.E, 0};
  const int o = min((sub % lpg) * per, size);
  return {g * size + o, min(per, size - o)};
}

template <int P, typename T>
__device__ __forceinline__ void load_as(const void* base, int64_t at, int n, bool vec, float (&x)[P]) {
  const T* p = static_cast<const T*>(base) + at;
  constexpr int W = sizeof(T) * P >= 16 ? 16 / sizeof(T) : P;
  if (vec && n == P) {
#pragma unroll
    for (int i = 0; i < P; i += W) {
      const Pack<T, W> v = load_pack<W>(p + i);
      float f[W];
      unpack(v, f);
#pragma unroll
      for (int j = 0; j < W; ++j) x[i + j] = f[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = i < n ? to_f32(p[i]) : neg_inf();
  }
}
// The lane's logits, -inf behind the last.
template <int P>
__device__ __forceinline__ void load_logits(const Shape& s, const void* logits, int64_t t, Span sp, float (&x)[P]) {
  const int64_t at = t * s.ld + sp.e0;
  if (s.dtype == MOE_BF16) load_as<P, __nv_bfloat16>(logits, at, sp.n, s.vec, x);
  else if (s.dtype == MOE_FP16) load_as<P, __half>(logits, at, sp.n, s.vec, x);
  else load_as<P, float>(logits, at, sp.n, s.vec, x);
}

// e^-|x| / (1 + e^-|x|) forms: s and 1 - s without cancellation.
__device__ __forceinline__ void sigmoid_pair(float x, float* s, float* not_s) {
  const float z = expf(-fabsf(x)), d = __fdividef(1.f, 1.f + z);
  *s = x >= 0.f ? d : z * d;
  *not_s = x >= 0.f ? z * d : d;
}
__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ double sigmoid_exact(double x) { return 1.0 / (1.0 + exp(-x)); }

// Scores up to a common factor, for ratios of them: below -60 sigmoid(x) is e^x in
// fp32, so where the largest logit `most` is there, e^(x - most) keeps the ratios
// of scores that fp32 would not hold.
__device__ __forceinline__ float ratio_score(bool sigmoid, float x, float most) {
  if (!sigmoid) return most == neg_inf() ? 0.f : expf(x - most);
  if (most < -60.f) return most == neg_inf() ? 0.f : expf(x - most);
  float s, n;
  sigmoid_pair(x, &s, &n);
  return s;
}

struct Chosen {
  int idx;      // lane k: the k-th expert, -1 if none is left
  float x;      // its logit
  bool unsure;  // the token's: fp32 keys do not settle the choice
};

// What the lanes of a token know about all its logits.
struct Row {
  float most;  // largest logit
  float sum;   // sum of e^(x - most) (softmax where scores are needed)
};

// The K best of the token's experts. V: type of the keys. `slack`: largest
// error of an fp32 key beside 2^-22 of the key itself.
template <typename V, int P, int L>
__device__ __forceinline__ Chosen choose(const Shape& s, const float (&x)[P], Span sp, const float* bias, Row row,
                                         int sub, float slack) {
  constexpr bool kExact = sizeof(V) == 8;
  const V none = neg_inf();
  V key[P];
  const bool by_score = bias != nullptr || (s.G > 1 && !s.group_max);
  V total = 1;
  if (kExact && by_score && !s.sigmoid) {
    V t = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) t += x[i] > neg_inf() ? exp(static_cast<double>(x[i]) - static_cast<double>(row.most)) : 0.0;
    total = lane_sum<L>(t);
  } else if (by_score && !s.sigmoid) {
    total = __fdividef(1.f, row.sum);
  }
  // q: scores plus bias (what groups are ranked by); key: what experts are
#pragma unroll
  for (int i = 0; i < P; ++i) {
    V q = x[i] + 0.f;  // -0 and 0 are one value
    if (by_score) {
      if constexpr (kExact) {
        q = s.sigmoid ? sigmoid_exact(x[i]) : exp(static_cast<double>(x[i]) - static_cast<double>(row.most)) / total;
        if (bias != nullptr && i < sp.n) q += static_cast<double>(__ldg(bias + sp.e0 + i));
      } else {
        q = s.sigmoid ? sigmoid_fast(x[i]) : __expf(x[i] - row.most) * static_cast<float>(total);
        if (bias != nullptr && i < sp.n) q += __ldg(bias + sp.e0 + i);
      }
    }
    key[i] = i < sp.n && x[i] > neg_inf() && q > none ? q : none;
  }
  bool unsure = false;
  if (s.G > 1) {
    const int lpg = 1 << (31 - __clz(32 / s.G));
    V a = none, b = none;  // largest and second
#pragma unroll
    for (int i = 0; i < P; ++i) {
      b = fmax(b, fmin(a, key[i]));
      a = fmax(a, key[i]);
    }
    for (int o = lpg / 2; o > 0; o >>= 1) {
      const V a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
      b = fmax(fmin(a, a2), fmax(b, b2));
      a = fmax(a, a2);
    }
    const V value = s.group_max || b == none ? a : a + b;
    const int g = sub / lpg;
    int rank = 0;
    for (int j = 0; j < s.G; ++j) {
      const V v = __shfl_sync(kFull, value, j * lpg);
      rank += v > value || (v == value && j < g);
    }
    const bool in = rank < s.top_groups && g < s.G;
    if (!kExact && by_score) {
      const V worst = -lane_max<L>(in ? -value : none), best = lane_max<L>(in || g >= s.G ? none : value);
      unsure = worst - best <= 4.f * slack + 0x1p-20f * (fabsf(worst) + fabsf(best));
    }
    if (bias == nullptr) {  // within the groups the order is that of the logits
#pragma unroll
      for (int i = 0; i < P; ++i) key[i] = key[i] > none ? static_cast<V>(x[i] + 0.f) : none;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = in ? key[i] : none;
  }
  Chosen c = {-1, neg_inf(), unsure};
  V mine = none, last = none;
  int last_idx = -1;
  float last_x = 0.f;
  const bool check = !kExact && bias != nullptr;
  const int rounds = s.K + (check && s.K < s.E ? 1 : 0);
  for (int k = 0; k < rounds; ++k) {
    V best = key[0];
    int at = 0;
    float bx = x[0];
#pragma unroll
    for (int i = 1; i < P; ++i) {
      if (key[i] > best) {
        best = key[i];
        at = i;
        bx = x[i];
      }
    }
    const V top = lane_max<L>(best);
    unsigned who = __ballot_sync(kFull, best == top);
    const int lane = threadIdx.x & 31, first = lane - sub;
    if (L < 32) who = (who >> first) & ((1u << (L & 31)) - 1u);
    const int from = first + __ffs(who) - 1;
    int idx = __shfl_sync(kFull, sp.e0 + at, from);
    const float wx = __shfl_sync(kFull, bx, from);
    if (!(top > none)) idx = -1;
    if (lane == from) {
#pragma unroll
      for (int i = 0; i < P; ++i) key[i] = i == at ? none : key[i];
    }
    if (k == sub && k < s.K) {
      c.idx = idx;
      c.x = idx < 0 ? neg_inf() : wx;
      mine = top;
    }
    if (check) {
      const float gap = last - top;
      if (k > 0 && idx >= 0 && gap <= 2.f * slack + 0x1p-21f * (fabsf(last) + fabsf(top)) &&
          !(wx == last_x && __ldg(bias + idx) == __ldg(bias + last_idx)))
        c.unsure = true;
      last = top;
      last_idx = idx;
      last_x = wx;
    }
  }
  (void)mine;
  return c;
}

template <int P, int L>
__device__ __noinline__ int2 choose_exact(const Shape& s, const float (&x)[P], Span sp, const float* bias, Row row,
                                          int sub) {
  const Chosen c = choose<double, P, L>(s, x, sp, bias, row, sub, 0.f);
  return make_int2(c.idx, __float_as_int(c.x));
}

template <int P, int L>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(Shape s, const void* __restrict__ logits,
                                                              const float* __restrict__ bias, int32_t* __restrict__ idx,
                                                              float* __restrict__ w, float* __restrict__ partials) {
  constexpr int kTokens = kRouteThreads / L;  // a block at a time
  const int lane = threadIdx.x & 31, sub = lane % L;
  const Span sp = span_of<P, L>(s, sub);
  const bool mean = partials != nullptr;
  const bool scores = bias != nullptr || (s.G > 1 && !s.group_max);
  float acc[P];
#pragma unroll
  for (int i = 0; i < P; ++i) acc[i] = 0.f;
  pdl_wait();
  pdl_launch_dependents();
  // every lane walks the same number of tokens: the shuffles take whole warps
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens; t0 < s.T; t0 += static_cast<int64_t>(gridDim.x) * kTokens) {
    const int64_t t = t0 + threadIdx.x / L;
    const bool valid = t < s.T;
    float x[P];
    load_logits<P>(s, logits, valid ? t : s.T - 1, sp, x);
    Row row = {neg_inf(), 1.f};
    bool nan = false;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      row.most = fmaxf(row.most, x[i]);
      nan |= x[i] != x[i];
    }
    row.most = lane_max<L>(row.most);
    unsigned any_nan = __ballot_sync(kFull, nan);
    if (L < 32) any_nan = (any_nan >> (lane - sub)) & ((1u << (L & 31)) - 1u);
    if (!s.sigmoid && (scores || !s.renorm || mean)) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) sum += x[i] > neg_inf() ? __expf(x[i] - row.most) : 0.f;
      row.sum = lane_sum<L>(sum);
    }
    // Errors of an fp32 score: sigmoid: below 3e-7 (its slope times the
    // exponential's 2^-22 and its argument's |x| 2^-23, the sum's and the
    // quotient's roundings); softmax: those of the exponential and of the sum, in
    // all below 1.2e-6 of the largest score.
    const float slack = s.sigmoid ? 4e-7f : __fdividef(1.5e-6f, row.sum);
    Chosen c = choose<float, P, L>(s, x, sp, bias, row, sub, slack);
    if (__any_sync(kFull, c.unsure)) {
      const int2 e = choose_exact<P, L>(s, x, sp, bias, row, sub);
      c.idx = e.x;
      c.x = __int_as_float(e.y);
    }
    float weight;
    const bool have = sub < s.K && c.idx >= 0;
    if (s.renorm) {
      const float most = lane_max<L>(have ? c.x : neg_inf());
      const float score = have ? ratio_score(s.sigmoid, c.x, most) : 0.f;
      const float sum = lane_sum<L>(score);
      weight = have ? score / sum * s.scale : 0.f;
    } else if (s.sigmoid) {
      float sc, n;
      sigmoid_pair(c.x, &sc, &n);
      weight = have ? sc * s.scale : 0.f;
    } else {
      weight = have ? expf(c.x - row.most) / row.sum * s.scale : 0.f;
    }
    if (any_nan) weight = __int_as_float(0x7fffffff);
    if (valid && sub < s.K) {
      idx[t * s.K + sub] = c.idx;
      w[t * s.K + sub] = weight;
    }
    if (mean) {
      float p[P], sum = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (!s.sigmoid) p[i] = x[i] == neg_inf() ? 0.f : __expf(x[i] - row.most);
        else if (row.most < -60.f) p[i] = x[i] == neg_inf() ? 0.f : __expf(x[i] - row.most);
        else p[i] = sigmoid_fast(x[i]);
        sum += p[i];
      }
      sum = lane_sum<L>(sum);
      const float f = valid && sum != 0.f ? __fdividef(1.f, sum) : 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) acc[i] += valid ? p[i] * f : 0.f;
    }
  }
  if (!mean) return;
  // lanes that hold the same experts, then the block's warps, in a fixed order
#pragma unroll
  for (int i = 0; i < P; ++i) {
#pragma unroll
    for (int o = 16; o >= L; o >>= 1) acc[i] += __shfl_xor_sync(kFull, acc[i], o);
  }
  __shared__ float cols[kRouteThreads / 32][kMaxExperts];
  if (lane < L) {
    for (int i = 0; i < P; ++i)
      if (i < sp.n) cols[threadIdx.x / 32][sp.e0 + i] = acc[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < s.E; e += kRouteThreads) {
    float v = 0.f;
    for (int k = 0; k < kRouteThreads / 32; ++k) v += cols[k][e];
    partials[static_cast<size_t>(blockIdx.x) * s.E + e] = v;
  }
}

// mean[e] = sum of the blocks' columns / T: a warp an expert.
__global__ void __launch_bounds__(256) route_mean_kernel(const float* __restrict__ partials, int blocks, int E, float T,
                                                         float* __restrict__ mean) {
  const int e = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  if (e >= E) return;
  float v = 0.f;
  for (int b = lane; b < blocks; b += 32) v += partials[static_cast<size_t>(b) * E + e];
  v = warp_sum(v);
  if (lane == 0) mean[e] = T > 0.f ? v / T : 0.f;
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
template <int P, int L>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(Shape s, const float* __restrict__ dw,
                                                                       const float* __restrict__ dmean,
                                                                       const void* __restrict__ logits,
                                                                       const int32_t* __restrict__ idx, bool vec_out,
                                                                       void* __restrict__ dx) {
  constexpr int kTokens = kRouteThreads / L;
  const int lane = threadIdx.x & 31, sub = lane % L;
  const Span sp = span_of<P, L>(s, sub);
  const bool dense = dmean != nullptr || (!s.sigmoid && !s.renorm);
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
        const int64_t at = tr * s.ld + e;
        xk = s.dtype == MOE_BF16   ? to_f32(static_cast<const __nv_bfloat16*>(logits)[at])
             : s.dtype == MOE_FP16 ? to_f32(static_cast<const __half*>(logits)[at])
                                   : static_cast<const float*>(logits)[at];
      }
    }
    float most = neg_inf(), sum = 0.f;
    if (dense) {
#pragma unroll
      for (int i = 0; i < P; ++i) most = fmaxf(most, x[i]);
      most = lane_max<L>(most);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (!s.sigmoid || most < -60.f) d[i] = x[i] == neg_inf() ? 0.f : __expf(x[i] - most);
        else d[i] = sigmoid_fast(x[i]);
        sum += d[i];
      }
      sum = lane_sum<L>(sum);
    }
    const float inv = sum != 0.f ? __fdividef(1.f, sum) : 0.f;
    // the chosen experts' part: dx += add at expert e
    float add = 0.f, all = 0.f;  // all: <ds, s>, taken off every expert (softmax without renormalisation)
    if (s.renorm) {
      const float top = lane_max<L>(e >= 0 ? xk : neg_inf());
      const float sc = e >= 0 ? ratio_score(s.sigmoid, xk, top) : 0.f;
      const float S = lane_sum<L>(sc);
      const float wn = S != 0.f ? sc / S : 0.f;
      const float inner = lane_sum<L>(e >= 0 ? v * wn : 0.f);
      add = e >= 0 ? wn * (v - inner) : 0.f;
      if (s.sigmoid) {
        float a, b;
        sigmoid_pair(xk, &a, &b);
        add *= b;
      }
    } else if (s.sigmoid) {
      float a, b;
      sigmoid_pair(xk, &a, &b);
      add = e >= 0 ? v * a * b : 0.f;
    } else {
      const float sc = e >= 0 && most > neg_inf() ? expf(xk - most) * inv : 0.f;
      add = e >= 0 ? v * sc : 0.f;
      all = lane_sum<L>(add);
    }
    if (dense) {
      float h[P], inner = 0.f;
      if (dmean != nullptr) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          h[i] = i < sp.n ? __ldg(dmean + sp.e0 + i) * inv_T : 0.f;
          inner += d[i] * inv * h[i];
        }
        inner = lane_sum<L>(inner);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float g = -all;
        if (dmean != nullptr) g += h[i] - inner;
        float v = d[i] * inv * g;
        if (s.sigmoid) {
          float a, b;
          sigmoid_pair(x[i], &a, &b);
          v *= b;
        }
        d[i] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) d[i] = 0.f;
    }
    for (int k = 0; k < s.K; ++k) {
      const int ek = __shfl_sync(kFull, e, lane - sub + k);
      const float ak = __shfl_sync(kFull, add, lane - sub + k);
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i < sp.n && sp.e0 + i == ek) d[i] += ak;
    }
    if (valid) {
      const int64_t at = t * s.E + sp.e0;
      if (s.dtype == MOE_BF16) store_as<P, __nv_bfloat16>(dx, at, sp.n, vec_out, d);
      else if (s.dtype == MOE_FP16) store_as<P, __half>(dx, at, sp.n, vec_out, d);
      else store_as<P, float>(dx, at, sp.n, vec_out, d);
    }
  }
}

// Lanes a token and logits a lane: at least K lanes (lane k keeps the k-th
// choice), at most 8 logits a lane where 32 lanes allow it.
struct Split {
  int L, P;
};
Split split_of(int E, int K, int G) {
  auto pow2 = [](int v) {
    int p = 1;
    while (p < v) p *= 2;
    return p;
  };
  if (G > 1) {
    int lpg = 1;
    while (lpg * 2 * G <= 32) lpg *= 2;
    const int per = ceil_div(E / G, lpg);
    return {32, per <= 8 ? 8 : per <= 16 ? 16 : 32};
  }
  const int L = pow2(ceil_div(E, 8) > K ? ceil_div(E, 8) : K) > 32 ? 32 : pow2(ceil_div(E, 8) > K ? ceil_div(E, 8) : K);
  const int per = ceil_div(E, L);
  return {L, per <= 2 ? 2 : per <= 4 ? 4 : per <= 8 ? 8 : 16};
}

// Calls f(P, L) with the split's constants.
template <typename F>
cudaError_t with_split(Split sp, F&& f) {
  using std::integral_constant;
#define BSMOE_SPLIT(p, l) \
  if (sp.P == p && sp.L == l) return f(integral_constant<int, p>(), integral_constant<int, l>());
#define BSMOE_SPLITS(l) BSMOE_SPLIT(2, l) BSMOE_SPLIT(4, l) BSMOE_SPLIT(8, l)
  BSMOE_SPLITS(1) BSMOE_SPLITS(2) BSMOE_SPLITS(4) BSMOE_SPLITS(8) BSMOE_SPLITS(16) BSMOE_SPLITS(32)
  BSMOE_SPLIT(16, 32) BSMOE_SPLIT(32, 32)
#undef BSMOE_SPLITS
#undef BSMOE_SPLIT
  return cudaErrorInvalidValue;
}

Shape shape_of(int dtype, const RouteArgs& a, const void* vec_ptr, int64_t ld, Split sp) {
  Shape s = {a.T, a.E, a.K, dtype, a.G, a.top_groups, a.group_max, a.sigmoid, a.renorm, a.ld, a.scale, false};
  const int es = dtype == MOE_FP32 ? 4 : 2, bytes = sp.P * es < 16 ? sp.P * es : 16;
  // a lane's run starts at a multiple of its load's width and is a whole number of them
  const int lpg = a.G == 1 ? sp.L : 1 << (31 - __builtin_clz(32 / a.G));
  const int run = a.G == 1 ? sp.P : ceil_div(a.E / a.G, lpg);
  s.vec = run == sp.P && (a.G == 1 || a.E / a.G == run * lpg) && reinterpret_cast<uintptr_t>(vec_ptr) % bytes == 0 &&
          ld * es % bytes == 0;
  return s;
}

int route_blocks(const RouteArgs& a, Split sp, int num_sms) {
  const int64_t need = (static_cast<int64_t>(a.T) * sp.L + kRouteThreads - 1) / kRouteThreads;
  const int64_t most = a.mean != nullptr ? kRouteParts : 16 * num_sms;
  return static_cast<int>(need < most ? need : most);
}

}  // namespace

cudaError_t launch_route_tokens(int dtype, const RouteArgs& a, int num_sms, cudaStream_t st) {
  const Split sp = split_of(a.E, a.K, a.G);
  const Shape s = shape_of(dtype, a, a.logits, a.ld, sp);
  const int blocks = route_blocks(a, sp, num_sms);
  if (blocks > 0) {
    const cudaError_t e = with_split(sp, [&](auto P, auto L) {
      return launch_kernel(false, route_kernel<decltype(P)::value, decltype(L)::value>, blocks, kRouteThreads, 0, st, s,
                           a.logits, a.bias, a.idx, a.w, a.mean != nullptr ? a.partials : nullptr);
    });
    if (e != cudaSuccess) return e;
  }
  if (a.mean == nullptr) return cudaSuccess;
  return launch_kernel(true, route_mean_kernel, ceil_div(a.E, 8), 256, 0, st, static_cast<const float*>(a.partials),
                       blocks, a.E, static_cast<float>(a.T), a.mean);
}

cudaError_t launch_route_tokens_backward(int dtype, const RouteArgs& a, const float* dw, const float* dmean, void* dx,
                                         int num_sms, cudaStream_t st) {
  const Split sp = split_of(a.E, a.K, 1);
  const Shape s = shape_of(dtype, a, a.logits, a.ld, sp);
  const bool vec_out = shape_of(dtype, a, dx, a.E, sp).vec;
  return with_split(sp, [&](auto P, auto L) {
    return launch_kernel(false, route_backward_kernel<decltype(P)::value, decltype(L)::value>,
                         route_blocks(a, sp, num_sms), kRouteThreads, 0, st, s, dw, dmean, a.logits,
                         static_cast<const int32_t*>(a.idx), vec_out, dx);
  });
}

}  // namespace bsmoe
