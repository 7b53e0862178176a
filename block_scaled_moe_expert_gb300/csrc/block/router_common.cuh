// Routing: what the forward and the gradient share.
//
// A token's E logits are held by L lanes of a warp, P consecutive ones each, so
// that 32 / L tokens share a warp and the reductions over a token's experts are
// log2(L) shuffles. With groups a token has the whole warp and each group a run of
// lanes of its own, whatever the group's size.
#pragma once
#include <type_traits>

#include "block_internal.cuh"

namespace bsmoe {

namespace {

constexpr int kRouteThreads = 128;
constexpr unsigned kFull = 0xffffffffu;

struct Shape {
  int T, E, K, dtype, G, top_groups, group_max, renorm;
  int lanes_log2, size, per;  // of a group: lanes (their logarithm), experts, experts a lane
  int64_t ld;
  float scale;
  bool vec;       // a lane's logits are whole 16-byte (or, below that, whole power-of-two) loads
  bool vec_bias;  // and its biases
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
__device__ __forceinline__ Span span_of(const Shape& s, int sub) {
  const int g = sub >> s.lanes_log2;
  if (g >= s.G) return {s.E, 0};
  const int o = min((sub & ((1 << s.lanes_log2) - 1)) * s.per, s.size);
  return {g * s.size + o, min(s.per, s.size - o)};
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

__device__ __forceinline__ float logit_at(const Shape& s, const void* logits, int64_t at) {
  return s.dtype == MOE_BF16   ? to_f32(static_cast<const __nv_bfloat16*>(logits)[at])
         : s.dtype == MOE_FP16 ? to_f32(static_cast<const __half*>(logits)[at])
                               : static_cast<const float*>(logits)[at];
}

// 2^-22 of the value, and 1.5 |x| 2^-24 from the rounding of the argument; subnormal results as 0.
__device__ __forceinline__ float exp_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
// 2^-23 of the value.
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_fast(1.f + exp_fast(-x)); }
// s and 1 - s without cancellation.
__device__ __forceinline__ void sigmoid_pair(float x, float* s, float* not_s) {
  const float z = expf(-fabsf(x)), d = __fdividef(1.f, 1.f + z);
  *s = x >= 0.f ? d : z * d;
  *not_s = x >= 0.f ? z * d : d;
}
// Scores up to a common factor, for ratios of them: below -60 sigmoid(x) is e^x in
// fp32, so where the largest logit `most` is there, e^(x - most) keeps the ratios
// of scores that fp32 would not hold.
template <bool SIGMOID>
__device__ __forceinline__ float ratio_score(float x, float most) {
  if (!SIGMOID || most < -60.f) return most == neg_inf() ? 0.f : expf(x - most);
  float s, n;
  sigmoid_pair(x, &s, &n);
  return s;
}

// Lanes a token and logits a lane: at most 8 logits a lane where 32 lanes allow it.
struct Split {
  int L, P;
};
inline Split split_of(int E, int K, int G) {
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
  // lane k keeps the k-th choice, lane K the one behind the last
  const int lanes = pow2(ceil_div(E, 8)), choices = pow2(K < E ? K + 1 : K);
  int L = lanes > choices ? lanes : choices;
  L = L < 2 ? 2 : L > 32 ? 32 : L;
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
  BSMOE_SPLITS(2) BSMOE_SPLITS(4) BSMOE_SPLITS(8) BSMOE_SPLITS(16) BSMOE_SPLITS(32)
  BSMOE_SPLIT(16, 32) BSMOE_SPLIT(32, 32)
#undef BSMOE_SPLITS
#undef BSMOE_SPLIT
  return cudaErrorInvalidValue;
}

inline Shape shape_of(int dtype, const RouteArgs& a, const void* vec_ptr, int64_t ld, Split sp) {
  int lanes = sp.L;  // of a group: with groups the largest power of two that fits
  if (a.G > 1)
    for (lanes = 1; lanes * 2 * a.G <= 32;) lanes *= 2;
  const int size = a.E / a.G, per = a.G == 1 ? sp.P : ceil_div(size, lanes);
  const int es = dtype == MOE_FP32 ? 4 : 2, bytes = sp.P * es < 16 ? sp.P * es : 16;
  const int bias_bytes = sp.P * 4 < 16 ? sp.P * 4 : 16;
  // a lane's run starts at a multiple of its load's width and is a whole number of them
  const bool whole = per == sp.P && (a.G == 1 || size == per * lanes);
  Shape s = {a.T, a.E, a.K, dtype, a.G, a.top_groups, a.group_max, a.renorm, 0, size, per, a.ld, a.scale, false, false};
  while (1 << s.lanes_log2 < lanes) ++s.lanes_log2;
  s.vec = whole && reinterpret_cast<uintptr_t>(vec_ptr) % bytes == 0 && ld * es % bytes == 0;
  s.vec_bias = whole && reinterpret_cast<uintptr_t>(a.bias) % bias_bytes == 0;
  return s;
}

inline int route_blocks(const RouteArgs& a, Split sp, int most) {
  const int64_t need = (static_cast<int64_t>(a.T) * sp.L + kRouteThreads - 1) / kRouteThreads;
  return static_cast<int>(need < most ? need : most);
}

}  // namespace

}  // namespace bsmoe
