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

// What the lanes of a token know about all its logits.
struct Row {
  float most;  // largest logit
  float sum;   // sum of e^(x - most), where softmax scores are needed
};

// A monotone map of floats to whole numbers above 0, and back.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int64_t ordered(double v) {
  const int64_t u = __double_as_longlong(v);
  return u ^ static_cast<int64_t>(static_cast<uint64_t>(u >> 63) >> 1);
}
constexpr int64_t kNone64 = INT64_MIN;  // below the image of every number

template <int L>
__device__ __forceinline__ uint32_t lane_max_u32(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(kFull, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
    return v;
  }
}
// The lowest lane of the token for which `mine` holds.
template <int L>
__device__ __forceinline__ int first_lane(bool mine, int first) {
  unsigned who = __ballot_sync(kFull, mine);
  if (L < 32) who = (who >> first) & ((1u << (L & 31)) - 1u);
  return first + __ffs(who) - 1;
}

// Descending sort of a lane's keys (Batcher's odd-even merge network).
template <int P>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[P]) {
#pragma unroll
  for (int p = 1; p < P; p *= 2) {
#pragma unroll
    for (int q = p; q > 0; q /= 2) {
#pragma unroll
      for (int j = q % p; j + q < P; j += 2 * q) {
#pragma unroll
        for (int i = 0; i < q; ++i) {
          const int a = i + j, b = i + j + q;
          if (b < P && a / (2 * p) == b / (2 * p)) {
            const uint32_t hi = max(k[a], k[b]), lo = min(k[a], k[b]);
            k[a] = hi;
            k[b] = lo;
          }
        }
      }
    }
  }
}

// fp32 scores plus bias of a lane's experts, NaN or -inf where one is not available.
// Errors of an fp32 score: sigmoid: below 3e-7 (its slope times the exponential's
// 2^-22 and its argument's |x| 2^-23, the sum's and the quotient's roundings);
// softmax: those of the exponential and of the sum, in all below 1.2e-6 of the
// largest score. `score_slack` is above both.
__device__ __forceinline__ float score_slack(const Shape& s, Row row) {
  return s.sigmoid ? 4e-7f : __fdividef(1.5e-6f, row.sum);
}
template <int P>
__device__ __forceinline__ void add_bias(const float* bias, Span sp, bool vec, float (&q)[P]) {
  float b[P];
  load_as<P, float>(bias, sp.e0, sp.n, vec, b);
#pragma unroll
  for (int i = 0; i < P; ++i) q[i] += b[i];
}

// 64-bit scores of a few of a lane's experts (bits of `need`) into keys. All lanes call it.
template <int P>
__device__ __forceinline__ void exact_keys(const Shape& s, const float (&x)[P], Span sp, const float* bias, float most,
                                           double total, unsigned need, int64_t (&key)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) key[i] = kNone64;
  while (__any_sync(kFull, need != 0)) {
    const int at = need != 0 ? __ffs(need) - 1 : 0;
    float xv = x[0];
#pragma unroll
    for (int i = 1; i < P; ++i) xv = i == at ? x[i] : xv;
    const double e = exp(s.sigmoid ? -static_cast<double>(xv) : static_cast<double>(xv) - static_cast<double>(most));
    double q = s.sigmoid ? 1.0 / (1.0 + e) : e / total;
    if (bias != nullptr && at < sp.n) q += static_cast<double>(__ldg(bias + sp.e0 + at));
    const int64_t k = ordered(q);
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = need != 0 && i == at ? k : key[i];
    need &= need - 1;
  }
}

template <int L>
__device__ __forceinline__ int64_t lane_max_i64(int64_t v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    const int64_t w = __shfl_xor_sync(kFull, v, o);
    v = v > w ? v : w;
  }
  return v;
}

// The choice with keys in 64 bits: the whole warp calls it where a token of it is
// unsure. Only experts whose fp32 key is within its error of the border get one.
// Returns the index of the sub-th choice.
template <int P, int L>
__device__ __noinline__ int choose_exact(Shape s, const void* logits, int64_t t, const float* bias, Row row, int sub) {
  const int first = (threadIdx.x & 31) - sub;
  const Span sp = span_of<P, L>(s, sub);
  const bool by_score = bias != nullptr || (s.G > 1 && !s.group_max);
  const float slack = score_slack(s, row);
  float x[P], q[P];
  load_logits<P>(s, logits, t, sp, x);
  double total = 1;
  if (by_score && !s.sigmoid) {
    double sum = 0;
#pragma unroll 1
    for (int i = 0; i < P; ++i) {
      float xv = x[0];
#pragma unroll
      for (int j = 1; j < P; ++j) xv = j == i ? x[j] : xv;
      sum += xv > neg_inf() ? exp(static_cast<double>(xv) - static_cast<double>(row.most)) : 0.0;
    }
    total = lane_sum<L>(sum);
  }
  const float inv = by_score && !s.sigmoid ? __fdividef(1.f, row.sum) : 1.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    q[i] = x[i] + 0.f;
    if (by_score) q[i] = s.sigmoid ? sigmoid_fast(x[i]) : __expf(x[i] - row.most) * inv;
  }
  if (bias != nullptr) add_bias<P>(bias, sp, false, q);
#pragma unroll
  for (int i = 0; i < P; ++i) q[i] = i < sp.n && x[i] > neg_inf() && q[i] > neg_inf() ? q[i] : neg_inf();
  int64_t key[P];
  // the experts that may reach a border at `edge`
  auto near = [&](float edge) {
    const float from = fabsf(edge) < INFINITY ? edge - 4.f * slack - 0x1p-20f * fabsf(edge) : edge;
    unsigned need = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) need |= static_cast<unsigned>(q[i] > neg_inf() && q[i] >= from) << i;
    return need;
  };
  if (s.G > 1) {
    const int lpg = 1 << (31 - __clz(32 / s.G));
    float a = neg_inf(), b = neg_inf();
#pragma unroll
    for (int i = 0; i < P; ++i) {
      b = fmaxf(b, fminf(a, q[i]));
      a = fmaxf(a, q[i]);
    }
    for (int o = lpg / 2; o > 0; o >>= 1) {
      const float a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
      b = fmaxf(fminf(a, a2), fmaxf(b, b2));
      a = fmaxf(a, a2);
    }
    if (by_score) {
      exact_keys<P>(s, x, sp, bias, row.most, total, near(s.group_max ? a : b), key);
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) key[i] = q[i] > neg_inf() ? ordered(static_cast<double>(q[i])) : kNone64;
    }
    int64_t c = kNone64, d = kNone64;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int64_t lo = key[i] < c ? key[i] : c;
      d = d > lo ? d : lo;
      c = c > key[i] ? c : key[i];
    }
    for (int o = lpg / 2; o > 0; o >>= 1) {
      const int64_t c2 = __shfl_xor_sync(kFull, c, o), d2 = __shfl_xor_sync(kFull, d, o);
      const int64_t lo = c < c2 ? c : c2, hi = d > d2 ? d : d2;
      d = lo > hi ? lo : hi;
      c = c > c2 ? c : c2;
    }
    auto value_of = [](int64_t o) { return __longlong_as_double(o ^ static_cast<int64_t>(static_cast<uint64_t>(o >> 63) >> 1)); };
    const int64_t value = s.group_max || d == kNone64 ? c : ordered(value_of(c) + value_of(d));
    const int g = sub / lpg;
    int rank = 0;
    for (int j = 0; j < s.G; ++j) {
      const int64_t v = __shfl_sync(kFull, value, j * lpg);
      rank += v > value || (v == value && j < g);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) q[i] = rank < s.top_groups && g < s.G ? q[i] : neg_inf();
  }
  // the K-th fp32 key, then 64-bit keys from there up
  float edge = neg_inf();
  {
    uint32_t k[P];
#pragma unroll
    for (int i = 0; i < P; ++i) k[i] = q[i] > neg_inf() ? ordered(q[i] + 0.f) : 0u;
    for (int r = 0; r < s.K; ++r) {
      uint32_t best = k[0];
      int at = 0;
#pragma unroll
      for (int i = 1; i < P; ++i) {
        at = k[i] > best ? i : at;
        best = max(best, k[i]);
      }
      const uint32_t top = lane_max_u32<L>(best);
      const bool mine = first + sub == first_lane<L>(best == top, first);
#pragma unroll
      for (int i = 0; i < P; ++i) k[i] = mine && i == at ? 0u : k[i];
      edge = top != 0 ? unordered(top) : neg_inf();
    }
  }
  if (bias != nullptr) {
    exact_keys<P>(s, x, sp, bias, row.most, total, near(edge), key);
  } else {  // the order is that of the logits
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = q[i] > neg_inf() ? static_cast<int64_t>(ordered(x[i] + 0.f)) : kNone64;
  }
  int chosen = -1;
  for (int r = 0; r < s.K; ++r) {
    int64_t best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < P; ++i) {
      at = key[i] > best ? i : at;
      best = key[i] > best ? key[i] : best;
    }
    const int64_t top = lane_max_i64<L>(best);
    const int from = first_lane<L>(best == top, first);
    const int idx = __shfl_sync(kFull, sp.e0 + at, from);
    if (r == sub) chosen = top != kNone64 ? idx : -1;
    const bool mine = first + sub == from;
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = mine && i == at ? kNone64 : key[i];
  }
  return chosen;
}

__device__ __forceinline__ float logit_at(const Shape& s, const void* logits, int64_t at) {
  return s.dtype == MOE_BF16   ? to_f32(static_cast<const __nv_bfloat16*>(logits)[at])
         : s.dtype == MOE_FP16 ? to_f32(static_cast<const __half*>(logits)[at])
                               : static_cast<const float*>(logits)[at];
}

// Over the first `width` lanes of a token (a power of two), valid in these.
__device__ __forceinline__ float head_max(float v, int width) {
  for (int o = width / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float head_sum(float v, int width) {
  for (int o = width / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Keys of the fast choice: the fp32 key as a whole number, its low log2(P) bits
// replaced by the expert's place in the lane (lower places larger). A lane sorts
// its keys once; a round is then one maximum over the lanes' heads, and the lane that
// has it moves up. What the cut bits and the scores' errors leave open
// is found afterwards, between neighbours of the result.
template <int P, int L, bool MEAN>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(Shape s, const void* __restrict__ logits,
                                                              const float* __restrict__ bias, int32_t* __restrict__ idx,
                                                              float* __restrict__ w, float* __restrict__ partials) {
  constexpr int kTokens = kRouteThreads / L;  // a block at a time
  constexpr float kCut = P * 0x1p-22f;        // of a key: the cut bits, and its own rounding
  const int lane = threadIdx.x & 31, sub = lane % L, first = lane - sub;
  const Span sp = span_of<P, L>(s, sub);
  const bool by_score = bias != nullptr || (s.G > 1 && !s.group_max);
  const bool softmax_sum = !s.sigmoid && (by_score || !s.renorm || MEAN);
  // 16-bit logits keep all their bits in a key
  const bool check = by_score || s.dtype == MOE_FP32;
  const int rounds = s.K + (check && s.K < s.E ? 1 : 0);
  const int width = s.K > 1 ? 2 << (31 - __clz(s.K - 1)) : 1;
  const bool vec_bias = bias != nullptr && s.vec_bias;
  float acc[MEAN ? P : 1];
  if constexpr (MEAN) {
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i] = 0.f;
  }
  pdl_wait();
  pdl_launch_dependents();
  // every lane walks the same number of tokens: the shuffles take whole warps
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens; t0 < s.T; t0 += static_cast<int64_t>(gridDim.x) * kTokens) {
    const int64_t t = t0 + threadIdx.x / L;
    const bool valid = t < s.T;
    const int64_t tr = valid ? t : s.T - 1;
    float x[P], q[P];  // logits; scores (softmax: times their sum)
    load_logits<P>(s, logits, tr, sp, x);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < P; ++i) nan |= x[i] != x[i];
    unsigned any_nan = __ballot_sync(kFull, nan);
    if (L < 32) any_nan = (any_nan >> first) & ((1u << (L & 31)) - 1u);
    Row row = {neg_inf(), 1.f};
    if (softmax_sum) {
#pragma unroll
      for (int i = 0; i < P; ++i) row.most = fmaxf(row.most, x[i]);
      row.most = lane_max<L>(row.most);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        q[i] = x[i] > neg_inf() ? __expf(x[i] - row.most) : 0.f;
        sum += q[i];
      }
      row.sum = lane_sum<L>(sum);
    } else if (s.sigmoid && (by_score || MEAN)) {
#pragma unroll
      for (int i = 0; i < P; ++i) q[i] = sigmoid_fast(x[i]);
    }
    uint32_t key[P];
    {
      float v[P];
      const float inv = by_score && !s.sigmoid ? __fdividef(1.f, row.sum) : 1.f;
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = by_score ? q[i] * inv : x[i];
      if (bias != nullptr) add_bias<P>(bias, sp, vec_bias, v);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const bool ok = x[i] > neg_inf() && v[i] > neg_inf();  // -inf behind the lane's last
        key[i] = ok ? (ordered(v[i] + 0.f) & ~static_cast<uint32_t>(P - 1)) | (P - 1 - i) : 0u;
      }
    }
    sort_keys<P>(key);
    const float slack = by_score ? score_slack(s, row) : 0.f;
    bool unsure = false;
    if (s.G > 1) {
      const int lpg = 1 << (31 - __clz(32 / s.G));
      uint32_t a = key[0], b = key[P > 1 ? 1 : 0];
      for (int o = lpg / 2; o > 0; o >>= 1) {
        const uint32_t a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
        b = max(min(a, a2), max(b, b2));
        a = max(a, a2);
      }
      const float va = a != 0 ? unordered(a & ~static_cast<uint32_t>(P - 1)) : neg_inf();
      const float vb = s.group_max || b == 0 ? 0.f : unordered(b & ~static_cast<uint32_t>(P - 1));
      const float value = va + vb;
      const int g = sub / lpg;
      int rank = 0;
      for (int j = 0; j < s.G; ++j) {
        const float v = __shfl_sync(kFull, value, j * lpg);
        rank += v > value || (v == value && j < g);
      }
      const bool in = rank < s.top_groups && g < s.G;
      if (check && s.top_groups < s.G) {
        const float err = 2.f * slack + kCut * (fabsf(va) + fabsf(vb));
        const float worst = -lane_max<L>(in ? err - value : neg_inf());
        const float best = lane_max<L>(in || g >= s.G ? neg_inf() : value + err);
        unsure = worst <= best;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) key[i] = in ? key[i] : 0u;
    }
    // lane k keeps the k-th key and the lane that had it; `next`: the one behind the last lane's
    uint32_t mine = 0, next = 0;
    int from_k = lane, from_next = lane;
    for (int k = 0; k < rounds; ++k) {
      // between lanes the places do not count: equal keys go to the lowest lane
      const uint32_t head = key[0] & ~static_cast<uint32_t>(P - 1);
      const int from = first_lane<L>(head == lane_max_u32<L>(head), first);
      const uint32_t top = __shfl_sync(kFull, key[0], from);
      if (k == sub) {
        mine = top;
        from_k = from;
      }
      if (k == L) {
        next = top;
        from_next = from;
      }
      if (lane == from) {
#pragma unroll
        for (int i = 0; i + 1 < P; ++i) key[i] = key[i + 1];
        key[P - 1] = 0u;
      }
    }
    const int place = P - 1 - static_cast<int>(mine & (P - 1));
    int e = __shfl_sync(kFull, sp.e0, from_k) + place;
    if (mine == 0) e = -1;
    float xe = e >= 0 ? logit_at(s, logits, tr * s.ld + e) : neg_inf();
    if (check) {
      float be = e >= 0 && bias != nullptr ? __ldg(bias + e) : 0.f;
      // the neighbour behind: the next lane's, or the extra one
      uint32_t after = __shfl_sync(kFull, mine, (lane + 1) & 31);
      float xa = __shfl_sync(kFull, xe, (lane + 1) & 31), ba = __shfl_sync(kFull, be, (lane + 1) & 31);
      const int ea = __shfl_sync(kFull, sp.e0, from_next) + P - 1 - static_cast<int>(next & (P - 1));
      if (sub == L - 1) {
        after = next;
        if (next != 0) {
          xa = logit_at(s, logits, tr * s.ld + ea);
          ba = bias != nullptr ? __ldg(bias + ea) : 0.f;
        }
      }
      if (sub < s.K && sub + 1 < rounds && mine != 0 && after != 0) {
        const float a = unordered(mine & ~static_cast<uint32_t>(P - 1)), b = unordered(after & ~static_cast<uint32_t>(P - 1));
        const float err = by_score ? 2.f * slack + kCut * (fabsf(a) + fabsf(b)) : 0.f;
        unsure |= a - b <= err && !(xe == xa && be == ba);
      }
      if (__any_sync(kFull, unsure)) {
        e = choose_exact<P, L>(s, logits, tr, bias, row, sub);
        if (sub >= s.K) e = -1;
        xe = e >= 0 ? logit_at(s, logits, tr * s.ld + e) : neg_inf();
      }
    }
    const bool have = sub < s.K && e >= 0;
    float weight = 0.f;
    if (s.sigmoid) {
      float score = 0.f, n;
      if (have) sigmoid_pair(xe, &score, &n);
      if (s.renorm) {
        float sum = head_sum(score, width);
        if (__any_sync(kFull, sub < width && sum < 1e-20f)) {  // below fp32's range the ratios are those of e^x
          const float most = head_max(have ? xe : neg_inf(), width);
          const float low = have ? ratio_score(true, xe, most) : 0.f;
          const float low_sum = head_sum(low, width);
          if (sum < 1e-20f) {
            score = low;
            sum = low_sum;
          }
        }
        score = have ? score / sum : 0.f;
      }
      weight = score * s.scale;
    } else if (s.renorm) {
      const float most = head_max(have ? xe : neg_inf(), width);
      const float score = have ? expf(xe - most) : 0.f;
      const float sum = head_sum(score, width);
      weight = have ? score / sum * s.scale : 0.f;
    } else {
      weight = have ? expf(xe - row.most) / row.sum * s.scale : 0.f;
    }
    if (any_nan) weight = __int_as_float(0x7fffffff);
    if (valid && sub < s.K) {
      idx[t * s.K + sub] = e;
      w[t * s.K + sub] = weight;
    }
    if constexpr (MEAN) {
      float sum = row.sum;
      if (s.sigmoid) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) sum += q[i];
        sum = lane_sum<L>(sum);
        if (__any_sync(kFull, sum < 1e-20f)) {
          float most = neg_inf(), low = 0.f;
#pragma unroll
          for (int i = 0; i < P; ++i) most = fmaxf(most, x[i]);
          most = lane_max<L>(most);
          const bool small = sum < 1e-20f;
#pragma unroll
          for (int i = 0; i < P; ++i) {
            if (small) q[i] = x[i] == neg_inf() ? 0.f : __expf(x[i] - most);
            low += q[i];
          }
          low = lane_sum<L>(low);
          if (small) sum = low;
        }
      }
      if (any_nan) sum = __int_as_float(0x7fffffff);
      const float f = sum != 0.f ? __fdividef(1.f, sum) : 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) acc[i] += valid ? q[i] * f : 0.f;
    }
  }
  if constexpr (MEAN) {
    // lanes that hold the same experts, then the block's warps, in a fixed order
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int o = 16; o >= L; o >>= 1) acc[i] += __shfl_xor_sync(kFull, acc[i], o);
    }
    __shared__ float cols[kRouteThreads / 32][kMaxExperts];
    if (lane < L) {
#pragma unroll
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
        if (s.sigmoid) d[i] *= sigmoid_fast(-x[i]);
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
      float p = !s.sigmoid || most < -60.f ? __expf(xk - most) : sigmoid_fast(xk);
      p *= inv * ((dmean != nullptr ? (__ldg(dmean + e) - inner) * inv_T : 0.f) - all);
      if (s.sigmoid) p *= sigmoid_fast(-xk);
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
  Shape s = {a.T, a.E, a.K, dtype, a.G, a.top_groups, a.group_max, a.sigmoid, a.renorm, a.ld, a.scale, false, false};
  const int es = dtype == MOE_FP32 ? 4 : 2, bytes = sp.P * es < 16 ? sp.P * es : 16;
  // a lane's run starts at a multiple of its load's width and is a whole number of them
  const int lpg = a.G == 1 ? sp.L : 1 << (31 - __builtin_clz(32 / a.G));
  const int run = a.G == 1 ? sp.P : ceil_div(a.E / a.G, lpg);
  s.vec = run == sp.P && (a.G == 1 || a.E / a.G == run * lpg) && reinterpret_cast<uintptr_t>(vec_ptr) % bytes == 0 &&
          ld * es % bytes == 0;
  const int bias_bytes = sp.P * 4 < 16 ? sp.P * 4 : 16;
  s.vec_bias = run == sp.P && (a.G == 1 || a.E / a.G == run * lpg) && reinterpret_cast<uintptr_t>(a.bias) % bias_bytes == 0;
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
      constexpr int p = decltype(P)::value, l = decltype(L)::value;
      return launch_kernel(false, a.mean != nullptr ? route_kernel<p, l, true> : route_kernel<p, l, false>, blocks,
                           kRouteThreads, 0, st, s, a.logits, a.bias, a.idx, a.w, a.partials);
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
  Shape s = shape_of(dtype, a, a.logits, a.ld, sp);
  s.vec_bias = s.vec_bias && reinterpret_cast<uintptr_t>(dmean) % 16 == 0;  // dmean is read as a bias is
  const bool vec_out = shape_of(dtype, a, dx, a.E, sp).vec;
  return with_split(sp, [&](auto P, auto L) {
    return launch_kernel(false, route_backward_kernel<decltype(P)::value, decltype(L)::value>,
                         route_blocks(a, sp, num_sms), kRouteThreads, 0, st, s, dw, dmean, a.logits,
                         static_cast<const int32_t*>(a.idx), vec_out, dx);
  });
}

}  // namespace bsmoe
