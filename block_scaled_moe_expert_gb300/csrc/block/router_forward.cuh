// The router's choice of experts, its weights and mean scores (moe_route_tokens), for
// one kind of score.
//
// The K best are taken one after the other (largest of the lanes' largest, lowest
// lane first: lanes hold ascending indices, so ties go to the lowest index); lane k
// keeps the k-th. Keys are fp32 as whole numbers, the low log2(P) bits replaced by the
// expert's place in the lane (lower places larger): a lane sorts its keys once, a
// round is one maximum over the lanes' heads, and the lane that has it moves up.
//
// The choice is that of the exact scores. Without a bias the order is that of the
// logits. With a bias, or where groups are ranked by sums of scores, neighbours of the
// result that are nearer than the keys' error and do not come from the same inputs
// are settled by pairs of floats (about 2^-43 of the scores), in the lanes that hold them; what
// pairs leave open, or needs experts that no lane holds yet, by 64 bits. Of a million tokens
// with 256 sigmoid scores of normal logits and a bias one in 410 took the first way (with 8
// groups one in 510, and one in 4500 for the groups), none the second.
//
// Bounds: the logits are read once, 2 or 4 bytes for what a lane does to sort its 8 and to pass
// through the rounds (369 instructions a token of 256 logits and one choice), most of it comparisons,
// selections and whole numbers: instruction issue for large batches (issue slots 58% busy, memory at
// a fifth of its rate), the launch for small ones. A call among others, 65536 x 256 fp32: one expert by
// sigmoid 36.3 us, eight with a bias 50.7, in groups 61.6 (67 MB: 10 us at the memory's rate);
// 8192 x 256 in groups 10.5; 16384 x 128 bf16 with mean scores 11.1 (their second launch included);
// 4 tokens 5.4, the kernel 3.2. Registers for 7 blocks per SM, chosen with 8 logits a lane: with 6, 7, 8 and 10
// blocks 8192 x 256 in groups took 11.3, 10.0, 11.4 and 12.4 us. 16 logits a lane spill 400 to 500 bytes
// (8192 x 384 24.6 us, 8192 x 512 in 16 groups 32.2), 32 a lane some 1600 (8192 x 510 in 17 groups 110).
#pragma once
#include <cfloat>

#include "router_common.cuh"

namespace bsmoe {

namespace {

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
// Errors of an fp32 score, in units u = 2^-24. ex2.approx is good to 4 u of its value, its argument x log2(e)
// adds 1.5 |x| u, the subtraction of the largest logit |x| u; rcp.approx is good to 2 u.
// Sigmoid: 4 u and 1.5 |x| u times s (1 - s), u of 1 + e^-x, 2 u of the quotient: below 4.4 u.
// Softmax, of the largest score 1 / sum: 4 u and 2.5 |x| u times e^-|x| (at most 0.92 u), the expert's
// own; and what all of a token's scores have in common: 2 u of the quotient, the same of the terms
// of the sum (4 u and 2.5 u times at most 3.9, the mean |x| of 511 terms beside one of 1 weighted by
// them), P - 1 + log2(L) <= P + 4 roundings of the sum. That part moves the difference of two keys by
// no more than itself, so half of it goes to each: 4.92 + (P + 19.75) / 2 u, and 1 u for what is
// of second order.
template <int P, bool SIGMOID>
__device__ __forceinline__ float score_slack(Row row) {
  return SIGMOID ? 5.f * 0x1p-24f : (16.f + 0.5f * P) * 0x1p-24f * rcp_fast(row.sum);
}
template <int P>
__device__ __forceinline__ void add_bias(const float* bias, Span sp, bool vec, float (&q)[P]) {
  float b[P];
  load_as<P, float>(bias, sp.e0, sp.n, vec, b);
#pragma unroll
  for (int i = 0; i < P; ++i) q[i] += b[i];
}

// 64-bit scores of a few of a lane's experts (bits of `need`) into keys. All lanes call it.
template <int P, bool SIGMOID>
__device__ __forceinline__ void exact_keys(const Shape& s, const float (&x)[P], Span sp, const float* bias, float most,
                                           double total, unsigned need, int64_t (&key)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) key[i] = kNone64;
  while (__any_sync(kFull, need != 0)) {
    const int at = need != 0 ? __ffs(need) - 1 : 0;
    float xv = x[0];
#pragma unroll
    for (int i = 1; i < P; ++i) xv = i == at ? x[i] : xv;
    const double e = exp(SIGMOID ? -static_cast<double>(xv) : static_cast<double>(xv) - static_cast<double>(most));
    double q = SIGMOID ? 1.0 / (1.0 + e) : e / total;
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
template <int P, int L, bool SIGMOID>
__device__ __noinline__ int choose_exact(Shape s, const void* logits, int64_t t, const float* bias, Row row, int sub) {
  const int first = (threadIdx.x & 31) - sub;
  const Span sp = span_of(s, sub);
  const bool by_score = bias != nullptr || (s.G > 1 && !s.group_max);
  const float slack = score_slack<P, SIGMOID>(row);
  float x[P], q[P];
  load_logits<P>(s, logits, t, sp, x);
  if (by_score && !SIGMOID) {
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = x[i] < INFINITY ? x[i] : neg_inf();  // +inf and NaN: as in the kernel
  }
  double total = 1;
  if (by_score && !SIGMOID) {
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
  const float inv = by_score && !SIGMOID ? rcp_fast(row.sum) : 1.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    q[i] = x[i] + 0.f;
    if (by_score) q[i] = SIGMOID ? sigmoid_fast(x[i]) : exp_fast(x[i] - row.most) * inv;
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
    const int lpg = 1 << s.lanes_log2;
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
      exact_keys<P, SIGMOID>(s, x, sp, bias, row.most, total, near(s.group_max ? a : b), key);
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
    const int g = sub >> s.lanes_log2;
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
    exact_keys<P, SIGMOID>(s, x, sp, bias, row.most, total, near(edge), key);
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

// ------------------------------------------------- sums of two floats
// hi + lo with |lo| at most half a unit of hi: the error-free sums and products of
// T. J. Dekker, A floating-point technique for extending the available precision
// (1971), and D. E. Knuth's sum of two.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two renormalise(float a, float b) {  // |a| >= |b|
  const float s = a + b;
  return {s, b - (s - a)};
}
__device__ __forceinline__ Two sum_of(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = sum_of(a.hi, b.hi);
  return renormalise(s.hi, s.lo + (a.lo + b.lo));
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  const float p = a.hi * b.hi;
  return renormalise(p, fmaf(a.lo, b.hi, fmaf(a.hi, b.lo, fmaf(a.hi, b.hi, -p))));
}
__device__ __forceinline__ Two reciprocal(Two a) {  // one Newton step from the fp32 value
  const float q = 1.f / a.hi;
  const float r = fmaf(-q, a.lo, fmaf(-q, a.hi, 1.f));
  return renormalise(q, q * r);
}
// e^y for -80 <= y <= 80 to about 2^-44: y = n ln 2 + 8 r, ln 2 as 1419 / 2048 (n times it is
// exact) and two floats; Taylor's series of e^r, |r| < 0.0434, its terms from the fifth on
// in fp32; three squarings.
__device__ __forceinline__ Two exp_two(Two y) {
  const float n = rintf(y.hi * 1.44269504f);
  const float p = n * 0x1.217f7ep-12f;
  Two r = add(add(sum_of(y.hi, -n * 0.69287109375f), {y.lo, 0.f}),
              {-p, -fmaf(n, 0x1.217f7ep-12f, -p) - n * -0x1.c610cap-37f});
  r = {r.hi * 0.125f, r.lo * 0.125f};
  const float t = fmaf(r.hi, fmaf(r.hi, 0x1.a01a02p-13f, 0x1.6c16c2p-10f), 0x1.111112p-7f);  // 1/5! + r/6! + r^2/7!
  Two e = add(mul(r, {t, 0.f}), {0x1.555556p-5f, -0x1.555556p-30f});                          // 1/4!
  e = add(mul(r, e), {0x1.555556p-3f, -0x1.555556p-28f});                                     // 1/3!
  e = add(mul(r, e), {0.5f, 0.f});
  e = add(mul(r, e), {1.f, 0.f});
  e = add(mul(r, e), {1.f, 0.f});
  e = mul(e, e);
  e = mul(e, e);
  e = mul(e, e);
  return {ldexpf(e.hi, static_cast<int>(n)), ldexpf(e.lo, static_cast<int>(n))};
}

// A key of two floats as a whole number above 0 in the same order.
__device__ __forceinline__ uint64_t packed(Two v) {
  return static_cast<uint64_t>(ordered(v.hi + 0.f)) << 32 | ordered(v.lo + 0.f);
}
__device__ __forceinline__ Two unpacked(uint64_t k) {
  return {unordered(static_cast<uint32_t>(k >> 32)), unordered(static_cast<uint32_t>(k))};
}
// Whether pairs of floats settle the order of two keys, `err` the sum of their errors. The same
// pair is a tie where the same inputs give it (`Inputs`): other inputs may leave a pair that 64
// bits tell apart, as sigmoids next to 1 with a bias whose sum fills the low part.
__device__ __forceinline__ bool settled(Two a, Two b, float err) {
  return fabsf((a.hi - b.hi) + (a.lo - b.lo)) > err;
}
struct Inputs {
  float x, b;  // logit and bias, zeros without a sign
  __device__ __forceinline__ bool operator==(Inputs o) const { return x == o.x && b == o.b; }
};
__device__ __forceinline__ Inputs shfl_xor(Inputs v, int o) {
  return {__shfl_xor_sync(kFull, v.x, o), __shfl_xor_sync(kFull, v.b, o)};
}
__device__ __forceinline__ Inputs shfl_from(Inputs v, int lane) {
  return {__shfl_sync(kFull, v.x, lane), __shfl_sync(kFull, v.b, lane)};
}

// Score plus bias and a bound on its error; `ok` is cleared where exp_two does not reach. The
// score is off by at most 2^-42 of itself (2^-43 the exponential, the rest its quotient or product), which
// a bias that cancels it leaves as it is; the sum adds 2^-46 of what it adds up. Four times
// that, and 2^-120 for products whose low parts leave fp32's range.
template <bool SIGMOID>
__device__ __forceinline__ Two key_two(float x, float bias, float most, Two inv_total, bool* ok, float* err) {
  const Two y = SIGMOID ? Two{-fabsf(x), 0.f} : sum_of(x, -most);
  *err = 0.f;
  if (!(fabsf(y.hi) <= 80.f)) {
    *ok = false;
    return {0.f, 0.f};
  }
  const Two z = exp_two(y);
  Two s;
  if (SIGMOID) {
    s = reciprocal(add({1.f, 0.f}, z));
    if (x < 0.f) s = mul(s, z);
  } else {
    s = mul(z, inv_total);
  }
  const Two k = bias == 0.f ? s : add(s, {bias, 0.f});
  *err = fmaf(fabsf(s.hi) + fabsf(k.hi), 0x1p-40f, 0x1p-120f);
  return k;
}
// 1 / sum of e^(x - most) over the token (softmax).
template <int P, int L>
__device__ __forceinline__ Two inv_total_two(const Shape& s, const void* logits, int64_t t, Span sp, float most) {
  Two sum = {0.f, 0.f};
#pragma unroll 1
  for (int i = 0; i < P; ++i) {
    const float x = i < sp.n ? logit_at(s, logits, t * s.ld + sp.e0 + i) : neg_inf();
    const Two y = sum_of(x, -most);
    // less than e^-80 of the sum does not show; no logit of +inf or NaN counts
    if (x - most >= -80.f && x < INFINITY) sum = add(sum, exp_two(y));
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1)
    sum = add(sum, {__shfl_xor_sync(kFull, sum.hi, o), __shfl_xor_sync(kFull, sum.lo, o)});
  return reciprocal(sum);
}

// The order of the candidates that lanes 0..K of a token hold, settled by pairs
// of floats: the sub-th expert, or -2 for the whole warp where they do not.
template <int P, int L, bool SIGMOID>
__device__ __noinline__ int order_candidates(Shape s, const void* logits, int64_t t, const float* bias, Row row, int sub,
                                             int e, float x) {
  const int first = (threadIdx.x & 31) - sub;
  const bool have = e >= 0;
  const float b = have && bias != nullptr ? __ldg(bias + e) : 0.f;
  bool ok = true;
  float err = 0.f;
  uint64_t key = 0;
  if (bias == nullptr) {  // within groups: the order of the logits
    if (have) key = packed({x, 0.f});
  } else {
    Two inv = {1.f, 0.f};
    if (!SIGMOID) inv = inv_total_two<P, L>(s, logits, t, span_of(s, sub), row.most);
    if (have) key = packed(key_two<SIGMOID>(x, b, row.most, inv, &ok, &err));
  }
  int rank = 0;
  for (int j = 0; j <= s.K; ++j) {
    const uint64_t kj = __shfl_sync(kFull, key, first + j);
    const int ej = __shfl_sync(kFull, e, first + j);
    const float both = __shfl_sync(kFull, err, first + j) + err;
    const Inputs from = shfl_from({x, b}, first + j);
    if (j != sub && have && ej >= 0) {
      rank += kj > key || (kj == key && ej < e);
      if (bias != nullptr && !(from == Inputs{x, b}) && !settled(unpacked(kj), unpacked(key), both)) ok = false;
    } else if (j != sub && !have && (ej >= 0 || j < sub)) {
      ++rank;
    }
  }
  if (sub > s.K) rank = sub;
  int out = -1;
  for (int j = 0; j <= s.K; ++j) {
    const int rj = __shfl_sync(kFull, rank, first + j), ej = __shfl_sync(kFull, e, first + j);
    if (rj == sub) out = ej;
  }
  return __all_sync(kFull, ok) ? out : -2;
}

// Whether the lane has an expert that is not taken, next to the K-th (taken[K - 1]) by its
// fp32 key and of other inputs. All lanes' groups that are not `in` are out.
template <int P, bool SIGMOID>
__device__ __noinline__ bool near_the_last(Shape s, const void* logits, int64_t t, const float* bias, Row row, Span sp,
                                           const uint2* taken, bool in) {
  auto expert = [&](uint2 v) { return v.x != 0 ? static_cast<int>(v.y) - static_cast<int>(v.x & (P - 1)) : -1; };
  const bool by_score = bias != nullptr || (s.G > 1 && !s.group_max);
  const float slack = by_score ? score_slack<P, SIGMOID>(row) : 0.f, inv = rcp_fast(row.sum);
  const uint2 last = taken[s.K - 1];
  const int el = expert(last);
  const Inputs from = {logit_at(s, logits, t * s.ld + el), bias != nullptr ? __ldg(bias + el) : 0.f};
  const float a = unordered(last.x & ~static_cast<uint32_t>(P - 1));
  float x[P], b[P];
  load_logits<P>(s, logits, t, sp, x);
  if (bias != nullptr) load_as<P, float>(bias, sp.e0, sp.n, s.vec_bias, b);
  unsigned other = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (bias == nullptr) b[i] = 0.f;
    other |= static_cast<unsigned>(in && x[i] > neg_inf() && b[i] > neg_inf() && !(Inputs{x[i], b[i]} == from)) << i;
  }
  bool near = false;
  for (; other != 0; other &= other - 1) {
    const int e = sp.e0 + __ffs(other) - 1;
    const float be = bias != nullptr ? __ldg(bias + e) : 0.f;
    float v = logit_at(s, logits, t * s.ld + e);
    if (by_score) v = (SIGMOID ? sigmoid_fast(v) : exp_fast(v - row.most) * inv) + be;
    if (a - v > (by_score ? 2.f * slack + P * 0x1p-22f * (fabsf(a) + fabsf(v)) : 0.f)) continue;
    bool has = false;
    for (int k = 0; k <= s.K; ++k) has |= expert(taken[k]) == e;
    near |= !has;
  }
  return near;
}

// Whether this lane's group is among the best, from the two best keys of each lane in
// pairs of floats (key: the lane's three best fp32 keys; edge: the fp32 value
// that a group's third may not come near). Only the groups `near` the border by their fp32 values
// take part; the others are `in` or not. L is 32. -1 where the pairs do not settle it.
template <int P, bool SIGMOID>
__device__ __noinline__ int rank_groups(Shape s, const void* logits, int64_t t, const float* bias, Row row, int sub,
                                        uint3 key, float edge, float slack, bool near, bool in_now) {
  const Span sp = span_of(s, sub);
  Two inv = {1.f, 0.f};
  if (!SIGMOID) inv = inv_total_two<P, 32>(s, logits, t, sp, row.most);
  bool ok = true;
  float err = 0.f;  // the largest of the group's keys
  uint64_t c[2] = {0, 0};
  Inputs in[2] = {};
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t k = j == 0 ? key.x : key.y;
    if (k != 0) {
      const int e = sp.e0 + P - 1 - static_cast<int>(k & (P - 1));
      float of_key;
      in[j] = {logit_at(s, logits, t * s.ld + e), bias != nullptr ? __ldg(bias + e) : 0.f};
      c[j] = packed(key_two<SIGMOID>(in[j].x, in[j].b, row.most, inv, &ok, &of_key));
      err = fmaxf(err, of_key);
    }
  }
  if (key.z != 0 && unordered(key.z & ~static_cast<uint32_t>(P - 1)) + slack >= edge) ok = false;
  const bool first = c[0] >= c[1];
  uint64_t a = first ? c[0] : c[1], b = first ? c[1] : c[0];  // the group's two best, and where they are from
  Inputs from_a = in[first ? 0 : 1], from_b = in[first ? 1 : 0];
  for (int o = 1 << s.lanes_log2 >> 1; o > 0; o >>= 1) {
    const uint64_t a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
    const Inputs from_a2 = shfl_xor(from_a, o), from_b2 = shfl_xor(from_b, o);
    if (b2 > b) {
      b = b2;
      from_b = from_b2;
    }
    if (min(a, a2) > b) {
      b = min(a, a2);
      from_b = a2 > a ? from_a : from_a2;
    }
    if (a2 > a) {
      a = a2;
      from_a = from_a2;
    }
    err = fmaxf(err, __shfl_xor_sync(kFull, err, o));
  }
  // whether the value is that of these two surely, which a tie needs
  const uint64_t last = s.group_max ? a : b;
  bool sure = true;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const bool is = in[j] == from_a || (!s.group_max && in[j] == from_b);
    if (c[j] != 0 && !is && !settled(unpacked(last), unpacked(c[j]), 2.f * err)) sure = false;
  }
  const bool sum = !s.group_max && b != 0;
  if (!sum) from_b = {0.f, neg_inf()};
  const uint64_t value = !near ? 0 : sum ? packed(add(unpacked(a), unpacked(b))) : a;
  err *= 2.f;  // of the sum of two
  const int g = sub >> s.lanes_log2;
  const bool first_of_group = (sub & ((1 << s.lanes_log2) - 1)) == 0;
  const int open = s.top_groups - __popc(__ballot_sync(kFull, first_of_group && in_now && !near));
  int rank = 0;
  for (int j = 0; j < s.G; ++j) {
    const uint64_t v = __shfl_sync(kFull, value, j << s.lanes_log2);
    rank += v > value || (v == value && j < g);
  }
  const bool mine = near ? rank < open : in_now;
  // a group of the near ones that is in against each that is not
  for (int j = 0; j < s.G; ++j) {
    const int lane = j << s.lanes_log2;
    const uint64_t v = __shfl_sync(kFull, value, lane);
    const float both = __shfl_sync(kFull, err, lane) + err;
    const Inputs its_a = shfl_from(from_a, lane), its_b = shfl_from(from_b, lane);
    const bool its = __shfl_sync(kFull, mine, lane), same = its_a == from_a && its_b == from_b;
    if (v != 0 && its != mine && (same ? !sure : !settled(unpacked(v), unpacked(value), both))) ok = false;
  }
  return __all_sync(kFull, ok || !near) ? mine : -1;
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

template <int P, int L, bool SIGMOID, bool MEAN>
__global__ void __launch_bounds__(kRouteThreads, MEAN ? 4 : 7)
    route_kernel(Shape s, const void* __restrict__ logits, const float* __restrict__ bias, int32_t* __restrict__ idx,
                 float* __restrict__ w, float* __restrict__ partials) {
  constexpr int kTokens = kRouteThreads / L;  // a block at a time
  constexpr float kCut = P * 0x1p-22f;        // of a key: the cut bits, and its own rounding
  const int lane = threadIdx.x & 31, sub = lane % L, first = lane - sub;
  const Span sp = span_of(s, sub);
  const bool by_score = bias != nullptr || (s.G > 1 && !s.group_max);
  const bool softmax_sum = !SIGMOID && (by_score || !s.renorm || MEAN);
  // 16-bit logits keep all their bits in a key
  const bool check = by_score || s.dtype == MOE_FP32;
  const int rounds = s.K + (check && s.K < s.E ? 1 : 0);
  const int width = s.K > 1 ? 2 << (31 - __clz(s.K - 1)) : 1;
  const bool vec_bias = s.vec_bias;
  __shared__ uint2 slots[kTokens][L + 1];  // keys in the order they are taken, and where their lane starts
  uint2* taken = slots[threadIdx.x / L];
  const unsigned below = ((1u << lane) - 1u) & ~((1u << first) - 1u);  // lower lanes of the token
  // Mean scores: a lane adds up kMeanRun tokens, then its sums so far and what their additions lost
  // (float2, in shared memory: few blocks walk as many), so that the roundings do not grow with T.
  constexpr int kMeanRun = 16;
  constexpr int kColsBytes = kRouteThreads / 32 * kMaxExperts * 4, kSumsBytes = P * kRouteThreads * 8;
  __shared__ __align__(16) uint8_t mean_smem[MEAN ? (kColsBytes > kSumsBytes ? kColsBytes : kSumsBytes) : 16];
  float2(*sums)[kRouteThreads] = reinterpret_cast<float2(*)[kRouteThreads]>(mean_smem);  // [P][threads]
  float acc[MEAN ? P : 1];
  int walked = 0;
  if constexpr (MEAN) {
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i] = 0.f;
  }
  pdl_wait();
  pdl_launch_dependents();
  const int step = gridDim.x * kTokens;  // T is at most 2^26
  float ahead[MEAN ? P : 1];  // blocks that take many tokens: the next one's logits are on their way
  if constexpr (MEAN) {
    const int t = blockIdx.x * kTokens + threadIdx.x / L;
    load_logits<P>(s, logits, t < s.T ? t : s.T - 1, sp, ahead);
  }
  // every lane walks the same number of tokens: the shuffles take whole warps
  for (int t0 = blockIdx.x * kTokens; t0 < s.T; t0 += step) {
    const int t = t0 + threadIdx.x / L;
    const bool valid = t < s.T;
    const int tr = valid ? t : s.T - 1;
    float x[P], q[P];  // logits; scores (softmax: times their sum)
    if constexpr (MEAN) {
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = ahead[i];
      if (t0 + step < s.T) load_logits<P>(s, logits, t + step < s.T ? t + step : s.T - 1, sp, ahead);
    } else {
      load_logits<P>(s, logits, tr, sp, x);
    }
    // Comparisons, selections and whole numbers share a pipe of half the rate, which is
    // what the kernel is bound by; so whether any logit or bias of the warp's tokens needs
    // a second look (infinite, NaN, behind the last expert) is a sum, 0 if none does.
    float v[P], look = 0.f;
    if (bias != nullptr) load_as<P, float>(bias, sp.e0, sp.n, vec_bias, v);
#pragma unroll
    for (int i = 0; i < P; ++i) look = fmaf(x[i], 0.f, look);
    if (bias != nullptr) {
#pragma unroll
      for (int i = 0; i < P; ++i) look = fmaf(v[i], 0.f, look);
    }
    const bool plain = __all_sync(kFull, look == 0.f);
    unsigned any_nan = 0;
    if (!plain) {
      // a logit of +inf has no softmax: where scores choose it is out like a NaN one
      bool nan = false;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const bool lost = x[i] != x[i] || (!SIGMOID && x[i] == INFINITY);
        if (lost && by_score) x[i] = __int_as_float(0x7fffffff);
        nan |= lost;
      }
      any_nan = __ballot_sync(kFull, nan);
      if (L < 32) any_nan = (any_nan >> first) & ((1u << (L & 31)) - 1u);
    }
    Row row = {neg_inf(), 1.f};
    if (softmax_sum) {
#pragma unroll
      for (int i = 0; i < P; ++i) row.most = fmaxf(row.most, x[i]);
      row.most = lane_max<L>(row.most);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        q[i] = exp_fast(x[i] - row.most);
        if (!plain) q[i] = x[i] > neg_inf() ? q[i] : 0.f;
        sum += q[i];
      }
      row.sum = lane_sum<L>(sum);
    } else if (SIGMOID && (by_score || MEAN)) {
#pragma unroll
      for (int i = 0; i < P; ++i) q[i] = sigmoid_fast(x[i]);
    }
    uint32_t key[P];
    const float inv = SIGMOID ? 1.f : rcp_fast(row.sum);
    if (bias != nullptr) {
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = fmaf(q[i], inv, v[i]);
    } else if (by_score) {
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = q[i] * inv;
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = x[i] + 0.f;  // -0 and 0 are one value
    }
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = (ordered(v[i]) & ~static_cast<uint32_t>(P - 1)) | (P - 1 - i);
    if (!plain) {
#pragma unroll
      for (int i = 0; i < P; ++i) key[i] = x[i] > neg_inf() && v[i] > neg_inf() ? key[i] : 0u;
    }
    sort_keys<P>(key);
    const float slack = by_score ? score_slack<P, SIGMOID>(row) : 0.f;
    bool unsure = false, exact = false;  // settled by pairs of floats; by 64 bits
    bool in = true;                      // the lane's group is among the best
    if (s.G > 1) {
      const int lpg = 1 << s.lanes_log2;
      uint32_t a = key[0], b = key[P > 1 ? 1 : 0];
      for (int o = lpg / 2; o > 0; o >>= 1) {
        const uint32_t a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
        b = max(min(a, a2), max(b, b2));
        a = max(a, a2);
      }
      const float va = a != 0 ? unordered(a & ~static_cast<uint32_t>(P - 1)) : neg_inf();
      const float vb = s.group_max || b == 0 ? 0.f : unordered(b & ~static_cast<uint32_t>(P - 1));
      // below every other value without an expert, not below the type's range with some
      const float value = a != 0 ? fmaxf(va + vb, -FLT_MAX) : neg_inf();
      const int g = sub >> s.lanes_log2;
      int rank = 0;
      for (int j = 0; j < s.G; ++j) {
        const float v = __shfl_sync(kFull, value, j * lpg);
        rank += v > value || (v == value && j < g);
      }
      in = rank < s.top_groups && g < s.G;
      if (check && s.top_groups < s.G) {
        // of a value; an infinite one is itself, and a group without an expert is near no other
        const float err = fabsf(value) < INFINITY ? 2.f * slack + (kCut * fabsf(va) + kCut * fabsf(vb)) : 0.f;
        const bool some = a != 0;
        const float worst = -unordered(lane_max_u32<L>(ordered(in && some ? err - value : neg_inf())));
        const float best = unordered(lane_max_u32<L>(ordered(!in && some && g < s.G ? value + err : neg_inf())));
        if (worst <= best) {  // the token's lanes are the warp's: all agree
          int settled_in = -1;
          if (by_score)
            settled_in = rank_groups<P, SIGMOID>(s, logits, tr, bias, row, sub, make_uint3(key[0], key[1], P > 2 ? key[P > 2 ? 2 : 0] : 0u),
                                                 (s.group_max ? va : b == 0 ? neg_inf() : vb) - err, err,
                                                 some && g < s.G && (in ? value - err <= best : value + err >= worst), in);
          exact = settled_in < 0;
          if (!exact) in = settled_in != 0;
        }
      }
#pragma unroll
      for (int i = 0; i < P; ++i) key[i] = in ? key[i] : 0u;
    }
    // The lane of the best key left writes it down and moves up; between lanes the places
    // do not count: equal keys go to the lowest lane.
    for (int k = 0; k < rounds; ++k) {
      const uint32_t head = key[0] & ~static_cast<uint32_t>(P - 1);
      const bool best = head == lane_max_u32<L>(head);
      const unsigned who = __ballot_sync(kFull, best);
      if (best && (who & below) == 0) {
        taken[k] = make_uint2(key[0], sp.e0 + P - 1);
#pragma unroll
        for (int i = 0; i + 1 < P; ++i) key[i] = key[i + 1];
        key[P - 1] = 0u;
      }
    }
    __syncwarp();
    // lane k: the k-th choice and the one behind it
    auto expert = [&](uint2 t) { return t.x != 0 ? static_cast<int>(t.y) - static_cast<int>(t.x & (P - 1)) : -1; };
    const uint2 mine = sub < rounds ? taken[sub] : make_uint2(0, 0);
    const uint2 after = sub + 1 < rounds ? taken[sub + 1] : make_uint2(0, 0);
    int e = expert(mine);
    float xe = e >= 0 ? logit_at(s, logits, tr * s.ld + e) : neg_inf();
    if (check) {
      if (sub < s.K && mine.x != 0 && after.x != 0) {
        const float a = unordered(mine.x & ~static_cast<uint32_t>(P - 1)), b = unordered(after.x & ~static_cast<uint32_t>(P - 1));
        unsure |= a - b <= (by_score ? 2.f * slack + kCut * (fabsf(a) + fabsf(b)) : 0.f);
      }
      if (__any_sync(kFull, unsure)) {  // the same inputs are the same key
        bool border = false;            // the K-th and the one behind it are
        if (unsure) {
          const int ea = expert(after);
          unsure = !(xe == logit_at(s, logits, tr * s.ld + ea) && (bias == nullptr || __ldg(bias + e) == __ldg(bias + ea)));
          border = !unsure && sub == s.K - 1;
        }
        // then others that are as near may be left in the lanes
        unsigned who = __ballot_sync(kFull, border);
        if (L < 32) who = (who >> first) & ((1u << (L & 31)) - 1u);
        if (who != 0) unsure |= near_the_last<P, SIGMOID>(s, logits, tr, bias, row, span_of(s, sub), taken, in);
      }
      if (__any_sync(kFull, unsure || exact)) {
        // candidates: the K + 1 that the lanes hold, if the next one is surely none
        const uint32_t head = lane_max_u32<L>(key[0]);
        const uint32_t kth = taken[s.K - 1].x;
        if (head != 0 && s.K < L) {
          const float a = unordered(kth & ~static_cast<uint32_t>(P - 1)), b = unordered(head & ~static_cast<uint32_t>(P - 1));
          exact |= a - b <= (by_score ? 2.f * slack + kCut * (fabsf(a) + fabsf(b)) : 0.f);
        }
        exact |= s.K == L;
        int chosen = -2;
        if (!__any_sync(kFull, exact)) chosen = order_candidates<P, L, SIGMOID>(s, logits, tr, bias, row, sub, e, xe);
        if (chosen == -2) chosen = choose_exact<P, L, SIGMOID>(s, logits, tr, bias, row, sub);
        e = sub < s.K ? chosen : -1;
        xe = e >= 0 ? logit_at(s, logits, tr * s.ld + e) : neg_inf();
      }
    }
    const bool have = sub < s.K && e >= 0;
    float weight = 0.f;
    if (SIGMOID) {
      float score = 0.f, n;
      if (have) sigmoid_pair(xe, &score, &n);
      if (s.renorm) {
        float sum = head_sum(score, width);
        if (__any_sync(kFull, sub < width && sum < 1e-20f)) {  // below fp32's range the ratios are those of e^x
          const float most = head_max(have ? xe : neg_inf(), width);
          const float low = have ? ratio_score<true>(xe, most) : 0.f;
          const float low_sum = head_sum(low, width);
          if (sum < 1e-20f) {
            score = low;
            sum = low_sum;
          }
        }
        score = have ? __fdividef(score, sum) : 0.f;
      }
      weight = score * s.scale;
    } else if (s.renorm) {
      const float most = head_max(have ? xe : neg_inf(), width);
      const float score = have ? expf(xe - most) : 0.f;
      const float sum = head_sum(score, width);
      weight = have ? __fdividef(score, sum) * s.scale : 0.f;
    } else {
      weight = have ? __fdividef(expf(xe - row.most), row.sum) * s.scale : 0.f;
    }
    __syncwarp();  // `taken` has been read
    if (any_nan) weight = __int_as_float(0x7fffffff);
    if (valid && sub < s.K) {
      idx[t * s.K + sub] = e;
      w[t * s.K + sub] = weight;
    }
    if constexpr (MEAN) {
      float sum = row.sum;
      if (SIGMOID) {
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
            if (small) q[i] = x[i] == neg_inf() ? 0.f : exp_fast(x[i] - most);
            low += q[i];
          }
          low = lane_sum<L>(low);
          if (small) sum = low;
        }
      }
      if (any_nan) sum = __int_as_float(0x7fffffff);
      const float f = sum != 0.f ? rcp_fast(sum) : 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) acc[i] += valid ? q[i] * f : 0.f;
      if (++walked % kMeanRun == 0) {  // every thread of the block at once
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 so_far = walked > kMeanRun ? sums[i][threadIdx.x] : make_float2(0.f, 0.f);
          const Two v = sum_of(so_far.x, acc[i]);
          sums[i][threadIdx.x] = make_float2(v.hi, so_far.y + v.lo);
          acc[i] = 0.f;
        }
      }
    }
  }
  if constexpr (MEAN) {
    if (walked >= kMeanRun) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 so_far = sums[i][threadIdx.x];
        acc[i] = (acc[i] + so_far.y) + so_far.x;
      }
      __syncthreads();  // the columns take their place
    }
    // lanes that hold the same experts, then the block's warps, in a fixed order
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int o = 16; o >= L; o >>= 1) acc[i] += __shfl_xor_sync(kFull, acc[i], o);
    }
    float(*cols)[kMaxExperts] = reinterpret_cast<float(*)[kMaxExperts]>(mean_smem);  // [warps][experts]
    if (lane < L) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i < sp.n) cols[threadIdx.x / 32][sp.e0 + i] = acc[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < s.E; e += kRouteThreads) {
      float v = 0.f;
      for (int k = 0; k < kRouteThreads / 32; ++k) v += cols[k][e];
      // one block's columns are the means already
      partials[static_cast<size_t>(blockIdx.x) * s.E + e] = gridDim.x == 1 ? v / static_cast<float>(s.T) : v;
    }
  }
}

template <bool SIGMOID>
cudaError_t launch_route_kind(int dtype, const RouteArgs& a, int num_sms, cudaStream_t st) {
  const Split sp = split_of(a.E, a.K, a.G);
  const Shape s = shape_of(dtype, a, a.logits, a.ld, sp);
  const int blocks = route_blocks(a, sp, a.mean != nullptr ? kRouteParts : 16 * num_sms);
  // A dependent launch hides the start of a large grid (8192 x 256: 14.3 us without, 11.5 with) and
  // costs the host 0.7 us, which is what a small call takes longest.
  return with_split(sp, [&](auto P, auto L) {
    constexpr int p = decltype(P)::value, l = decltype(L)::value;
    return launch_kernel(blocks >= num_sms, a.mean != nullptr ? route_kernel<p, l, SIGMOID, true> : route_kernel<p, l, SIGMOID, false>,
                         blocks, kRouteThreads, 0, st, s, a.logits, a.bias, a.idx, a.w,
                         blocks == 1 ? a.mean : a.partials);
  });
}

}  // namespace

}  // namespace bsmoe
