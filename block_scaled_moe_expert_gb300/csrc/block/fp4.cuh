// Units of 16 elements and their FP4 codes: what the quantizing kernels (fp4.cu) and the
// product that quantizes its own activations (matmul_fp4.cu) share.
#pragma once
#include <type_traits>

#include "../act_quant.cuh"
#include "block_internal.cuh"

namespace bsmoe {

constexpr int kUnit = 16;  // elements a thread

// A unit's elements as they lie in memory.
template <typename T>
struct alignas(32) Unit {
  uint32_t w[kUnit * sizeof(T) / 4];
};

// How a row's units may be loaded.
enum : int { kLoadWide = 2, kLoad16 = 1, kLoadAny = 0 };

template <typename T>
__device__ __forceinline__ Unit<T> load_unit(const T* p, int how) {
  constexpr int W = kUnit * sizeof(T) / 4;
  Unit<T> u;
  if (how == kLoadWide) {
#pragma unroll
    for (int i = 0; i < W; i += 8)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(u.w[i]), "=r"(u.w[i + 1]), "=r"(u.w[i + 2]), "=r"(u.w[i + 3]), "=r"(u.w[i + 4]),
                     "=r"(u.w[i + 5]), "=r"(u.w[i + 6]), "=r"(u.w[i + 7])
                   : "l"(reinterpret_cast<const uint32_t*>(p) + i));
  } else if (how == kLoad16) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
      u.w[i] = v.x;
      u.w[i + 1] = v.y;
      u.w[i + 2] = v.z;
      u.w[i + 3] = v.w;
    }
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < W; ++i) u.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  } else {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < W; ++i) u.w[i] = q[2 * i] | static_cast<uint32_t>(q[2 * i + 1]) << 16;
  }
  return u;
}
template <typename T>
__device__ __forceinline__ Unit<T> zero_unit() {
  Unit<T> u;
#pragma unroll
  for (uint32_t& w : u.w) w = 0;
  return u;
}

// Codes of a unit and its block's scale byte; both lanes of a block call it. The
// magnitudes are compared as whole numbers, where a NaN is above infinity and both are
// above every number.
template <typename T>
__device__ __forceinline__ uint2 quantize_unit(const Unit<T>& u, uint32_t* scale) {
  constexpr int W = kUnit * sizeof(T) / 4;
  float amax;
  bool finite;
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) m = max(m, u.w[i] & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    amax = __uint_as_float(m);
    finite = m < 0x7f800000u;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) m = __vmaxu2(m, u.w[i] & 0x7fff7fffu);
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m & 0xffffu, m >> 16);
    amax = unpack2(m, T()).x;
    finite = m < (std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u);
  }
  if (!finite) {
    *scale = 255;
    return make_uint2(0, 0);
  }
  const int n = act_exponent_e2m1(amax);
  const float2 m = make_float2(exp2_neg(n), exp2_neg(n));
  *scale = static_cast<uint32_t>(n + 127);
  float2 f[kUnit / 2];
#pragma unroll
  for (int i = 0; i < kUnit / 2; ++i) {
    if constexpr (sizeof(T) == 4) f[i] = make_float2(__uint_as_float(u.w[2 * i]), __uint_as_float(u.w[2 * i + 1]));
    else f[i] = unpack2(u.w[i], T());
    f[i] = mul2(f[i], m);
  }
  return make_uint2(pack8_e2m1(f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y),
                    pack8_e2m1(f[4].x, f[4].y, f[5].x, f[5].y, f[6].x, f[6].y, f[7].x, f[7].y));
}

inline int how_aligned(const void* p, int64_t ld, size_t es) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * es);
  return a % 32 == 0 ? kLoadWide : a % 16 == 0 ? kLoad16 : kLoadAny;
}

}  // namespace bsmoe
