// The experts' FP4 format: rows to e2m1 codes with a UE8M0 scale per 32 elements
// (moe_quantize_fp4), back (moe_dequantize_fp4), and the activations of
// moe_matmul_fp4 in the layout its tensor-core kernels stage.
//
// A block's exponent is n = min{n : amax <= 6 * 2^n}; x * 2^-n is exact in fp32 and is
// rounded once, to the nearest e2m1 value, ties to even. A block with a NaN or an
// infinity, which e2m1 has no code for, gets the scale byte 255 (NaN) and zero codes.
//
// A thread takes 16 elements, two lanes a block, so that loads and stores are 32
// and 8 bytes a lane (packs of 16 bytes or single elements where the alignment
// does not allow them). Bound by memory.
#include "../act_quant.cuh"
#include "block_internal.cuh"

namespace bsmoe {

namespace {

constexpr int kUnit = 16;  // elements a thread
constexpr int kQuantThreads = 256;

struct alignas(32) Wide {
  uint32_t w[8];
};
__device__ __forceinline__ Wide load_wide(const void* p) {
  Wide v;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                 "=r"(v.w[7])
               : "l"(p));
  return v;
}

// How a row's packs may be loaded.
enum : int { kLoadWide = 2, kLoad16 = 1, kLoadAny = 0 };

template <typename T>
__device__ __forceinline__ void load_unit(const T* p, int how, float (&f)[kUnit]) {
  if (how == kLoadWide) {
    constexpr int W = 32 / sizeof(T);
#pragma unroll
    for (int i = 0; i < kUnit; i += W) {
      const Wide v = load_wide(p + i);
      float g[W];
      unpack(*reinterpret_cast<const Pack<T, W>*>(&v), g);
#pragma unroll
      for (int j = 0; j < W; ++j) f[i + j] = g[j];
    }
  } else if (how == kLoad16) {
    constexpr int W = kVec<T>;
#pragma unroll
    for (int i = 0; i < kUnit; i += W) {
      const Pack<T, W> v = load_pack<W>(p + i);
      float g[W];
      unpack(v, g);
#pragma unroll
      for (int j = 0; j < W; ++j) f[i + j] = g[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) f[i] = to_f32(p[i]);
  }
}

// Codes of a unit and its block's scale byte; both lanes of a block call it.
__device__ __forceinline__ uint2 quantize_unit(const float (&f)[kUnit], uint32_t* scale) {
  float amax = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    amax = fmaxf(amax, fabsf(f[i]));
    finite &= fabsf(f[i]) < INFINITY;
  }
  amax = finite ? amax : INFINITY;
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  if (!(amax < INFINITY)) {
    *scale = 255;
    return make_uint2(0, 0);
  }
  const int n = act_exponent_e2m1(amax);
  const float m = exp2_neg(n);
  *scale = static_cast<uint32_t>(n + 127);
  return make_uint2(pack8_e2m1(f[0] * m, f[1] * m, f[2] * m, f[3] * m, f[4] * m, f[5] * m, f[6] * m, f[7] * m),
                    pack8_e2m1(f[8] * m, f[9] * m, f[10] * m, f[11] * m, f[12] * m, f[13] * m, f[14] * m, f[15] * m));
}

// Units of all rows in order; `cols`: units a row.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const T* __restrict__ x, int64_t ld, int64_t units,
                                                                 int cols, int how, uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scale) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kQuantThreads;
  pdl_wait();
  pdl_launch_dependents();
  // whole warps walk together: two lanes share a block
  for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * kQuantThreads; u0 < units; u0 += step) {
    const int64_t u = u0 + threadIdx.x;
    const bool valid = u < units;
    const int64_t v = valid ? u : units - 1;
    float f[kUnit];
    load_unit(x + (cols == 0 ? v * kUnit : v / cols * ld + v % cols * kUnit), how, f);
    uint32_t sc;
    const uint2 q = quantize_unit(f, &sc);
    if (valid) {
      *reinterpret_cast<uint2*>(codes + v * 8) = q;
      if (v % 2 == 0) scale[v / 2] = static_cast<uint8_t>(sc);
    }
  }
}

// Activations for the product: codes [T][Kp / 2], zeros behind K, and scale words
// in the chunk layout of the tensor cores (sf_word_index). A unit row has Kp / 16
// units: eight lanes make the four scale bytes of 128 columns.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quantize_act_kernel(const T* __restrict__ x, int64_t ld, int rows, int K,
                                                                     int KB, int how, uint8_t* __restrict__ codes,
                                                                     uint32_t* __restrict__ sf, uint32_t* status) {
  const int64_t units = static_cast<int64_t>(rows) * KB * 8, step = static_cast<int64_t>(gridDim.x) * kQuantThreads;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * kQuantThreads; u0 < units; u0 += step) {
    const int64_t u = u0 + threadIdx.x;
    const bool valid = u < units;
    const int64_t v = valid ? u : units - 1;
    const int row = static_cast<int>(v / (KB * 8)), c = static_cast<int>(v % (KB * 8));
    float f[kUnit];
    if (c * kUnit < K) {
      load_unit(x + row * ld + c * kUnit, how, f);
    } else {
#pragma unroll
      for (int i = 0; i < kUnit; ++i) f[i] = 0.f;
    }
    uint32_t sc;
    const uint2 q = quantize_unit(f, &sc);
    uint32_t word = sc << (8 * ((c / 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    if (valid) {
      *reinterpret_cast<uint2*>(codes + v * 8) = q;
      if (c % 8 == 0) sf[sf_word_index(row, c / 8, KB)] = word;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kQuantThreads) dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scale, int64_t units,
                                                                   bool wide_in, int out_how, T* __restrict__ out) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kQuantThreads;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kQuantThreads + threadIdx.x; u < units; u += step) {
    uint32_t w[2];
    if (wide_in) {
      const uint2 c = *reinterpret_cast<const uint2*>(codes + u * 8);
      w[0] = c.x;
      w[1] = c.y;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i] |= static_cast<uint32_t>(codes[u * 8 + 4 * i + j]) << (8 * j);
      }
    }
    const uint32_t b = scale[u / 2];
    const float m = b == 255 ? __int_as_float(0x7fffffff) : b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
    float f[kUnit];
#pragma unroll
    for (int i = 0; i < kUnit; i += 2) {
      // two codes of a byte as fp16 values, exact
      uint32_t h;
      asm("{\n\t.reg .b8 q, r;\n\t.reg .b16 z;\n\tcvt.u16.u32 z, %1;\n\tmov.b16 {q, r}, z;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, q;\n\t}"
          : "=r"(h)
          : "r"((w[i / 8] >> (4 * (i % 8))) & 0xffu));
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[i] = v.x * m;
      f[i + 1] = v.y * m;
    }
    T* o = out + u * kUnit;
    if (out_how == kLoadWide) {
      constexpr int W = 32 / sizeof(T);
#pragma unroll
      for (int i = 0; i < kUnit; i += W) {
        float g[W];
#pragma unroll
        for (int j = 0; j < W; ++j) g[j] = f[i + j];
        const Pack<T, W> p = pack<T>(g);
        const uint32_t* r = reinterpret_cast<const uint32_t*>(&p);
        st_global_v8(o + i, r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7]);
      }
    } else if (out_how == kLoad16) {
      constexpr int W = kVec<T>;
#pragma unroll
      for (int i = 0; i < kUnit; i += W) {
        float g[W];
#pragma unroll
        for (int j = 0; j < W; ++j) g[j] = f[i + j];
        store_pack(o + i, pack<T>(g));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kUnit; ++i) o[i] = from_f32<T>(f[i]);
    }
  }
}

int how_aligned(const void* p, int64_t ld, size_t es) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * es);
  return a % 32 == 0 ? kLoadWide : a % 16 == 0 ? kLoad16 : kLoadAny;
}

int unit_blocks(int64_t units, int num_sms) {
  const int64_t need = (units + kQuantThreads - 1) / kQuantThreads, most = static_cast<int64_t>(num_sms) * 8;
  return static_cast<int>(need < most ? need : most);
}

}  // namespace

cudaError_t launch_quantize_fp4(int dtype, const void* x, int64_t ld, int R, int C, uint8_t* codes, uint8_t* scale,
                                int num_sms, cudaStream_t st) {
  const int64_t units = static_cast<int64_t>(R) * (C / kUnit);
  const int cols = ld == C || R == 1 ? 0 : C / kUnit;  // 0: one run of units
  return with_dtype(dtype, [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return launch_kernel(false, quantize_kernel<T>, unit_blocks(units, num_sms), kQuantThreads, 0, st,
                         static_cast<const T*>(x), ld, units, cols, how_aligned(x, cols == 0 ? 0 : ld, sizeof(T)), codes,
                         scale);
  });
}

cudaError_t launch_dequantize_fp4(int dtype, const uint8_t* codes, const uint8_t* scale, int64_t blocks, void* out,
                                  int num_sms, cudaStream_t st) {
  const int64_t units = blocks * 2;
  return with_dtype(dtype, [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return launch_kernel(false, dequantize_kernel<T>, unit_blocks(units, num_sms), kQuantThreads, 0, st, codes, scale,
                         units, reinterpret_cast<uintptr_t>(codes) % 8 == 0, how_aligned(out, 0, sizeof(T)),
                         static_cast<T*>(out));
  });
}

cudaError_t launch_quantize_act(int dtype, const void* x, int64_t ld, int T, int K, uint8_t* codes, uint32_t* sf,
                                uint32_t* status, int num_sms, cudaStream_t st) {
  const int KB = ceil_div(K, 128);
  return with_dtype(dtype, [&](auto* p) {
    using E = std::remove_pointer_t<decltype(p)>;
    return launch_kernel(false, quantize_act_kernel<E>, unit_blocks(static_cast<int64_t>(T) * KB * 8, num_sms),
                         kQuantThreads, 0, st, static_cast<const E*>(x), ld, T, K, KB, how_aligned(x, ld, sizeof(E)),
                         codes, sf, status);
  });
}

}  // namespace bsmoe
