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
// does not allow them). Bound by memory: 28672 x 4096 bf16 to FP4 44 us (297 MB, 6.7 TB/s), back
// 49 us; the activations of 8192 x 7168 24 us (6.2 TB/s), of 8192 x 2048 9.9.
#include "fp4.cuh"

namespace bsmoe {

namespace {

constexpr int kQuantThreads = 256;

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
    uint32_t sc;
    const uint2 q = quantize_unit(load_unit(x + (cols == 0 ? v * kUnit : v / cols * ld + v % cols * kUnit), how), &sc);
    if (valid) {
      *reinterpret_cast<uint2*>(codes + v * 8) = q;
      if (v % 2 == 0) scale[v / 2] = static_cast<uint8_t>(sc);
    }
  }
}

// Activations for the product: codes [T][Kp / 2], zeros behind K, and scale words
// in the chunk layout of the tensor cores (sf_word_index). A row has 8 KB units: eight
// lanes make the four scale bytes of 128 columns. A warp takes kActUnits of a row, their
// loads in flight together.
constexpr int kActUnits = 64;
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quantize_act_kernel(const T* __restrict__ x, int64_t ld, int rows, int K,
                                                                     int KB, int how, uint8_t* __restrict__ codes,
                                                                     uint32_t* __restrict__ sf, uint32_t* status) {
  constexpr int U = kActUnits / 32;
  const int row = blockIdx.x * (kQuantThreads / 32) + threadIdx.x / 32, cols = KB * 8;
  const int c0 = blockIdx.y * kActUnits + threadIdx.x % 32;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = 0;
  if (row >= rows) return;
  Unit<T> u[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int k = (c0 + 32 * i) * kUnit;
    u[i] = k < K ? load_unit(x + row * ld + k, how) : zero_unit<T>();
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int c = c0 + 32 * i;
    uint32_t sc;
    const uint2 q = quantize_unit(u[i], &sc);
    uint32_t word = sc << (8 * ((c / 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    if (c < cols) {  // a multiple of 8: a word's lanes agree
      *reinterpret_cast<uint2*>(codes + (static_cast<int64_t>(row) * cols + c) * 8) = q;
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

// Grids of at least a block per SM are dependent launches: 28672 x 4096 there and back 99.6 us
// without, 95.9 with; below, the launch itself is what a call takes, and a dependent one
// costs the host 0.7 us more.
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
    const int blocks = unit_blocks(units, num_sms);
    return launch_kernel(blocks >= num_sms, quantize_kernel<T>, blocks, kQuantThreads, 0, st,
                         static_cast<const T*>(x), ld, units, cols, how_aligned(x, cols == 0 ? 0 : ld, sizeof(T)), codes,
                         scale);
  });
}

cudaError_t launch_dequantize_fp4(int dtype, const uint8_t* codes, const uint8_t* scale, int64_t blocks, void* out,
                                  int num_sms, cudaStream_t st) {
  const int64_t units = blocks * 2;
  return with_dtype(dtype, [&](auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    const int blocks = unit_blocks(units, num_sms);
    return launch_kernel(blocks >= num_sms, dequantize_kernel<T>, blocks, kQuantThreads, 0, st, codes, scale,
                         units, reinterpret_cast<uintptr_t>(codes) % 8 == 0, how_aligned(out, 0, sizeof(T)),
                         static_cast<T*>(out));
  });
}

cudaError_t launch_quantize_act(int dtype, const void* x, int64_t ld, int T, int K, uint8_t* codes, uint32_t* sf,
                                uint32_t* status, cudaStream_t st) {
  const int KB = ceil_div(K, 128);
  const dim3 grid(ceil_div(T, kQuantThreads / 32), ceil_div(KB * 8, kActUnits));
  return with_dtype(dtype, [&](auto* p) {
    using E = std::remove_pointer_t<decltype(p)>;
    return launch_kernel(true, quantize_act_kernel<E>, grid, kQuantThreads, 0, st, static_cast<const E*>(x), ld, T, K,
                         KB, how_aligned(x, ld, sizeof(E)), codes, sf, status);
  });
}

}  // namespace bsmoe
