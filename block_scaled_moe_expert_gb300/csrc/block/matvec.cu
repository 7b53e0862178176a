// Products of a few tokens with 4-bit weights and group scales:
//   y[t, n] = sum over groups g of scale[n, g] * sum_{k in g} x[t, k] code[n, k].
//
// Bound by the stream of weights from DRAM (half a byte and 1/32 of a scale
// per weight against 2 T operations), so everything is arranged around it:
// the weights are laid out once in blocks of 16 rows x 128 k that a warp
// reads as two 16-byte loads a lane plus the block's scales, the next blocks
// are in flight while one is multiplied, and the multiplication itself is
// kept off the critical path by the 16x8x16 tensor-core instruction (its
// fp32 accumulation is what the sums need; 8 tokens cost what one costs; the
// tcgen05 instructions would take the same weights through shared memory in a
// type that their operand tables do not pair with 16-bit activations). Codes
// become fp16 in registers, exactly; the group scale multiplies the group's
// fp32 sums.
//
// x is staged in shared memory as fp16. The 128 elements of a bf16 row that
// meet one block are scaled by a power of two that brings their largest finite
// value to [2^14, 2^15): fp16 then holds every element exactly down to 2^-29
// of the largest, and below that with an error under 2^-40 of the largest, far
// below the fp32 sums' own. The power is taken back on each group's sums.
#include <cooperative_groups.h>
#include <cmath>
#include <type_traits>

#include "block_internal.cuh"
#include "../ptx.cuh"

namespace cg = cooperative_groups;

namespace bsmoe {

namespace {

constexpr int kMvWarps = 16;
constexpr int kMvThreads = kMvWarps * 32;
constexpr int kMvRows = 16;    // weight rows of a block (the instruction's M)
constexpr int kMvStep = 128;   // k of a block
constexpr int kMvDepth = 4;    // blocks in flight per warp
constexpr int kMvTokens = 16;  // tokens of a pass, two N = 8 tiles
constexpr int kMvMaxSmem = 184 * 1024;  // for x
constexpr int kMvMaxCluster = 8;
template <typename X>
constexpr bool kScaledX = std::is_same<X, __nv_bfloat16>::value;
constexpr int kCodeBytes = kMvRows * kMvStep / 2;

// Block of 16 rows x 128 k: 1024 bytes of codes, then the scales.
// Lane l = 4 g + q reads code words (16 j + 4 i) bytes into 512 h + 16 l:
// word i of half h = row g + 8 (i & 1), k = 64 h + 32 (i >> 1) + 8 q .. + 7.
// FP4 words hold the codes in k order; INT4 words hold code 2p of the eight
// at bits 4p and code 2p + 1 at bits 16 + 4p, so that a shift and a mask give
// a pair in the halves of a register.
// Scales, FP4: 8 bytes for each g: rows g and g + 8, 4 groups each. INT4: for
// each g, per group of the block, rows g and g + 8: scale (16 bits), then
// 1024 + zero as fp16.
__host__ __device__ constexpr int block_bytes(int fmt, int group) {
  return kCodeBytes + (fmt == MOE_Q_FP4 ? 64 : 64 * (kMvStep / group));
}

struct MvArgs {
  const uint8_t* prepared;
  const void* x;
  void* y;
  int64_t ld_x;
  int T, N, K, tiles, steps;  // tiles of 16 rows, blocks along K
  int out_cols;
  int warps_k;   // warps that share a tile's K range
  int cluster;   // CTAs that share a tile's K range
  float limit;
  bool swiglu;
  bool x_vec;  // rows of x allow 16-byte loads
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The eight e2m1 codes of a word as fp16 pairs, in order.
__device__ __forceinline__ void fp4_pairs(uint32_t word, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(word));
}
// Four UE8M0 bytes as floats (bf16 holds them all; 255 is NaN).
__device__ __forceinline__ void ue8m0_scales(uint32_t word, float (&s)[4]) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(word));
  s[0] = __uint_as_float(lo << 16);
  s[1] = __uint_as_float(lo & 0xFFFF0000u);
  s[2] = __uint_as_float(hi << 16);
  s[3] = __uint_as_float(hi & 0xFFFF0000u);
}
// The eight codes of a word minus zero as fp16 pairs: with the bits of 1024
// above a code the half is 1024 + code, or 1024 + 16 code where the code sits
// four bits up; both differences are exact. zero: 1024 + z.
__device__ __forceinline__ void int4_pairs(uint32_t word, __half2 zero, uint32_t (&h)[4]) {
  const __half2 up = __float2half2_rn(0.0625f);
  const __half2 zero16 = __hsub2(__float2half2_rn(960.f), zero);  // -(64 + z)
#pragma unroll
  for (int p = 0; p < 4; p += 2) {
    const uint32_t w = word >> (4 * p);
    const uint32_t a = (w & 0x000F000Fu) | 0x64006400u, b = (w & 0x00F000F0u) | 0x64006400u;
    const __half2 va = __hsub2(*reinterpret_cast<const __half2*>(&a), zero);
    const __half2 vb = __hfma2(*reinterpret_cast<const __half2*>(&b), up, zero16);
    h[p] = *reinterpret_cast<const uint32_t*>(&va);
    h[p + 1] = *reinterpret_cast<const uint32_t*>(&vb);
  }
}

// What a warp holds of one block.
template <int SW>
struct Block {
  uint4 codes[2];
  uint32_t scale[SW];
};

template <int SW>
__device__ __forceinline__ void load_block(Block<SW>& b, const uint8_t* p, int lane) {
  b.codes[0] = __ldcs(reinterpret_cast<const uint4*>(p) + lane);
  b.codes[1] = __ldcs(reinterpret_cast<const uint4*>(p) + 32 + lane);
  const uint8_t* s = p + kCodeBytes + (lane >> 2) * (4 * SW);
#pragma unroll
  for (int i = 0; i < SW; i += 2) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(s) + i / 2);
    b.scale[i] = v.x;
    b.scale[i + 1] = v.y;
  }
}

// acc += block x tokens. GROUPS: scale groups per block (4, 2 or 1). xs: the
// tokens' rows at the block's k, x_scale: their powers for this block.
template <int FMT, int GROUPS, int NT, typename S, typename X, int SW>
__device__ __forceinline__ void multiply_block(float (&acc)[NT][4], const Block<SW>& b, const uint8_t* xs,
                                               int x_stride, const float* x_scale, int T, int lane) {
  const int g = lane >> 2, q = lane & 3;
  float scale[2][4];
  if constexpr (FMT == MOE_Q_FP4) {
    ue8m0_scales(b.scale[0], scale[0]);
    ue8m0_scales(b.scale[1], scale[1]);
  }
  float2 back[NT];
  if constexpr (kScaledX<X>) {
#pragma unroll
    for (int n = 0; n < NT; ++n) back[n] = *reinterpret_cast<const float2*>(x_scale + n * 8 + 2 * q);
  }
  float c[NT][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 32 k each
    uint4 xv[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      xv[n] = (n * 8 + g < T) ? *reinterpret_cast<const uint4*>(xs + (n * 8 + g) * x_stride + i * 64 + q * 16)
                              : make_uint4(0, 0, 0, 0);
    const uint32_t w0 = (i & 1) ? b.codes[i >> 1].z : b.codes[i >> 1].x;
    const uint32_t w1 = (i & 1) ? b.codes[i >> 1].w : b.codes[i >> 1].y;
    const bool first = (i * GROUPS) % 4 == 0, last = ((i + 1) * GROUPS) % 4 == 0;
    const int grp = i * GROUPS / 4;
    uint32_t a0[4], a1[4];
    float s0, s1;
    if constexpr (FMT == MOE_Q_FP4) {
      fp4_pairs(w0, a0);
      fp4_pairs(w1, a1);
      s0 = scale[0][i];
      s1 = scale[1][i];
    } else {
      const uint32_t sz0 = b.scale[2 * grp], sz1 = b.scale[2 * grp + 1];
      int4_pairs(w0, __half2half2(__ushort_as_half(sz0 >> 16)), a0);
      int4_pairs(w1, __half2half2(__ushort_as_half(sz1 >> 16)), a1);
      const uint16_t h0 = sz0 & 0xFFFF, h1 = sz1 & 0xFFFF;
      s0 = to_f32(*reinterpret_cast<const S*>(&h0));
      s1 = to_f32(*reinterpret_cast<const S*>(&h1));
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (first) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
      mma_16816(c[n], a0[0], a1[0], a0[1], a1[1], xv[n].x, xv[n].y);
      mma_16816(c[n], a0[2], a1[2], a0[3], a1[3], xv[n].z, xv[n].w);
      if (last) {
        if constexpr (kScaledX<X>) {
          c[n][0] *= back[n].x;
          c[n][1] *= back[n].y;
          c[n][2] *= back[n].x;
          c[n][3] *= back[n].y;
        }
        acc[n][0] = fmaf(s0, c[n][0], acc[n][0]);
        acc[n][1] = fmaf(s0, c[n][1], acc[n][1]);
        acc[n][2] = fmaf(s1, c[n][2], acc[n][2]);
        acc[n][3] = fmaf(s1, c[n][3], acc[n][3]);
      }
    }
  }
}

// A lane's sums: rows g and g + 8 of the tile for tokens 2q, 2q + 1.
template <typename X, int NT>
__device__ __forceinline__ void store_tile(const MvArgs& a, int tile, const float (&acc)[NT][4], int lane) {
  const int g = lane >> 2, q = lane & 3;
  X* y = static_cast<X*>(a.y);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = n * 8 + 2 * q + i;
      if (t >= a.T) continue;
      float lo = acc[n][i], hi = acc[n][2 + i];
      if (a.swiglu) {
        const int col = tile * 8 + g;
        if (a.limit > 0.f) {
          lo = lo > a.limit ? a.limit : lo;  // NaN stays NaN
          hi = hi > a.limit ? a.limit : hi < -a.limit ? -a.limit : hi;
        }
        if (col < a.out_cols)
          y[static_cast<size_t>(t) * a.out_cols + col] = from_f32<X>(lo / (1.f + expf(-lo)) * hi);
      } else {
        const int col = tile * kMvRows + g;
        if (col < a.out_cols) y[static_cast<size_t>(t) * a.out_cols + col] = from_f32<X>(lo);
        if (col + 8 < a.out_cols) y[static_cast<size_t>(t) * a.out_cols + col + 8] = from_f32<X>(hi);
      }
    }
  }
}

// Tiles are dealt round by round to groups of warps_k warps; the warps of a
// group (and the CTAs of a cluster, one tile each then) share the tile's K
// range in order and their sums are added in that order.
template <int FMT, int GROUPS, int NT, typename S, typename X>
__global__ void __launch_bounds__(kMvThreads, 1) matvec_kernel(MvArgs a) {
  constexpr int SW = FMT == MOE_Q_FP4 ? 2 : 2 * GROUPS;
  extern __shared__ __align__(16) uint8_t s_x[];
  __shared__ float s_red[2][kMvWarps][NT][4][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = a.cluster > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int first_step = static_cast<int>(static_cast<int64_t>(a.steps) * rank / a.cluster);
  const int cta_steps = static_cast<int>(static_cast<int64_t>(a.steps) * (rank + 1) / a.cluster) - first_step;
  const int wk = warp % a.warps_k, group = warp / a.warps_k, groups = kMvWarps / a.warps_k;
  const int s0 = cta_steps * wk / a.warps_k, ns = cta_steps * (wk + 1) / a.warps_k - s0;
  const int bytes = block_bytes(FMT, kMvStep / GROUPS);
  const int cluster_id = blockIdx.x / a.cluster, clusters = gridDim.x / a.cluster;
  const int tile0 = cluster_id * groups + group, tile_step = clusters * groups;
  const int rounds = (a.tiles - cluster_id * groups + tile_step - 1) / tile_step;  // of this CTA
  pdl_wait();
  pdl_launch_dependents();

  Block<SW> ring[kMvDepth];
  // cursor of the next block to load
  int ld_tile = tile0, ld_s = 0;
  auto advance = [&](Block<SW>& slot) {
    if (ld_tile < a.tiles) {
      load_block(slot, a.prepared + (static_cast<size_t>(ld_tile) * a.steps + first_step + s0 + ld_s) * bytes, lane);
      if (++ld_s == ns) {
        ld_s = 0;
        ld_tile += tile_step;
      }
    }
  };
#pragma unroll
  for (int d = 0; d < kMvDepth; ++d) advance(ring[d]);

  // x: this CTA's K range as fp16, rows 64 bytes apart modulo 128 (the four
  // 16-byte reads of two tokens fill the banks), then the powers [step][token]
  const int x_stride = cta_steps * kMvStep * 2 + 64;
  float* s_power = reinterpret_cast<float*>(s_x + static_cast<size_t>(a.T) * x_stride);
  const X* x = static_cast<const X*>(a.x);
  for (int unit = tid >> 4; unit < a.T * cta_steps; unit += kMvThreads / 16) {
    const int t = unit / cta_steps, step = unit - t * cta_steps;
    const int at = step * kMvStep + (lane & 15) * 8, k = first_step * kMvStep + at;
    Pack<X, 8> p;
    if (a.x_vec && k < a.K) {
      p = load_pack<8>(x + t * a.ld_x + k);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) p.e[i] = k < a.K ? x[t * a.ld_x + k + i] : from_f32<X>(0.f);
    }
    uint4 out;
    if constexpr (kScaledX<X>) {
      float f[8], m = 0.f;
      unpack(p, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fabsf(f[i]) < INFINITY ? fmaxf(m, fabsf(f[i])) : m;
      const unsigned half = 0xFFFFu << (lane & 16);  // the units of a warp end apart
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(half, m, o));
      // 2^(14 - e) and back, e the exponent of m (at least -112: both are normal)
      const int e = max(15, static_cast<int>(__float_as_uint(m) >> 23));
      const float scale = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
      uint32_t* w = &out.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(f[2 * i] * scale, f[2 * i + 1] * scale);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if ((lane & 15) == 0) s_power[step * kMvTokens + t] = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
    } else {
      out = *reinterpret_cast<const uint4*>(&p);
    }
    *reinterpret_cast<uint4*>(s_x + static_cast<size_t>(t) * x_stride + at * 2) = out;
  }
  __syncthreads();

  const uint8_t* xs = s_x + s0 * (kMvStep * 2);
  const float* xp = s_power + s0 * kMvTokens;
  float acc[NT][4] = {};
  int tile = tile0, s = 0;
  int parity = 0;
  auto finish = [&]() {  // the tile's sums are complete in this warp
    if (a.warps_k > 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_red[parity][warp][n][i][lane] = acc[n][i];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(a.warps_k * 32) : "memory");
      if (wk == 0) {
        for (int w = 1; w < a.warps_k; ++w)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] += s_red[parity][warp + w][n][i][lane];
      }
      parity ^= 1;
    }
    if (wk == 0 && a.cluster == 1 && tile < a.tiles) store_tile<X, NT>(a, tile, acc, lane);
  };
  if (a.cluster > 1) {
    // one tile: the whole CTA shares it
    for (int i = 0; i < ns; i += kMvDepth) {
#pragma unroll
      for (int d = 0; d < kMvDepth; ++d) {
        if (i + d >= ns) break;
        multiply_block<FMT, GROUPS, NT, S, X>(acc, ring[d], xs + (i + d) * (kMvStep * 2), x_stride,
                                                xp + (i + d) * kMvTokens, a.T, lane);
        advance(ring[d]);
      }
    }
    finish();
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // rank 0 runs, and is done with its own sums
    if (warp == 0) {
      float* to = cluster.map_shared_rank(&s_red[1][0][0][0][0], 0) + rank * (NT * 128);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) to[(n * 4 + i) * 32 + lane] = acc[n][i];
    }
    cluster.sync();
    if (rank == 0 && warp == 0) {
      for (int r = 1; r < a.cluster; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] += (&s_red[1][0][0][0][0])[r * (NT * 128) + (n * 4 + i) * 32 + lane];
      store_tile<X, NT>(a, tile, acc, lane);
    }
    return;
  }
  const int total = rounds * ns;
  for (int i = 0; i < total; i += kMvDepth) {
#pragma unroll
    for (int d = 0; d < kMvDepth; ++d) {
      if (i + d >= total) break;
      if (tile < a.tiles)
        multiply_block<FMT, GROUPS, NT, S, X>(acc, ring[d], xs + s * (kMvStep * 2), x_stride, xp + s * kMvTokens,
                                                a.T, lane);
      advance(ring[d]);
      if (++s == ns) {
        finish();
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        s = 0;
        tile += tile_step;
      }
    }
  }
}

// ------------------------------------------------------------------ layout

// One thread per code word of the prepared weights, then the block's scales.
template <int FMT>
__global__ void __launch_bounds__(256)
matvec_prepare_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scale,
                      const uint8_t* __restrict__ zero, uint8_t* __restrict__ out, int N, int K, int group,
                      bool swiglu, int steps) {
  pdl_wait();
  pdl_launch_dependents();
  const int tile = blockIdx.x, step = blockIdx.y;
  const int bytes = block_bytes(FMT, group), per_row = (K + group - 1) / group;
  uint8_t* dst = out + (static_cast<size_t>(tile) * steps + step) * bytes;
  auto source_row = [&](int r) {  // row r of the tile -> row of W, -1: padding
    if (!swiglu) {
      const int n = tile * kMvRows + r;
      return n < N ? n : -1;
    }
    const int n = tile * 8 + (r & 7);
    return n < N / 2 ? n + (r >> 3) * (N / 2) : -1;
  };
  {
    const int w = threadIdx.x, half = w >> 7, lane = (w >> 2) & 31, i = w & 3;
    const int n = source_row((lane >> 2) + 8 * (i & 1));
    const int k = step * kMvStep + half * 64 + (i >> 1) * 32 + (lane & 3) * 8;
    uint32_t v = 0;
    if (n >= 0 && k < K) {
      const uint8_t* src = codes + static_cast<size_t>(n) * (K / 2) + k / 2;
#pragma unroll
      for (int j = 0; j < 4; ++j) v |= static_cast<uint32_t>(src[j]) << (8 * j);
    }
    if (FMT == MOE_Q_INT4) {
      uint32_t p = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p |= ((v >> (8 * j)) & 0xF) << (4 * j) | ((v >> (8 * j + 4)) & 0xF) << (16 + 4 * j);
      v = p;
    }
    reinterpret_cast<uint32_t*>(dst)[w] = v;
  }
  dst += kCodeBytes;
  const int groups = kMvStep / group;
  if (threadIdx.x < kMvRows * groups) {
    const int r = threadIdx.x / groups, grp = threadIdx.x % groups;
    const int n = source_row(r), sg = step * groups + grp;
    const bool ok = n >= 0 && sg < per_row;
    const size_t at = static_cast<size_t>(n) * per_row + sg;
    if (FMT == MOE_Q_FP4) {
      dst[(r & 7) * 8 + (r >> 3) * 4 + grp] = ok ? scale[at] : 0;
    } else {
      const uint16_t s = ok ? reinterpret_cast<const uint16_t*>(scale)[at] : 0;
      const int z = ok && zero != nullptr ? zero[at] : 8;
      const uint16_t zb = __half_as_ushort(__int2half_rn(1024 + z));
      reinterpret_cast<uint32_t*>(dst)[(r & 7) * (2 * groups) + 2 * grp + (r >> 3)] =
          s | static_cast<uint32_t>(zb) << 16;
    }
  }
}

int row_tiles(const MatvecShape& s) { return s.swiglu ? ceil_div(s.N / 2, 8) : ceil_div(s.N, kMvRows); }

template <int FMT, int GROUPS, typename S, typename X>
cudaError_t run(const MvArgs& a, int grid, size_t smem, cudaStream_t st) {
  auto* k = a.T <= 8 ? matvec_kernel<FMT, GROUPS, 1, S, X> : matvec_kernel<FMT, GROUPS, 2, S, X>;
  if (smem > 8 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = kMvThreads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

template <int FMT, typename S, typename X>
cudaError_t run_groups(int group, const MvArgs& a, int grid, size_t smem, cudaStream_t st) {
  if (FMT == MOE_Q_FP4 || group == 32) return run<FMT, 4, S, X>(a, grid, smem, st);
  if (group == 64) return run<FMT, FMT == MOE_Q_FP4 ? 4 : 2, S, X>(a, grid, smem, st);
  return run<FMT, FMT == MOE_Q_FP4 ? 4 : 1, S, X>(a, grid, smem, st);
}

template <typename X>
cudaError_t run_format(int fmt, int scale_dtype, int group, const MvArgs& a, int grid, size_t smem, cudaStream_t st) {
  if (fmt == MOE_Q_FP4) return run_groups<MOE_Q_FP4, __half, X>(group, a, grid, smem, st);
  if (scale_dtype == MOE_BF16) return run_groups<MOE_Q_INT4, __nv_bfloat16, X>(group, a, grid, smem, st);
  return run_groups<MOE_Q_INT4, __half, X>(group, a, grid, smem, st);
}

}  // namespace

size_t matvec_prepared_bytes(const MatvecShape& s) {
  if (s.fmt != MOE_Q_FP4 && s.fmt != MOE_Q_INT4) return 0;
  if (s.K < 32 || s.K > 32768 || s.K % 32 || s.N < 1 || s.N > (1 << 20)) return 0;
  if (s.swiglu && s.N % 2) return 0;
  if (s.group != 32 && (s.fmt == MOE_Q_FP4 || (s.group != 64 && s.group != 128))) return 0;
  return static_cast<size_t>(row_tiles(s)) * ceil_div(s.K, kMvStep) * block_bytes(s.fmt, s.group);
}

cudaError_t launch_matvec_prepare(const MatvecShape& s, const void* codes, const void* scale, int scale_dtype,
                                  const void* zero, void* prepared, cudaStream_t st) {
  const int steps = ceil_div(s.K, kMvStep), tiles = row_tiles(s);
  auto* k = s.fmt == MOE_Q_FP4 ? matvec_prepare_kernel<MOE_Q_FP4> : matvec_prepare_kernel<MOE_Q_INT4>;
  return launch_kernel(false, k, dim3(tiles, steps), 256, 0, st, static_cast<const uint8_t*>(codes),
                       static_cast<const uint8_t*>(scale), static_cast<const uint8_t*>(zero),
                       static_cast<uint8_t*>(prepared), s.N, s.K, s.group, s.swiglu != 0, steps);
}

cudaError_t launch_matvec(const MatvecShape& s, float limit, int scale_dtype, const void* prepared, int dtype,
                          const void* x, int64_t ld_x, int T, void* y, int num_sms, cudaStream_t st) {
  MvArgs a;
  a.prepared = static_cast<const uint8_t*>(prepared);
  a.ld_x = ld_x;
  a.N = s.N;
  a.K = s.K;
  a.tiles = row_tiles(s);
  a.steps = ceil_div(s.K, kMvStep);
  a.out_cols = s.swiglu ? s.N / 2 : s.N;
  a.limit = limit > 0.f && std::isfinite(limit) ? limit : 0.f;
  a.swiglu = s.swiglu != 0;
  // K is shared by enough warps to give every SM a few rounds of tiles, and
  // by the CTAs of a cluster where the tiles alone leave SMs idle.
  a.cluster = 1;
  a.warps_k = 1;
  while (a.warps_k < kMvWarps && a.tiles * a.warps_k < 4 * kMvWarps * num_sms && a.steps >= 4 * a.warps_k)
    a.warps_k *= 2;
  if (a.warps_k == kMvWarps)
    while (a.cluster < kMvMaxCluster && a.tiles * a.cluster * 2 <= num_sms && a.steps >= 2 * kMvWarps * a.cluster)
      a.cluster *= 2;
  const int cta_k = ceil_div(a.steps, a.cluster) * kMvStep;
  // of a token: fp16 and its place among the powers
  const int x_row = 2 * cta_k + 64, power = cta_k / kMvStep * kMvTokens * 4;
  const int pass = std::max(1, std::min<int>(kMvTokens, (kMvMaxSmem - power) / x_row));
  const int cta_tiles = ceil_div(a.tiles, kMvWarps / a.warps_k);
  const int grid = a.cluster > 1 ? a.tiles * a.cluster : std::min(cta_tiles, num_sms);
  const size_t es = 2;
  for (int t0 = 0; t0 < T; t0 += pass) {
    a.T = std::min(pass, T - t0);
    a.x_vec = aligned16(x) && ld_x % 8 == 0;
    a.x = static_cast<const uint8_t*>(x) + static_cast<size_t>(t0) * ld_x * es;
    a.y = static_cast<uint8_t*>(y) + static_cast<size_t>(t0) * a.out_cols * es;
    const size_t smem = static_cast<size_t>(a.T) * x_row + power;
    const cudaError_t e = dtype == MOE_BF16 ? run_format<__nv_bfloat16>(s.fmt, scale_dtype, s.group, a, grid, smem, st)
                                            : run_format<__half>(s.fmt, scale_dtype, s.group, a, grid, smem, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace bsmoe
