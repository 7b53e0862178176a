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
// Measured, a call among others: FP4 131072 x 4096, one token 43.7 us, 6.5 TB/s,
// 96% of a plain copy's rate; FP4 4096 x 7168 with SwiGLU, one token 6.2 us;
// INT4 28671 x 4096, 7 tokens 15 us, 4.1 TB/s, where the fixed 4 us of launch,
// staging and joining and the conversion of the codes (13 cycles a word of
// eight, FP4 8) take their part. Without the ring in shared memory (blocks
// loaded into registers four ahead) the first took 88 us: the scoreboard makes
// a warp wait for more than the block it needs.
//
// x is staged in shared memory as fp16. The 128 elements of a bf16 row that
// meet one block are scaled by a power of two that brings their largest finite
// value to [2^14, 2^15): fp16 then holds every element exactly that is at least
// 2^-31 of the largest. The power is taken back on each group's sums before the
// group's scale. A CTA that meets an element that fp16 does not hold (or a block
// with a value of 2^96 or more, whose sums could leave fp32's range before the
// scale brings them back) says so while it stages, and takes x as it is instead:
// bf16 through the bf16 instruction, with codes that bf16 holds just as exactly.
// Then nothing is lost over bf16's whole range. The conversion of the codes costs
// more there, so that this is the way of the few rows that need it (131072 x 4096,
// one token: 78 us against 44).
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
constexpr int kMvTokens = 16;  // tokens of a pass, two N = 8 tiles
constexpr int kMvMaxSmem = 227 * 1024 - 18 * 1024;  // for x and the blocks in flight, beside the sums' join
constexpr int kMvMaxCluster = 8;
template <typename X>
constexpr bool kScaledX = std::is_same<X, __nv_bfloat16>::value;
constexpr int kMvHuge = 96;  // exponent from which bf16 activations are taken as they are
// Codes that meet bf16 activations are held times this power, so that the sums
// of a group's products stay below 2^128: 32 of 6 2^128, or 128 of 255 2^128.
template <int FMT>
constexpr float kWideCode = FMT == MOE_Q_FP4 ? 1.f / 256 : 1.f / 65536;
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

// X: the type of both operands.
template <typename X>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  if constexpr (std::is_same<X, __nv_bfloat16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
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
// four bits up; both differences are exact. zero: 1024 + z, zero16: -(64 + z).
// (In PTX: from the half intrinsics the compiler made 20 cycles a word, not 13.)
__device__ __forceinline__ uint32_t code_bits(uint32_t word, uint32_t mask) {
  uint32_t d;  // (word & mask) | 0x64006400
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(word), "r"(mask), "r"(0x64006400u));
  return d;
}
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t half2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ void int4_pairs(uint32_t word, uint32_t zero, uint32_t zero16, uint32_t (&h)[4]) {
  const uint32_t up = word >> 8, sixteenth = 0x2C002C00u;
  h[0] = half2_sub(code_bits(word, 0x000F000Fu), zero);
  h[1] = half2_fma(code_bits(word, 0x00F000F0u), sixteenth, zero16);
  h[2] = half2_sub(code_bits(up, 0x000F000Fu), zero);
  h[3] = half2_fma(code_bits(up, 0x00F000F0u), sixteenth, zero16);
}

// fp16 pairs of codes as bf16 pairs times kWideCode, exactly.
template <int FMT>
__device__ __forceinline__ void wide_pairs(uint32_t (&h)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = pack2(mul2(unpack2(h[i], __half()), make_float2(kWideCode<FMT>, kWideCode<FMT>)), __nv_bfloat16());
}

// What a lane holds of one block.
template <int SW>
struct Block {
  uint4 codes[2];
  uint32_t scale[SW];
};

// A block's way from global memory through a warp's ring.
template <int BYTES>
__device__ __forceinline__ void fetch_block(uint8_t* slot, const uint8_t* p, int lane) {
  cp_async16(slot + lane * 16, p + lane * 16);
  cp_async16(slot + 512 + lane * 16, p + 512 + lane * 16);
  if (lane < (BYTES - kCodeBytes) / 16) cp_async16(slot + kCodeBytes + lane * 16, p + kCodeBytes + lane * 16);
}
template <int SW>
__device__ __forceinline__ void read_block(Block<SW>& b, const uint8_t* slot, int lane) {
  b.codes[0] = *reinterpret_cast<const uint4*>(slot + lane * 16);
  b.codes[1] = *reinterpret_cast<const uint4*>(slot + 512 + lane * 16);
  const uint8_t* s = slot + kCodeBytes + (lane >> 2) * (4 * SW);
#pragma unroll
  for (int i = 0; i < SW; i += 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(s + 4 * i);
    b.scale[i] = v.x;
    b.scale[i + 1] = v.y;
  }
}

// acc += block x tokens. GROUPS: scale groups per block (4, 2 or 1). xs: this
// lane's part of its token's row at the block's k, x_scale: the tokens' powers
// for this block. WIDE: x is bf16 as it is, without powers.
template <int FMT, int GROUPS, int NT, bool WIDE, typename S, typename X, int SW>
__device__ __forceinline__ void multiply_block(float (&acc)[NT][4], const Block<SW>& b,
                                               const uint8_t* const (&xs)[NT], const float* x_scale, int lane) {
  const int q = lane & 3;
  float scale[2][4];
  if constexpr (FMT == MOE_Q_FP4) {
    ue8m0_scales(b.scale[0], scale[0]);
    ue8m0_scales(b.scale[1], scale[1]);
  }
  constexpr bool POWERS = kScaledX<X> && !WIDE;
  using Operand = std::conditional_t<WIDE, __nv_bfloat16, __half>;
  float2 back[NT];
  if constexpr (POWERS) {
#pragma unroll
    for (int n = 0; n < NT; ++n) back[n] = *reinterpret_cast<const float2*>(x_scale + n * 8 + 2 * q);
  }
  float c[NT][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 32 k each
    uint4 xv[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      xv[n] = *reinterpret_cast<const uint4*>(xs[n] + i * 64);
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
      const uint32_t z0 = __byte_perm(sz0, 0, 0x3232), z1 = __byte_perm(sz1, 0, 0x3232);
      int4_pairs(w0, z0, half2_sub(0x63806380u, z0), a0);  // 960 - (1024 + z)
      int4_pairs(w1, z1, half2_sub(0x63806380u, z1), a1);
      const uint16_t h0 = sz0 & 0xFFFF, h1 = sz1 & 0xFFFF;
      s0 = to_f32(*reinterpret_cast<const S*>(&h0));
      s1 = to_f32(*reinterpret_cast<const S*>(&h1));
    }
    if constexpr (WIDE) {
      wide_pairs<FMT>(a0);
      wide_pairs<FMT>(a1);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (first) mma_16816<Operand>(c[n], a0[0], a1[0], a0[1], a1[1], xv[n].x, xv[n].y, 0.f, 0.f, 0.f, 0.f);
      else mma_16816<Operand>(c[n], a0[0], a1[0], a0[1], a1[1], xv[n].x, xv[n].y, c[n][0], c[n][1], c[n][2], c[n][3]);
      mma_16816<Operand>(c[n], a0[2], a1[2], a0[3], a1[3], xv[n].z, xv[n].w, c[n][0], c[n][1], c[n][2], c[n][3]);
      if (last) {
        float2 lo = make_float2(c[n][0], c[n][1]), hi = make_float2(c[n][2], c[n][3]);
        float2 scale_lo = make_float2(s0, s0), scale_hi = make_float2(s1, s1);
        if constexpr (POWERS) {
          lo = mul2(lo, back[n]);
          hi = mul2(hi, back[n]);
        }
        if constexpr (WIDE) {  // the codes' power after the scale, see kWideCode
          lo = mul2(lo, scale_lo);
          hi = mul2(hi, scale_hi);
          scale_lo = scale_hi = make_float2(1.f / kWideCode<FMT>, 1.f / kWideCode<FMT>);
        }
        lo = fma2(lo, scale_lo, make_float2(acc[n][0], acc[n][1]));
        hi = fma2(hi, scale_hi, make_float2(acc[n][2], acc[n][3]));
        acc[n][0] = lo.x;
        acc[n][1] = lo.y;
        acc[n][2] = hi.x;
        acc[n][3] = hi.y;
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

template <int FMT, int GROUPS, int NT, int DEPTH, typename S, typename X>
__device__ __noinline__ void matvec_cta_wide(const MvArgs a, uint8_t* s_dyn, float (*s_red)[NT][4][32],
                                             uint8_t* s_zero);

// What a CTA does. Tiles are dealt round by round to groups of warps_k warps; the
// warps of a group (and the CTAs of a cluster, one tile each then) share the
// tile's K range in order and their sums are added in that order. DEPTH: blocks
// that a warp has in flight or in work. WIDE: bf16 x as it is, which is where a
// CTA goes whose x does not fit into fp16. That way is a function of its own, and
// the CTA's answer goes through shared memory (behind s_zero): 131072 x 4096, one
// token, takes 43.9 us so, and 46.2 with the barrier's own vote or with the
// arguments passed by reference.
template <int FMT, int GROUPS, int NT, int DEPTH, bool WIDE, typename S, typename X>
__device__ __forceinline__ void matvec_cta(const MvArgs a, uint8_t* s_dyn, float (*s_red)[NT][4][32],
                                           uint8_t* s_zero) {
  constexpr int SW = FMT == MOE_Q_FP4 ? 2 : 2 * GROUPS;
  constexpr int BYTES = block_bytes(FMT, kMvStep / GROUPS);
  constexpr bool SCALED = kScaledX<X> && !WIDE;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same for the warp's lanes, as the compiler now knows
  const int rank = a.cluster > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  const int first_step = static_cast<int>(static_cast<int64_t>(a.steps) * rank / a.cluster);
  const int cta_steps = static_cast<int>(static_cast<int64_t>(a.steps) * (rank + 1) / a.cluster) - first_step;
  const int wk = warp % a.warps_k, group = warp / a.warps_k, groups = kMvWarps / a.warps_k;
  const int s0 = cta_steps * wk / a.warps_k, ns = cta_steps * (wk + 1) / a.warps_k - s0;
  const int cluster_id = blockIdx.x / a.cluster, clusters = gridDim.x / a.cluster;
  const int tile0 = cluster_id * groups + group, tile_step = clusters * groups;
  const int rounds = (a.tiles - cluster_id * groups + tile_step - 1) / tile_step;  // of this CTA
  uint8_t* ring = s_dyn + warp * (DEPTH * BYTES);
  uint8_t* s_x = s_dyn + kMvWarps * DEPTH * BYTES;

  // the next block to fetch, and its slot
  int f_tile = tile0, f_s = 0, f_slot = 0;
  const uint8_t* f_at = a.prepared + (static_cast<size_t>(tile0) * a.steps + first_step + s0) * BYTES;
  const size_t tile_bytes = static_cast<size_t>(a.steps) * BYTES;
  auto fetch = [&]() {
    if (f_tile < a.tiles) {
      fetch_block<BYTES>(ring + f_slot, f_at, lane);
      f_at += BYTES;
      if (++f_s == ns) {
        f_s = 0;
        f_tile += tile_step;
        f_at += tile_step * tile_bytes - static_cast<size_t>(ns) * BYTES;
      }
    }
    cp_async_commit();
    f_slot = f_slot + BYTES == DEPTH * BYTES ? 0 : f_slot + BYTES;
  };
#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d) fetch();
  // The weights are on their way before the kernel in front has finished: they
  // were laid out before it (the layout kernel lets nothing start before its
  // end). x and y are touched after it.
  if (!WIDE) {
    pdl_wait();
    pdl_launch_dependents();
  }

  // x: this CTA's K range as fp16, rows 64 bytes apart modulo 128 (the four
  // 16-byte reads of two tokens fill the banks), then the powers [step][token]
  const int x_stride = cta_steps * kMvStep * 2 + 64;
  float* s_power = reinterpret_cast<float*>(s_x + static_cast<size_t>(a.T) * x_stride);
  const X* x = static_cast<const X*>(a.x);
  constexpr int kAhead = 8;  // loads in flight
  bool inexact = false;  // some element does not come out as scaled fp16
  for (int unit0 = tid >> 4; unit0 < a.T * cta_steps; unit0 += kAhead * (kMvThreads / 16)) {
    Pack<X, 8> p[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int unit = unit0 + j * (kMvThreads / 16);
      if (unit >= a.T * cta_steps) continue;
      const int t = unit / cta_steps, k = (first_step + unit - t * cta_steps) * kMvStep + (lane & 15) * 8;
      if (a.x_vec && k < a.K) {
        p[j] = load_pack<8>(x + t * a.ld_x + k);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[j].e[i] = k < a.K ? x[t * a.ld_x + k + i] : from_f32<X>(0.f);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int unit = unit0 + j * (kMvThreads / 16);
      if (unit >= a.T * cta_steps) continue;
      const int t = unit / cta_steps, step = unit - t * cta_steps;
      uint4 out;
      if constexpr (SCALED) {
        float f[8], m = 0.f;
        unpack(p[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fabsf(f[i]) < INFINITY ? fmaxf(m, fabsf(f[i])) : m;
        const unsigned half = 0xFFFFu << (lane & 16);  // the units of a warp end apart
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(half, m, o));
        // 2^(14 - e) and back, e the exponent of m (at least -112: both are normal)
        const int e = max(15, static_cast<int>(__float_as_uint(m) >> 23));
        const float scale = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
        const float back = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
        inexact |= e >= 127 + kMvHuge;
        uint32_t* w = &out.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = make_float2(f[2 * i], f[2 * i + 1]);
          w[i] = pack2(mul2(v, make_float2(scale, scale)), __half());
          const float2 held = mul2(unpack2(w[i], __half()), make_float2(back, back));
          inexact |= held.x != v.x || held.y != v.y;  // (a NaN says so too)
        }
        if ((lane & 15) == 0) s_power[step * kMvTokens + t] = back;
      } else {
        out = *reinterpret_cast<const uint4*>(&p[j]);
      }
      *reinterpret_cast<uint4*>(s_x + static_cast<size_t>(t) * x_stride + step * (kMvStep * 2) + (lane & 15) * 16) = out;
    }
  }
  // what the lanes of absent tokens read, at every step
  if (tid < kMvStep * 2 / 16) reinterpret_cast<uint4*>(s_zero)[tid] = make_uint4(0, 0, 0, 0);
  if constexpr (SCALED) {
    int* any = reinterpret_cast<int*>(s_zero + kMvStep * 2);
    if (tid == 0) *any = 0;
    __syncthreads();
    if (inexact) *any = 1;
    __syncthreads();
    if (*any) {
      cp_async_wait<0>();
      return matvec_cta_wide<FMT, GROUPS, NT, DEPTH, S, X>(a, s_dyn, s_red, s_zero);
    }
  } else {
    __syncthreads();
  }

  const uint8_t* xs[NT];  // this lane's token (in each N tile) at the warp's first block
  int xs_step[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = n * 8 + (lane >> 2);
    xs[n] = (t < a.T ? s_x + t * x_stride + s0 * (kMvStep * 2) : s_zero) + (lane & 3) * 16;
    xs_step[n] = t < a.T ? kMvStep * 2 : 0;
  }
  const float* xp = s_power + s0 * kMvTokens;
  float acc[NT][4] = {};
  int at_slot = 0;
  auto multiply = [&](const uint8_t* const (&x_at)[NT], const float* p_at) {  // the next block of the ring
    __syncwarp();  // every lane is done with the slot that is fetched into
    fetch();
    cp_async_wait<DEPTH - 1>();
    __syncwarp();  // every lane's share has arrived
    Block<SW> b;
    read_block(b, ring + at_slot, lane);
    multiply_block<FMT, GROUPS, NT, WIDE, S, X>(acc, b, x_at, p_at, lane);
    at_slot = at_slot + BYTES == DEPTH * BYTES ? 0 : at_slot + BYTES;
  };
  auto walk = [&]() {  // a tile's blocks of this warp
    const uint8_t* x_at[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x_at[n] = xs[n];
    const float* p_at = xp;
    for (int s = 0; s < ns; ++s) {
      multiply(x_at, p_at);
#pragma unroll
      for (int n = 0; n < NT; ++n) x_at[n] += xs_step[n];
      p_at += kMvTokens;
    }
  };
  auto join = [&]() {  // the sums of the group's warps, in its first one
    if (a.warps_k == 1) return;
    const int bar = 1 + group, threads = a.warps_k * 32;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");  // the join before is read
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_red[warp][n][i][lane] = acc[n][i];
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
    if (wk == 0) {
      for (int w = 1; w < a.warps_k; ++w)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] += s_red[warp + w][n][i][lane];
    }
  };
  if (a.cluster > 1) {  // one tile, which the whole CTA shares
    walk();
    join();
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // rank 0 runs, and is done with its own sums
    if (warp == 0) {
      float* to = cluster.map_shared_rank(&s_red[0][0][0][0], 0) + rank * (NT * 128);
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
          for (int i = 0; i < 4; ++i) acc[n][i] += (&s_red[0][0][0][0])[r * (NT * 128) + (n * 4 + i) * 32 + lane];
      store_tile<X, NT>(a, tile0, acc, lane);
    }
    return;
  }
  for (int r = 0, tile = tile0; r < rounds; ++r, tile += tile_step) {
    if (tile < a.tiles) walk();
    join();
    if (wk == 0 && tile < a.tiles) store_tile<X, NT>(a, tile, acc, lane);
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
  }
}

template <int FMT, int GROUPS, int NT, int DEPTH, typename S, typename X>
__device__ __noinline__ void matvec_cta_wide(const MvArgs a, uint8_t* s_dyn, float (*s_red)[NT][4][32],
                                             uint8_t* s_zero) {
  matvec_cta<FMT, GROUPS, NT, DEPTH, true, S, X>(a, s_dyn, s_red, s_zero);
}

template <int FMT, int GROUPS, int NT, int DEPTH, typename S, typename X>
__global__ void __launch_bounds__(kMvThreads, 1) matvec_kernel(MvArgs a) {
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ float s_red[kMvWarps][NT][4][32];
  // (the ring behind it has to start on a line: 16 bytes off, 131072 x 4096 takes 48.7 us)
  __shared__ __align__(128) uint8_t s_zero[kMvStep * 2 + 128];
  matvec_cta<FMT, GROUPS, NT, DEPTH, false, S, X>(a, s_dyn, s_red, s_zero);
}

// ------------------------------------------------------------------ layout

// One thread per code word of the prepared weights, then the block's scales.
template <int FMT>
__global__ void __launch_bounds__(256)
matvec_prepare_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scale,
                      const uint8_t* __restrict__ zero, uint8_t* __restrict__ out, int N, int K, int group,
                      bool swiglu, int steps) {
  // no early launch of dependents: moe_matvec fetches the weights without waiting
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

// Shared memory beside the ring: T tokens of x and their powers.
size_t x_smem(const MvArgs& a) {
  const size_t cta_steps = ceil_div(a.steps, a.cluster);
  return a.T * (cta_steps * kMvStep * 2 + 64) + cta_steps * kMvTokens * 4;
}

template <int FMT, int GROUPS, int NT, int DEPTH, typename S, typename X>
cudaError_t run(const MvArgs& a, int grid, cudaStream_t st) {
  auto* k = matvec_kernel<FMT, GROUPS, NT, DEPTH, S, X>;
  const size_t smem = kMvWarps * DEPTH * block_bytes(FMT, kMvStep / GROUPS) + x_smem(a);
  const cudaError_t e = allow_smem(k, smem, kMvMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = kMvThreads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, a);
}

// As many tokens as fit beside a ring of at least 4 blocks in one pass, at most 16; 8 blocks where they fit.
template <int FMT, int GROUPS, typename S, typename X>
cudaError_t run_passes(MvArgs a, int T, int grid, cudaStream_t st) {
  constexpr size_t ring = kMvWarps * block_bytes(FMT, kMvStep / GROUPS);
  constexpr int kMost = 8, kLeast = 4;
  a.T = std::min(T, kMvTokens);
  while (a.T > 1 && kLeast * ring + x_smem(a) > kMvMaxSmem) --a.T;
  const int pass = a.T;
  const bool deep = kMost * ring + x_smem(a) <= kMvMaxSmem;
  for (int t0 = 0; t0 < T; t0 += pass) {
    a.T = std::min(pass, T - t0);
    cudaError_t e;
    if (a.T > 8) e = deep ? run<FMT, GROUPS, 2, kMost, S, X>(a, grid, st) : run<FMT, GROUPS, 2, kLeast, S, X>(a, grid, st);
    else e = deep ? run<FMT, GROUPS, 1, kMost, S, X>(a, grid, st) : run<FMT, GROUPS, 1, kLeast, S, X>(a, grid, st);
    if (e != cudaSuccess) return e;
    a.x = static_cast<const X*>(a.x) + pass * a.ld_x;
    a.y = static_cast<X*>(a.y) + static_cast<size_t>(pass) * a.out_cols;
  }
  return cudaSuccess;
}

template <int FMT, typename S, typename X>
cudaError_t run_groups(int group, const MvArgs& a, int T, int grid, cudaStream_t st) {
  if (FMT == MOE_Q_FP4 || group == 32) return run_passes<FMT, 4, S, X>(a, T, grid, st);
  if (group == 64) return run_passes<FMT, FMT == MOE_Q_FP4 ? 4 : 2, S, X>(a, T, grid, st);
  return run_passes<FMT, FMT == MOE_Q_FP4 ? 4 : 1, S, X>(a, T, grid, st);
}

template <typename X>
cudaError_t run_format(int fmt, int scale_dtype, int group, const MvArgs& a, int T, int grid, cudaStream_t st) {
  if (fmt == MOE_Q_FP4) return run_groups<MOE_Q_FP4, __half, X>(group, a, T, grid, st);
  if (scale_dtype == MOE_BF16) return run_groups<MOE_Q_INT4, __nv_bfloat16, X>(group, a, T, grid, st);
  return run_groups<MOE_Q_INT4, __half, X>(group, a, T, grid, st);
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
  // The warps that share a tile's K range: what makes the longest warp's way
  // shortest, in blocks: its rounds of tiles, each its share of the K range and
  // a join that costs about as much as a block and a half.
  a.cluster = 1;
  a.warps_k = 1;
  float best = INFINITY;
  for (int wk = 1; wk <= kMvWarps && wk <= a.steps; wk *= 2) {
    const float rounds = static_cast<float>(ceil_div(a.tiles, kMvWarps / wk * num_sms));
    const float cost = rounds * (ceil_div(a.steps, wk) + (wk > 1 ? 1.5f : 0.f));
    if (cost < best) {
      best = cost;
      a.warps_k = wk;
    }
  }
  // and the CTAs of a cluster where the tiles alone leave SMs idle
  if (a.warps_k == kMvWarps)
    while (a.cluster < kMvMaxCluster && a.tiles * a.cluster * 2 <= num_sms && a.steps >= 2 * kMvWarps * a.cluster)
      a.cluster *= 2;
  const int cta_tiles = ceil_div(a.tiles, kMvWarps / a.warps_k);
  const int grid = a.cluster > 1 ? a.tiles * a.cluster : std::min(cta_tiles, num_sms);
  a.x = x;
  a.y = y;
  a.x_vec = aligned16(x) && ld_x % 8 == 0;
  return dtype == MOE_BF16 ? run_format<__nv_bfloat16>(s.fmt, scale_dtype, s.group, a, T, grid, st)
                           : run_format<__half>(s.fmt, scale_dtype, s.group, a, T, grid, st);
}

}  // namespace bsmoe
