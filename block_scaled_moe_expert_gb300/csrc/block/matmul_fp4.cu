// Products of many tokens with FP4 weights on the tensor cores: both operands e2m1
// in 1x32 blocks (tcgen05.mma kind::mxf4), the activations quantized by the kernel
// in front (launch_quantize_act) or, for a few tokens, by the product's own.
//
//   y[t, n] = sum_k dq(x)[t, k] * dq(W)[n, k], fp32 accumulators, one rounding;
//   with swiglu, tile columns alternate 64 gate and 64 up rows of W and the
//   epilogue stores silu(gate) * up.
//
// Large batches: pairs of CTAs (cta_group::2), persistent, one CTA per SM. A pair makes
// 256 x 256 tiles: each CTA holds 128 activation rows and 128 weight rows of a stage
// (K = 256), so that a stage is 35 KB a CTA where a CTA by itself would load 51 KB for a
// 128 x 256 tile: what the copies move from L2 is what bounds the loop. Warp 0
// of each CTA keeps five stages in flight (TMA tiles of codes and scale words, all counted on
// the leader's barriers), warp 1 of the leader issues the products of both, warps 4..11
// move the accumulators to registers, hand tensor memory back and store while the next
// tile is multiplied. 8192 x 4096 x 7168: 68 to 70 us, 6.9 PFLOP/s, the tensor pipe 72% busy;
// 8192 x 7168 x 2048: 45 us. What is left: a tile's drain before the next begins (9 us of the 70),
// copies (5), the rest products and scale copies.
#include <cuda.h>

#include "fp4.cuh"
#include "pair_ptx.cuh"

namespace bsmoe {

namespace {

constexpr int kMmThreads = 384;
constexpr int kMmEpiWarp0 = 4, kMmEpiThreads = 256;
constexpr int kMmStages = 5;
constexpr int kMmM = 128, kMmN = 256;  // rows of a CTA, columns of a pair
constexpr uint32_t kMmSfCol = 256, kMmSfCols = 24;  // per stage 8 columns of A's and 16 of B's scales
constexpr uint32_t kMmStageBytes = (kMmM + kMmN / 2) * 128 + 3 * 1024;  // of a CTA
constexpr uint32_t kMmOutBytes = 32 * 128;          // a warp's staging area: 32 rows of 64 columns

struct MmArgs {
  const uint8_t *a_sf, *w_sf;
  uint32_t* status;
  void* y;
  int T, N;  // N: columns of y
  int KB, MT, NT, swiglu;
  float limit;
  bool packs;  // rows of y are multiples of 16 bytes at 16-byte addresses
  // the stream kernel that quantizes the activations itself
  const void* x;
  int64_t ld;
  int K, how;
};

struct __align__(1024) MmSmem {
  uint8_t b[kMmStages][kMmN / 2 * 128];
  uint8_t a[kMmStages][kMmM * 128];
  uint8_t out[kMmEpiThreads / 32][kMmOutBytes];
  uint8_t sfa[kMmStages][1024];
  uint8_t sfb[kMmStages][2048];  // [128-row half][128-K chunk][512]
  // full (the leader's): both CTAs' copies; empty, tfull: the products; tempty (the leader's): both epilogues
  uint64_t full[kMmStages], empty[kMmStages], tfull, tempty;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(MmSmem) + 1024 <= 227 * 1024 && kMmSfCol + kMmStages * kMmSfCols <= 512, "shared, tensor memory");

// After a wait that gave up: the copies in flight land before the kernel ends
// (each wait bounded). Stage s has been filled as often as `issued` says.
__device__ __forceinline__ void drain_copies(uint64_t* full, int stages, int64_t issued) {
  for (int64_t i = issued > stages ? issued - stages : 0; i < issued; ++i) {
    const long long t0 = clock64();
    while (!mbar_try_wait(full + i % stages, static_cast<uint32_t>(i / stages) & 1) && clock64() - t0 < kWaitCycles) {
    }
  }
}

// silu(g) * u after the optional clamp, which leaves a NaN one.
__device__ __forceinline__ float swiglu_of(float g, float u, bool clamp, float limit) {
  if (clamp) {
    g = g > limit ? limit : g;
    u = u > limit ? limit : u < -limit ? -limit : u;
  }
  return __fdividef(g, 1.f + __expf(-g)) * u;
}

// 64 columns of a warp's 32 rows, staged in shared memory (16-byte chunk c of row r at
// c ^ (r % 8)), to rows of y that take no tensor map: words of two columns where their
// addresses are even, single columns at the ends.
template <typename T>
__device__ __forceinline__ void store_rows(const uint8_t* stage, T* y, int64_t row0, int rows, int col, int N) {
  const int lane = threadIdx.x & 31, cols = min(64, N - col);
  auto at = [&](int r, int c) {
    return *reinterpret_cast<const uint16_t*>(stage + r * 128 + ((c / 8) ^ (r & 7)) * 16 + c % 8 * 2);
  };
  for (int r = 0; r < rows; ++r) {
    uint16_t* o = reinterpret_cast<uint16_t*>(y) + (row0 + r) * N + col;
    const int odd = (reinterpret_cast<uintptr_t>(o) & 2) != 0;  // then column 0 goes by itself
    const int c = 2 * lane + odd;
    if (c + 1 < cols) *reinterpret_cast<uint32_t*>(o + c) = at(r, c) | static_cast<uint32_t>(at(r, c + 1)) << 16;
    else if (c < cols) o[c] = at(r, c);
    if (odd && lane == 0 && cols > 0) o[0] = at(r, 0);
  }
}

template <typename T>
__global__ void __launch_bounds__(kMmThreads, 1) matmul_fp4_kernel(const __grid_constant__ CUtensorMap ta,
                                                                   const __grid_constant__ CUtensorMap tb,
                                                                   const __grid_constant__ CUtensorMap tsa,
                                                                   const __grid_constant__ CUtensorMap tsb,
                                                                   const __grid_constant__ CUtensorMap ty, MmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  MmSmem& sm = *reinterpret_cast<MmSmem*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank()), pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  volatile int* abort_flag = &sm.abort_flag;
  if (tid == 0) {
    sm.abort_flag = 0;
    for (int s = 0; s < kMmStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.tfull, 1);
    mbar_init(&sm.tempty, 2 * kMmEpiThreads / 32);
    fence_mbar_init();
  }
  if (warp == 1) {
    pair_tmem_alloc(&sm.tmem_base, 512);
    pair_tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // the barriers of both CTAs are set up
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  const int tiles = a.MT * a.NT, KS = (a.KB + 1) / 2;
  pdl_wait();
  pdl_launch_dependents();

  if (warp < kMmEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      if (elect_one()) {
        tma_prefetch_desc(&ta);
        tma_prefetch_desc(&tb);
        tma_prefetch_desc(&tsa);
        tma_prefetch_desc(&tsb);
      }
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int idx = pair; idx < tiles && ok; idx += pairs) {
        const int mt = idx % a.MT * 2 + rank, nt = idx / a.MT;
        for (int ks = 0; ks < KS; ++ks) {
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.empty[stage], phase ^ 1, abort_flag)))) break;
          // boxes that run past K or T read zeros; a half stage's scale words come whole
          if (elect_one()) {
            const uint32_t bar = map_rank(smem_u32(&sm.full[stage]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&sm.full[stage], 2 * kMmStageBytes);
            pair_tma_load_2d(sm.a[stage], &ta, bar, ks * 128, mt * kMmM);
            pair_tma_load_2d(sm.b[stage], &tb, bar, ks * 128, nt * kMmN + rank * (kMmN / 2));
            pair_tma_load_3d(sm.sfa[stage], &tsa, bar, 0, 2 * ks, mt);
            pair_tma_load_3d(sm.sfb[stage], &tsb, bar, 0, 2 * ks, 2 * nt);
          }
          __syncwarp();
          ++issued;
          if (++stage == kMmStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // the last products have arrived on this CTA's barriers before it may end
      for (int s = 0; ok && s < kMmStages; ++s) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.empty[stage], phase ^ 1, abort_flag));
        if (++stage == kMmStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // (the leader's barriers count both CTAs' copies; the other's end with them, before
      // the cluster's last barrier)
      if (!ok && rank == 0 && lane == 0) drain_copies(sm.full, kMmStages, issued);
    } else if (warp == 1 && rank == 0) {
      // What one thread issues a stage must take less time than the products: descriptors
      // are steps from the first stage's, whole stages straight-line code.
      const uint64_t a0 = smem_desc(smem_u32(sm.a[0]), 16, 1024, kSwizzle128B);
      const uint64_t b0 = smem_desc(smem_u32(sm.b[0]), 16, 1024, kSwizzle128B);
      const uint64_t sfa0 = smem_desc(smem_u32(sm.sfa[0]), 0, 128, kSwizzleNone);
      const uint64_t sfb0 = smem_desc(smem_u32(sm.sfb[0]), 0, 128, kSwizzleNone);
      int stage = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      for (int idx = pair; idx < tiles && ok; idx += pairs) {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.tempty, tphase ^ 1, abort_flag)))) break;
        tc_fence_after();
        for (int ks = 0; ks < KS; ++ks) {
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[stage], phase, abort_flag)))) break;
          tc_fence_after();
          const uint32_t sfa = tbase + kMmSfCol + stage * kMmSfCols, sfb = sfa + 8;
          const uint64_t ad = a0 + stage * (kMmM * 128 / 16), bd = b0 + stage * (kMmN / 2 * 128 / 16);
          const uint64_t sad = sfa0 + stage * (1024 / 16), sbd = sfb0 + stage * (2048 / 16);
          auto chunk = [&](int ch, bool add) {  // 128 of K
            pair_tmem_cp_32x128b_warpx4(sfa + 4 * ch, sad + ch * (512 / 16));
            pair_tmem_cp_32x128b_warpx4(sfb + 8 * ch, sbd + ch * (512 / 16));
            pair_tmem_cp_32x128b_warpx4(sfb + 8 * ch + 4, sbd + 1024 / 16 + ch * (512 / 16));
            pair_mma_mxf4(tbase, ad + 4 * ch, bd + 4 * ch, idesc_mxf4(2 * kMmM, kMmN, 0, 0), sfa + 4 * ch, sfb + 8 * ch, add);
            pair_mma_mxf4(tbase, ad + 4 * ch + 2, bd + 4 * ch + 2, idesc_mxf4(2 * kMmM, kMmN, 2, 2), sfa + 4 * ch,
                          sfb + 8 * ch, true);
          };
          if (elect_one()) {
            chunk(0, ks > 0);
            if (2 * ks + 1 < a.KB) chunk(1, true);
            pair_mma_commit(&sm.empty[stage]);
          }
          __syncwarp();
          if (++stage == kMmStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (elect_one()) pair_mma_commit(&sm.tfull);
        __syncwarp();
        tphase ^= 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int wg = (warp - kMmEpiWarp0) / 4;  // column half
    const int quarter = warp & 3;
    const uint32_t src = tbase + (static_cast<uint32_t>(quarter * 32) << 16) + wg * 128;
    const bool clamp = a.limit > 0.f && a.limit < INFINITY;
    uint8_t* stage = sm.out[warp - kMmEpiWarp0];
    uint32_t tphase = 0;
    for (int idx = pair; idx < tiles; idx += pairs) {
      const int mt = idx % a.MT * 2 + rank, nt = idx / a.MT;
      // a warp stops as a whole: one that gives up raises the flag that stops the rest
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.tfull, tphase, abort_flag))) break;
      tphase ^= 1;
      tc_fence_after();
      uint32_t r[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(src + 32 * i, r[i]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(&sm.tempty, 0);
      const int row0 = mt * kMmM + quarter * 32, rows = min(32, a.T - row0);
      // 64 columns at a time: [0, 64) and [64, 128) of the half, or with swiglu its 64 outputs
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (a.swiglu && h == 1) break;
        const int col = a.swiglu ? nt * (kMmN / 2) + wg * 64 : nt * kMmN + wg * 128 + h * 64;
        if (lane == 0) bulk_wait_read();  // the store before has read the staging area
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int i = 8 * c + j;
            if (a.swiglu)
              f[j] = swiglu_of(__uint_as_float(r[i / 32][i % 32]), __uint_as_float(r[2 + i / 32][i % 32]), clamp, a.limit);
            else
              f[j] = __uint_as_float(r[2 * h + i / 32][i % 32]);
          }
          const Pack<T, 8> p = pack<T>(f);
          *reinterpret_cast<Pack<T, 8>*>(stage + lane * 128 + (c ^ (lane & 7)) * 16) = p;
        }
        if (a.packs) fence_proxy_async_smem();
        __syncwarp();
        if (rows > 0 && col < a.N) {
          if (!a.packs) {
            store_rows(stage, static_cast<T*>(a.y), row0, rows, col, a.N);
          } else if (lane == 0) {
            tma_store_2d(&ty, stage, col, row0);
            bulk_commit();
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  cluster_barrier();  // the other CTA's products and arrivals are over
  tc_fence_after();
  if (warp == 1) pair_tmem_dealloc(tbase, 512);
  if (tid == 0 && *abort_flag) atomicOr(a.status, MOE_DEV_TIMEOUT);
}

// ---------------------------------------------------- few tokens: the stream kernel

// For batches whose 128 x 256 tiles would leave most SMs idle the operands change
// places: 128 weight rows are the MMA's M, N <= 128 tokens its N, so that a CTA
// streams weights and the tokens' codes are the small side. K is split over a cluster
// of S CTAs (a rule on the number of tiles, launch below); each leaves its partial
// sums in its shared memory, and after a cluster barrier the CTAs add up the partials
// of their share of the tokens in rank order over distributed shared memory:
// no atomics, the same bits every time. Two CTAs per SM, all stages of weights in flight
// at once, before the quantizing kernel in front has finished where there is one. Bound by the
// weights' bytes: 28671 x 4096 (62 MB) in 13.5 us with one token, 13.8 with 16, 15.8 with 64 and
// 19.3 with 128; small ones by a chain of latencies: 4096 x 7168 with one token 6.2 us, 2880 x 2880
// 4.4 (a call among others, quantization included).
constexpr int kStThreads = 192;
// Up to so many tokens the kernel quantizes the activations itself, every CTA those of its
// part of K: one launch, and no way through memory.
constexpr int kOwnTokens = 8;
// Up to so many tokens this kernel, above it the pairs' tiles. 100 and 256 tokens, 28671 x 4096:
// 18 us and 30.4 here, 31 and 31.3 by tiles; 4096 x 7168: 10.7 and 12.7, 14.5 and 14.8;
// 7168 x 2048: 8.6 and 10.4, 8.9 and 9.0.
constexpr int kStreamTokens = 128;
template <int N>
constexpr int kStStages = N == 16 ? 5 : N <= 64 ? 4 : 3;

template <int N>
struct __align__(1024) StSmem {
  uint8_t a[kStStages<N>][kMmM * 128];  // weights
  uint8_t b[kStStages<N>][N * 128];     // tokens
  uint8_t sfa[kStStages<N>][1024], sfb[kStStages<N>][1024];
  uint64_t full[kStStages<N>], empty[kStStages<N>], tfull;
  uint32_t tmem_base;
  int abort_flag;
  __device__ float* partial() { return reinterpret_cast<float*>(a[0]); }  // [N][128] once the products are done
};
template <int N>
constexpr bool st_layout_ok() {
  // SWIZZLE_128B tiles start at multiples of 1024 bytes; two CTAs share an SM
  return N * 128 % 1024 == 0 && sizeof(StSmem<N>) + 1024 <= 113 * 1024 && offsetof(StSmem<N>, sfa) >= N * 128 * 4 &&
         (N < 32 ? 32 : N) + 16 * kStStages<N> <= 256;
}
static_assert(st_layout_ok<16>() && st_layout_ok<32>() && st_layout_ok<64>() && st_layout_ok<128>(), "shared memory");

// Sums of the partials of all S CTAs, in rank order, for this CTA's share of the tile's
// outputs: four columns of a token a thread, 8 / S of them at once.
template <typename T, int S>
__device__ __forceinline__ void add_partials(uint32_t base, int rank, int thread, const MmArgs& a, T* y, int count,
                                             int tile) {
  constexpr int U = 8 / S;
  const int per = a.swiglu ? 16 : 32, items = count * per;
  const bool clamp = a.limit > 0.f && a.limit < INFINITY;
  uint32_t from[S];
#pragma unroll
  for (int q = 0; q < S; ++q) from[q] = S == 1 ? base : map_rank(base, q);
  auto add = [](float4 u, float4 v) { return make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w); };
  for (int it0 = rank * 128 + thread; it0 < items; it0 += U * S * 128) {
    float4 v[2][U][S];
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      if (part == 1 && !a.swiglu) break;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int it = min(it0 + i * S * 128, items - 1);
        const uint32_t at = 4 * (it / per * 128 + it % per * 4 + part * 64);
#pragma unroll
        for (int q = 0; q < S; ++q) v[part][i][q] = S == 1 ? ld_shared_v4(from[q] + at) : ld_cluster(from[q] + at);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int it = it0 + i * S * 128, row = it % per * 4;
      if (it >= items) break;
      float4 s = v[0][i][0];
#pragma unroll
      for (int q = 1; q < S; ++q) s = add(s, v[0][i][q]);
      if (a.swiglu) {
        float4 u = v[1][i][0];
#pragma unroll
        for (int q = 1; q < S; ++q) u = add(u, v[1][i][q]);
        s = make_float4(swiglu_of(s.x, u.x, clamp, a.limit), swiglu_of(s.y, u.y, clamp, a.limit),
                        swiglu_of(s.z, u.z, clamp, a.limit), swiglu_of(s.w, u.w, clamp, a.limit));
      }
      T* o = y + static_cast<int64_t>(it / per) * a.N + tile + row;
      const float f[4] = {s.x, s.y, s.z, s.w};
      if (a.packs && tile + row + 4 <= a.N) {
        store_pack(o, pack<T>(f));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (tile + row + j < a.N) o[j] = from_f32<T>(f[j]);
      }
    }
  }
}

// Stages of at most 8 tokens' codes and scale words, made by the four warps that
// later store: a unit of 16 elements a thread and stage, the next stage's on its way.
// Rows are 128 bytes in the 128-byte swizzle: 16-byte chunk c of row t sits at c ^ (t % 8).
template <typename T, int kStages, typename Smem>
__device__ __forceinline__ void quantize_stages(Smem& sm, const MmArgs& a, int k0, int n, volatile int* abort_flag) {
  const int lane = threadIdx.x & 31, u = threadIdx.x - 64, t = u / 16, c = u % 16;
  const T* x = static_cast<const T*>(a.x) + t * a.ld + c * kUnit;
  Unit<T> next;
  auto load = [&](int i) {
    const int k = (k0 + i) * 256;
    next = i < n && t < a.T && k + c * kUnit < a.K ? load_unit(x + k, a.how) : zero_unit<T>();
  };
  load(0);
  int stage = 0;
  uint32_t phase = 0;
  for (int i = 0; i < n; ++i) {
    uint32_t sc;
    const uint2 q = quantize_unit(next, &sc);
    load(i + 1);
    uint32_t word = sc << (8 * ((c / 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    if (!__all_sync(0xffffffffu, mbar_wait(&sm.empty[stage], phase ^ 1, abort_flag))) return;
    *reinterpret_cast<uint2*>(sm.b[stage] + t * 128 + (((c / 2) ^ t) * 16) + c % 2 * 8) = q;
    if (c % 8 == 0) *reinterpret_cast<uint32_t*>(sm.sfb[stage] + c / 8 * 512 + t * 16) = word;
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.full[stage]);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
}

// blockIdx.x = (row tile * token tiles + token tile) * S + rank in the cluster
template <typename T, int N, bool OWN>
__global__ void __launch_bounds__(kStThreads) matmul_fp4_stream_kernel(const __grid_constant__ CUtensorMap tw,
                                                                       const __grid_constant__ CUtensorMap tx, MmArgs a,
                                                                       int S) {
  constexpr int kStages = kStStages<N>;
  constexpr uint32_t kSfCol = N < 32 ? 32 : N;
  extern __shared__ uint8_t smem_raw[];
  StSmem<N>& sm = *reinterpret_cast<StSmem<N>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const int rank = blockIdx.x % S, unit = blockIdx.x / S;
  const int tt = unit % a.MT, rt = unit / a.MT;  // MT: token tiles of N
  const int KS = (a.KB + 1) / 2, k0 = rank * KS / S, n = (rank + 1) * KS / S - k0;
  if (tid == 0) {
    sm.abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], OWN ? 5 : 1);  // the producer, the quantizing warps
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.tfull, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  int issued = 0;  // stages that warp 0 has copies for

  if (warp == 0) {
    auto weights = [&](int i, int st) {
      const int ks = k0 + i, nch = min(2, a.KB - 2 * ks);
      mbar_arrive_expect_tx(&sm.full[st], OWN ? kMmM * 128 + nch * 512 : (kMmM + N) * 128 + nch * 1024);
      tma_load_2d(sm.a[st], &tw, &sm.full[st], ks * 128, rt * kMmM);
      bulk_load(sm.sfa[st], a.w_sf + (static_cast<size_t>(rt) * a.KB + 2 * ks) * 512, nch * 512, &sm.full[st]);
    };
    auto tokens = [&](int i, int st) {
      if (OWN) return;
      const int ks = k0 + i, nch = min(2, a.KB - 2 * ks);
      tma_load_2d(sm.b[st], &tx, &sm.full[st], ks * 128, tt * N);
      // a 128-row block of scale words starts at row tt * N only for N = 128: else the tokens are one tile
      bulk_load(sm.sfb[st], a.a_sf + (static_cast<size_t>(tt) * a.KB + 2 * ks) * 512, nch * 512, &sm.full[st]);
    };
    const int pre = min(kStages, n);
    // The first weights are on their way while the quantization ends: that kernel waited for whatever
    // wrote them. With its own quantization the call's kernel in front may be the one that writes them,
    // whose stores are only promised to be seen behind the wait. (Loads in front of it: 4 tokens
    // 4096 x 7168 5.96 us a call, behind it 6.04; in a graph 5.9 and 6.3, 8 tokens 7168 x 2048 4.4 and 4.2.)
    if (!OWN) {
      for (int i = 0; i < pre; ++i)
        if (elect_one()) weights(i, i);
    }
    pdl_wait();
    pdl_launch_dependents();
    if (OWN) {
      for (int i = 0; i < pre; ++i)
        if (elect_one()) weights(i, i);
    }
    // a wait takes a second to give up, so no CTA can have set a flag by now
    if (OWN && tid == 0 && blockIdx.x == 0) *a.status = 0;
    for (int i = 0; i < pre; ++i)
      if (elect_one()) tokens(i, i);
    int stage = pre == kStages ? 0 : pre;
    uint32_t phase = pre == kStages ? 1 : 0;
    issued = pre;
    for (int i = pre; i < n; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.empty[stage], phase ^ 1, abort_flag))) break;
      if (elect_one()) {
        weights(i, stage);
        tokens(i, stage);
      }
      __syncwarp();
      ++issued;
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  } else if (warp == 1) {
    pdl_wait();  // the bounded waits begin when the kernel in front has ended
    const uint64_t a0 = smem_desc(smem_u32(sm.a[0]), 16, 1024, kSwizzle128B);
    const uint64_t b0 = smem_desc(smem_u32(sm.b[0]), 16, 1024, kSwizzle128B);
    const uint64_t sfa0 = smem_desc(smem_u32(sm.sfa[0]), 0, 128, kSwizzleNone);
    const uint64_t sfb0 = smem_desc(smem_u32(sm.sfb[0]), 0, 128, kSwizzleNone);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[stage], phase, abort_flag)))) break;
      tc_fence_after();
      const uint32_t sfa = tbase + kSfCol + stage * 16, sfb = sfa + 8;
      const uint64_t ad = a0 + stage * (kMmM * 128 / 16), bd = b0 + stage * (N * 128 / 16);
      const uint64_t sad = sfa0 + stage * (1024 / 16), sbd = sfb0 + stage * (1024 / 16);
      auto chunk = [&](int ch, bool add) {  // 128 of K
        tmem_cp_32x128b_warpx4(sfa + 4 * ch, sad + ch * (512 / 16));
        tmem_cp_32x128b_warpx4(sfb + 4 * ch, sbd + ch * (512 / 16));
        mma_mxf4(tbase, ad + 4 * ch, bd + 4 * ch, idesc_mxf4(kMmM, N, 0, 0), sfa + 4 * ch, sfb + 4 * ch, add);
        mma_mxf4(tbase, ad + 4 * ch + 2, bd + 4 * ch + 2, idesc_mxf4(kMmM, N, 2, 2), sfa + 4 * ch, sfb + 4 * ch, true);
      };
      if (elect_one()) {
        chunk(0, i > 0);
        if (2 * (k0 + i) + 1 < a.KB) chunk(1, true);
        mma_commit(&sm.empty[stage]);
      }
      __syncwarp();
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (ok && elect_one()) mma_commit(&sm.tfull);
  } else if (warp >= 2) {
    pdl_wait();
    if constexpr (OWN) quantize_stages<T, kStages>(sm, a, k0, n, abort_flag);
    const int quarter = warp & 3, m = quarter * 32 + lane;
    const int count = min(N, a.T - tt * N);  // tokens of the tile
    const bool ok = __all_sync(0xffffffffu, mbar_wait(&sm.tfull, 0, abort_flag));
    tc_fence_after();
    T* y = static_cast<T*>(a.y) + static_cast<int64_t>(tt) * N * a.N;
    const bool plain = S == 1 && !a.swiglu;
    const int64_t col = static_cast<int64_t>(rt) * kMmM + m;
    if (ok) {
#pragma unroll 1
      for (int c = 0; c < count; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tbase + (static_cast<uint32_t>(quarter * 32) << 16) + c, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          if (c + j < count) {
            if (!plain) sm.partial()[(c + j) * 128 + m] = __uint_as_float(r[j]);
            else if (col < a.N) y[static_cast<int64_t>(c + j) * a.N + col] = from_f32<T>(__uint_as_float(r[j]));
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (S > 1) cluster_barrier();
  else __syncthreads();
  // (warp 0 may have issued its last copies before another warp gave up on them)
  if (tid == 0 && *abort_flag) drain_copies(sm.full, kStages, issued);
  if (warp >= 2 && !(S == 1 && !a.swiglu)) {
    const int count = min(N, a.T - tt * N), thread = (warp - 2) * 32 + lane, tile = rt * (a.swiglu ? 64 : kMmM);
    T* y = static_cast<T*>(a.y) + static_cast<int64_t>(tt) * N * a.N;
    const uint32_t base = smem_u32(sm.partial());
    if (S == 1) add_partials<T, 1>(base, rank, thread, a, y, count, tile);
    else if (S == 2) add_partials<T, 2>(base, rank, thread, a, y, count, tile);
    else if (S == 4) add_partials<T, 4>(base, rank, thread, a, y, count, tile);
    else add_partials<T, 8>(base, rank, thread, a, y, count, tile);
  }
  __syncwarp();
  if (S > 1) cluster_barrier();  // nobody leaves while its partials are read
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 256);
  if (tid == 0 && *abort_flag) atomicOr(a.status, MOE_DEV_TIMEOUT);
}

// Weights [N][K / 2] and scales [N][K / 32] to the kernel's rows: padded with
// zeros to tiles of 256 and K blocks of 128; with swiglu in runs of 64 gate, 64 up. K / 2 is
// a multiple of 16: rows are whole 16-byte loads where the codes start at one.
__global__ void __launch_bounds__(128) matmul_prepare_kernel(MatmulShape s, int KB, bool packs,
                                                             const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scale, uint8_t* __restrict__ out,
                                                             uint32_t* __restrict__ sf) {
  const int p = blockIdx.x;  // prepared row
  int src = p;
  if (s.swiglu) {
    const int out_col = p / 256 * 128 + p % 256 / 128 * 64 + p % 64;
    src = out_col < s.N / 2 ? out_col + (p % 128 < 64 ? 0 : s.N / 2) : s.N;
  }
  const bool have = src < s.N;
  const int bytes = s.K / 2;
  const uint8_t* from = codes + static_cast<size_t>(src) * bytes;
  uint8_t* to = out + static_cast<size_t>(p) * KB * 64;
  for (int i = threadIdx.x * 16; i < KB * 64; i += 128 * 16) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (have && i < bytes) {
      if (packs) {
        v = *reinterpret_cast<const uint4*>(from + i);
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j / 4] |= static_cast<uint32_t>(from[i + j]) << (8 * (j % 4));
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    *reinterpret_cast<uint4*>(to + i) = v;
  }
  for (int b = threadIdx.x; b < KB; b += 128) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t v = have && 4 * b + j < s.K / 32 ? scale[static_cast<size_t>(src) * (s.K / 32) + 4 * b + j] : 127;
      w |= v << (8 * j);
    }
    sf[sf_word_index(p, b, KB)] = w;
  }
}

}  // namespace

MatmulLayout matmul_layout(const MatmulShape& s) {
  MatmulLayout l = {};
  if (s.N < 1 || s.N > (1 << 20) || s.K < 32 || s.K > 32768 || s.K % 32 || (s.swiglu && s.N % 2)) return l;
  l.KB = ceil_div(s.K, 128);
  l.NT = s.swiglu ? ceil_div(s.N / 2, kMmN / 2) : ceil_div(s.N, kMmN);
  l.codes_bytes = static_cast<size_t>(l.NT) * kMmN * l.KB * 64;
  l.total = l.codes_bytes + static_cast<size_t>(l.NT) * 2 * l.KB * 512;
  return l;
}

MatmulWorkspace matmul_workspace(int T, int K) {
  MatmulWorkspace w = {};
  const int KB = ceil_div(K, 128);
  w.sf = w.codes = w.total = 256;  // up to kOwnTokens: the status word alone
  if (T <= kOwnTokens) return w;
  w.codes = w.sf + static_cast<size_t>(ceil_div(T, 2 * kMmM)) * 2 * KB * 512;  // whole tiles of a pair
  w.total = w.codes + align_up(static_cast<size_t>(T) * KB * 64, 256);
  return w;
}

cudaError_t launch_matmul_prepare(const MatmulShape& s, const void* codes, const void* scale, void* prepared,
                                  cudaStream_t st) {
  const MatmulLayout l = matmul_layout(s);
  uint8_t* p = static_cast<uint8_t*>(prepared);
  return launch_kernel(false, matmul_prepare_kernel, l.NT * kMmN, 128, 0, st, s, l.KB, aligned16(codes),
                       static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scale), p,
                       reinterpret_cast<uint32_t*>(p + l.codes_bytes));
}

namespace {

// A launch in clusters of `cluster` CTAs that may begin while the kernel in front ends.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int grid, int threads, int cluster, size_t smem, cudaStream_t st,
                           const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int N, bool OWN, typename F>
cudaError_t launch_stream(const MatmulLayout& l, const uint8_t* prepared, const uint8_t* codes, MmArgs a, int num_sms,
                          cudaStream_t st, F&& quantize) {
  CUtensorMap tw, tx = {};
  const uint64_t row = static_cast<uint64_t>(l.KB) * 64;
  if (!byte_tmap(&tw, prepared, row, static_cast<uint64_t>(l.NT) * kMmN, kMmM) ||
      (!OWN && !byte_tmap(&tx, codes, row, a.T, N)))
    return cudaErrorInvalidValue;
  a.MT = ceil_div(a.T, N);
  // K is split while the CTAs are at most one per SM (two for the fewest tokens, whose
  // partials are cheap to add up) and have two stages each. 4096 x 7168, 128 tokens:
  // 128 CTAs 10.7 us, 256 12.8; 16 tokens 7.7 and 8.2; one token 7.8 and 6.2.
  const int units = 2 * l.NT * a.MT, KS = (l.KB + 1) / 2;
  int S = 1;
  while (S < 8 && units * S * 2 <= (OWN ? 2 : 1) * num_sms && KS >= 4 * S) S *= 2;
  auto* kernel = matmul_fp4_stream_kernel<T, N, OWN>;
  const size_t smem = sizeof(StSmem<N>) + 1024;
  cudaError_t e = allow_smem(kernel, smem);
  if (e == cudaSuccess && !OWN) e = quantize();
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, units * S, kStThreads, S, smem, st, tw, tx, a, S);
}

template <typename T, typename F>
cudaError_t launch_stream(const MatmulLayout& l, const uint8_t* prepared, const uint8_t* codes, const MmArgs& a,
                          int num_sms, cudaStream_t st, F&& quantize) {
  return a.T <= kOwnTokens ? launch_stream<T, 16, true>(l, prepared, codes, a, num_sms, st, quantize)
         : a.T <= 16 ? launch_stream<T, 16, false>(l, prepared, codes, a, num_sms, st, quantize)
         : a.T <= 32 ? launch_stream<T, 32, false>(l, prepared, codes, a, num_sms, st, quantize)
         : a.T <= 64 ? launch_stream<T, 64, false>(l, prepared, codes, a, num_sms, st, quantize)
                     : launch_stream<T, 128, false>(l, prepared, codes, a, num_sms, st, quantize);
}

}  // namespace

cudaError_t launch_matmul_fp4(const MatmulShape& s, float limit, const void* prepared, int dtype, const void* x,
                              int64_t ld, int T, void* y, uint8_t* ws, int num_sms, cudaStream_t st) {
  const MatmulLayout l = matmul_layout(s);
  const MatmulWorkspace w = matmul_workspace(T, s.K);
  const uint8_t* p = static_cast<const uint8_t*>(prepared);
  MmArgs a = {ws + w.sf, p + l.codes_bytes, reinterpret_cast<uint32_t*>(ws), y, T, s.swiglu ? s.N / 2 : s.N,
              l.KB, ceil_div(T, kMmM), l.NT, s.swiglu, limit, false, x, ld, s.K, how_aligned(x, ld, 2)};
  a.packs = aligned16(y) && a.N % 8 == 0;
  // enqueued when nothing is left that could refuse the product
  auto quantize = [&] {
    return launch_quantize_act(dtype, x, ld, T, s.K, ws + w.codes, reinterpret_cast<uint32_t*>(ws + w.sf), a.status, st);
  };
  if (T <= kStreamTokens)
    return dtype == MOE_BF16 ? launch_stream<__nv_bfloat16>(l, p, ws + w.codes, a, num_sms, st, quantize)
                             : launch_stream<__half>(l, p, ws + w.codes, a, num_sms, st, quantize);
  a.MT = ceil_div(T, 2 * kMmM);
  CUtensorMap ta, tb, tsa, tsb, ty = {};
  if (!byte_tmap(&ta, ws + w.codes, static_cast<uint64_t>(l.KB) * 64, T, kMmM) ||
      !byte_tmap(&tb, p, static_cast<uint64_t>(l.KB) * 64, static_cast<uint64_t>(l.NT) * kMmN, kMmN / 2) ||
      !scale_tmap(&tsa, ws + w.sf, l.KB, 2 * a.MT, 1) || !scale_tmap(&tsb, p + l.codes_bytes, l.KB, 2 * l.NT, 2) ||
      (a.packs && !store_tmap(&ty, y, a.N, T, 64, 32)))
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(MmSmem) + 1024;
  const int pairs = num_sms / 2, tiles = a.MT * a.NT;
  auto run = [&](auto* kernel) {
    cudaError_t e = allow_smem(kernel, smem);
    if (e == cudaSuccess) e = quantize();
    if (e != cudaSuccess) return e;
    return launch_cluster(kernel, 2 * (tiles < pairs ? tiles : pairs), kMmThreads, 2, smem, st, ta, tb, tsa, tsb, ty, a);
  };
  return dtype == MOE_BF16 ? run(matmul_fp4_kernel<__nv_bfloat16>) : run(matmul_fp4_kernel<__half>);
}

}  // namespace bsmoe
