// Products of many tokens with FP4 weights on the tensor cores: both operands e2m1
// in 1x32 blocks (tcgen05.mma kind::mxf4), the activations quantized by the kernel
// in front (launch_quantize_act).
//
//   y[t, n] = sum_k dq(x)[t, k] * dq(W)[n, k], fp32 accumulators, one rounding;
//   with swiglu, tile columns alternate 64 gate and 64 up rows of W and the
//   epilogue stores silu(gate) * up.
//
// One persistent CTA per SM: warp 0 keeps four stages of K = 256 in flight (TMA
// tiles of 128 activation rows and 256 weight rows, bulk copies of their scale
// words), warp 1 issues the MMAs, warps 4..11 move the accumulators to registers,
// hand tensor memory back and store while the next tile is multiplied.
#include <cuda.h>

#include "../act_quant.cuh"
#include "../ptx.cuh"
#include "block_internal.cuh"

namespace bsmoe {

namespace {

constexpr int kMmThreads = 384;
constexpr int kMmEpiWarp0 = 4, kMmEpiThreads = 256;
constexpr int kMmStages = 4;
constexpr int kMmM = 128, kMmN = 256;
constexpr uint32_t kMmSfCol = 256, kMmSfCols = 24;  // per stage 8 columns of A's and 16 of B's scales

struct MmArgs {
  const uint8_t *a_sf, *w_sf;
  uint32_t* status;
  void* y;
  int T, N;  // N: columns of y
  int KB, MT, NT, swiglu;
  float limit;
  bool packs;  // rows of y take 16-byte stores
};

struct __align__(1024) MmSmem {
  uint8_t b[kMmStages][kMmN * 128];
  uint8_t a[kMmStages][kMmM * 128];
  uint8_t sfa[kMmStages][1024];
  uint8_t sfb[kMmStages][2048];  // [128-row half][128-K chunk][512]
  uint64_t full[kMmStages], empty[kMmStages], tfull, tempty;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(MmSmem) + 1024 <= 227 * 1024, "shared memory");

template <typename T>
__device__ __forceinline__ void store_columns(T* row, int col, int limit_col, bool packs, const float (&v)[32]) {
  constexpr int W = kVec<T>;
  if (packs && col + 32 <= limit_col) {
#pragma unroll
    for (int i = 0; i < 32; i += W) {
      float f[W];
#pragma unroll
      for (int j = 0; j < W; ++j) f[j] = v[i + j];
      store_pack(row + col + i, pack<T>(f));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (col + i < limit_col) row[col + i] = from_f32<T>(v[i]);
  }
}

// After a wait that gave up: the copies in flight land before the kernel ends
// (each wait bounded). Stage s has been filled as often as `issued` says.
__device__ __forceinline__ void drain_copies(uint64_t* full, int stages, int64_t issued) {
  for (int64_t i = issued > stages ? issued - stages : 0; i < issued; ++i) {
    const long long t0 = clock64();
    while (!mbar_try_wait(full + i % stages, static_cast<uint32_t>(i / stages) & 1) && clock64() - t0 < kWaitCycles) {
    }
  }
}

// silu(g) * u after the optional clamp.
__device__ __forceinline__ float swiglu_of(float g, float u, bool clamp, float limit) {
  if (clamp) {
    g = fminf(g, limit);
    u = fminf(fmaxf(u, -limit), limit);
  }
  return __fdividef(g, 1.f + __expf(-g)) * u;
}

template <typename T>
__global__ void __launch_bounds__(kMmThreads, 1) matmul_fp4_kernel(const __grid_constant__ CUtensorMap ta,
                                                                   const __grid_constant__ CUtensorMap tb, MmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  MmSmem& sm = *reinterpret_cast<MmSmem*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sm.abort_flag;
  if (tid == 0) {
    sm.abort_flag = 0;
    for (int s = 0; s < kMmStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.tfull, 1);
    mbar_init(&sm.tempty, kMmEpiThreads / 32);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  const int tiles = a.MT * a.NT, KS = (a.KB + 1) / 2;
  pdl_wait();
  pdl_launch_dependents();

  if (warp < kMmEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      tma_prefetch_desc(&ta);
      tma_prefetch_desc(&tb);
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int idx = blockIdx.x; idx < tiles && ok; idx += gridDim.x) {
        const int mt = idx % a.MT, nt = idx / a.MT;
        for (int ks = 0; ks < KS; ++ks) {
          if (!(ok = mbar_wait(&sm.empty[stage], phase ^ 1, abort_flag))) break;
          const int nch = min(2, a.KB - 2 * ks);
          mbar_arrive_expect_tx(&sm.full[stage], (kMmM + kMmN) * 128 + nch * 1536);
          // boxes that run past K read zeros
          tma_load_2d(sm.a[stage], &ta, &sm.full[stage], ks * 128, mt * kMmM);
          tma_load_2d(sm.b[stage], &tb, &sm.full[stage], ks * 128, nt * kMmN);
          bulk_load(sm.sfa[stage], a.a_sf + (static_cast<size_t>(mt) * a.KB + 2 * ks) * 512, nch * 512, &sm.full[stage]);
          for (int h = 0; h < 2; ++h)
            bulk_load(sm.sfb[stage] + h * 1024, a.w_sf + (static_cast<size_t>(2 * nt + h) * a.KB + 2 * ks) * 512,
                      nch * 512, &sm.full[stage]);
          ++issued;
          if (++stage == kMmStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) drain_copies(sm.full, kMmStages, issued);
    } else if (warp == 1 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      for (int idx = blockIdx.x; idx < tiles && ok; idx += gridDim.x) {
        if (!(ok = mbar_wait(&sm.tempty, tphase ^ 1, abort_flag))) break;
        tc_fence_after();
        for (int ks = 0; ks < KS; ++ks) {
          if (!(ok = mbar_wait(&sm.full[stage], phase, abort_flag))) break;
          tc_fence_after();
          const int nch = min(2, a.KB - 2 * ks);
          const uint32_t sfa = tbase + kMmSfCol + stage * kMmSfCols, sfb = sfa + 8;
          for (int ch = 0; ch < nch; ++ch) {
            tmem_cp_32x128b_warpx4(sfa + 4 * ch, smem_desc(smem_u32(sm.sfa[stage] + ch * 512), 0, 128, kSwizzleNone));
            for (int h = 0; h < 2; ++h)
              tmem_cp_32x128b_warpx4(sfb + 8 * ch + 4 * h,
                                     smem_desc(smem_u32(sm.sfb[stage] + h * 1024 + ch * 512), 0, 128, kSwizzleNone));
          }
          const uint64_t ad = smem_desc(smem_u32(sm.a[stage]), 16, 1024, kSwizzle128B);
          const uint64_t bd = smem_desc(smem_u32(sm.b[stage]), 16, 1024, kSwizzle128B);
          for (int j = 0; j < 2 * nch; ++j)
            mma_mxf4(tbase, ad + 2 * j, bd + 2 * j, idesc_mxf4(kMmM, kMmN, 2 * (j & 1), 2 * (j & 1)), sfa + 4 * (j >> 1),
                     sfb + 8 * (j >> 1), (ks > 0 || j > 0) ? 1u : 0u);
          mma_commit(&sm.empty[stage]);
          if (++stage == kMmStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        mma_commit(&sm.tfull);
        tphase ^= 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int wg = (warp - kMmEpiWarp0) / 4;  // column half
    const int quarter = warp & 3;
    const uint32_t src = tbase + (static_cast<uint32_t>(quarter * 32) << 16) + wg * 128;
    const bool clamp = a.limit > 0.f && a.limit < INFINITY;
    uint32_t tphase = 0;
    for (int idx = blockIdx.x; idx < tiles; idx += gridDim.x) {
      const int mt = idx % a.MT, nt = idx / a.MT;
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
      if (lane == 0) mbar_arrive(&sm.tempty);
      const int t = mt * kMmM + quarter * 32 + lane;
      if (t < a.T) {
        T* row = static_cast<T*>(a.y) + static_cast<int64_t>(t) * a.N;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[32];
          if (!a.swiglu) {
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(r[i][j]);
            store_columns(row, nt * kMmN + wg * 128 + 32 * i, a.N, a.packs, f);
          } else if (i < 2) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              f[j] = swiglu_of(__uint_as_float(r[i][j]), __uint_as_float(r[(i + 2) % 4][j]), clamp, a.limit);
            store_columns(row, nt * (kMmN / 2) + wg * 64 + 32 * i, a.N, a.packs, f);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
  if (tid == 0 && *abort_flag) atomicOr(a.status, MOE_DEV_TIMEOUT);
}

// Weights [N][K / 2] and scales [N][K / 32] to the kernel's rows: padded with
// zeros to tiles of 256 and K blocks of 128; with swiglu in runs of 64 gate, 64 up.
__global__ void __launch_bounds__(256) matmul_prepare_kernel(MatmulShape s, int KB, const uint8_t* __restrict__ codes,
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
  for (int i = threadIdx.x * 4; i < KB * 64; i += 256 * 4) {
    uint32_t w = 0;
    if (have && i < bytes) {  // K / 2 is a multiple of 16
#pragma unroll
      for (int j = 0; j < 4; ++j) w |= static_cast<uint32_t>(codes[static_cast<size_t>(src) * bytes + i + j]) << (8 * j);
    }
    *reinterpret_cast<uint32_t*>(out + static_cast<size_t>(p) * KB * 64 + i) = w;
  }
  for (int b = threadIdx.x; b < KB; b += 256) {
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
  w.sf = 256;
  w.codes = w.sf + static_cast<size_t>(ceil_div(T, 128)) * KB * 512;
  w.total = w.codes + align_up(static_cast<size_t>(T) * KB * 64, 256);
  return w;
}

cudaError_t launch_matmul_prepare(const MatmulShape& s, const void* codes, const void* scale, void* prepared,
                                  cudaStream_t st) {
  const MatmulLayout l = matmul_layout(s);
  uint8_t* p = static_cast<uint8_t*>(prepared);
  return launch_kernel(false, matmul_prepare_kernel, l.NT * kMmN, 256, 0, st, s, l.KB,
                       static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scale), p,
                       reinterpret_cast<uint32_t*>(p + l.codes_bytes));
}

cudaError_t launch_matmul_fp4(const MatmulShape& s, float limit, const void* prepared, int dtype, int T, void* y,
                              uint8_t* ws, int num_sms, cudaStream_t st) {
  const MatmulLayout l = matmul_layout(s);
  const MatmulWorkspace w = matmul_workspace(T, s.K);
  const uint8_t* p = static_cast<const uint8_t*>(prepared);
  CUtensorMap ta, tb;
  if (!byte_tmap(&ta, ws + w.codes, static_cast<uint64_t>(l.KB) * 64, T, kMmM) ||
      !byte_tmap(&tb, p, static_cast<uint64_t>(l.KB) * 64, static_cast<uint64_t>(l.NT) * kMmN, kMmN))
    return cudaErrorInvalidValue;
  MmArgs a = {ws + w.sf, p + l.codes_bytes, reinterpret_cast<uint32_t*>(ws), y, T, s.swiglu ? s.N / 2 : s.N,
              l.KB, ceil_div(T, kMmM), l.NT, s.swiglu, limit, false};
  a.packs = aligned16(y) && a.N % 8 == 0;
  const size_t smem = sizeof(MmSmem) + 1024;
  const int grid = a.MT * a.NT < num_sms ? a.MT * a.NT : num_sms;
  auto run = [&](auto* kernel) {
    const cudaError_t e = allow_smem(kernel, smem);
    return e != cudaSuccess ? e : launch_kernel(true, kernel, grid, kMmThreads, smem, st, ta, tb, a);
  };
  return dtype == MOE_BF16 ? run(matmul_fp4_kernel<__nv_bfloat16>) : run(matmul_fp4_kernel<__half>);
}

}  // namespace bsmoe
