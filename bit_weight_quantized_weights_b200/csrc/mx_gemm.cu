// MXFP4 activations and their product with MXFP4 weights on the block-scaled
// FP4 tensor cores (any number of tokens).
//
// Source: "Multi-Scale Dequant: Eliminating Dequantization Bottleneck via
// Activation Decomposition for Efficient LLM Inference", Abstract: for MXFP4
// weights, two MXFP4 passes over the bf16 activations multiply the weights
// directly. Here the passes ("planes") are kept in 4 bits:
//   plane 1: blocks of 32 along K share 2^e, e the smallest with amax <= 6 2^e
//            (0 for a block of zeros, clamped to -127 .. 127); elements E2M1,
//            round to nearest, ties to the even code;
//   plane 2: the same of the residual x - x1, which is exact in fp32;
//   y[m, n] = sum_p sum_blk 2^(e_p + e_w) sum_{k in blk} x_p[m, k] w[n, k].
// One plane is the plain MXFP4 product.
#include <algorithm>

#include "sm100.cuh"

namespace wq {

__device__ unsigned int g_mx_gemm_error;

namespace {

// ---------------------------------------------------------------------------
// Quantization of activations: one warp takes 256 consecutive elements of a
// row, 8 elements a lane, so a block of 32 is 4 lanes (two shuffles for its
// largest magnitude) and a lane's codes are one 32-bit store.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float pow2f(int e) {  // exact for e in [-127, 127]
  return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(0x00400000u);
}

// Smallest e in [-127, 127] with a <= 1.5 * 2^(e + 2); 0 for a = 0. From the
// bits of a: exponent field F, and one more if the mantissa is above 1.5
// (a subnormal a gives the clamp's -127 as well).
__device__ __forceinline__ int e2m1_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  if (u == 0) return 0;
  const int e = (int)(u >> 23) - 127 - 2 + ((u & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return max(e, -127);
}

// Eight E2M1 codes of f[i] * scale, element i in nibble i; zeros are +0.
__device__ __forceinline__ uint32_t e2m1_x8(const float (&f)[8], float scale) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t b;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u16.u8 %0, t;\n\t}"
        : "=h"(b)
        : "f"(f[2 * i + 1] * scale), "f"(f[2 * i] * scale));
    w |= (uint32_t)b << (8 * i);
  }
  const uint32_t some = (w | (w >> 1) | (w >> 2)) & 0x11111111u;  // magnitude above 0
  return w & (0x77777777u | (some << 3));
}

// The value of one code: E2M1 magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t mag = c & 7u;
  // codes 2..7 are 2^((c >> 1) - 1) (1 + (c & 1) / 2); 0 and 1 are 0 and 1/2
  const uint32_t norm = (((mag >> 1) + 126u) << 23) | ((mag & 1u) << 22);
  const uint32_t bits = mag < 2 ? (mag ? 0x3F000000u : 0u) : norm;
  return __uint_as_float(bits | ((c & 8u) << 28));
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 v = ld_stream_u4(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo_to_f32(w[i]);
    f[2 * i + 1] = bf16_hi_to_f32(w[i]);
  }
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float (&f)[8]) {
  const uint4 v = ld_stream_u4(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
  const uint4 a = ld_stream_u4(p), b = ld_stream_u4(p + 4);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}

template <typename T, int PL>
__global__ void __launch_bounds__(256)
    mx_planes_kernel(const T* __restrict__ x, int64_t ldx, int M, int K,
                     uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int chunks = (K + 255) / 256;
  const int64_t total = (int64_t)M * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total;
       i += (int64_t)gridDim.x * 8) {
    const int m = (int)(i / chunks);
    const int k = (int)(i - (int64_t)m * chunks) * 256 + 8 * lane;
    const bool in = k < K;  // whole blocks: K is a multiple of 32
    float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (in) load8(x + (int64_t)m * ldx + k, f);
#pragma unroll
    for (int p = 0; p < PL; ++p) {
      float a = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(f[j]));
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
      const int e = e2m1_exponent(a);
      const uint32_t w = e2m1_x8(f, pow2f(-e));
      if (in) {
        const int64_t row = (int64_t)p * M + m;
        *reinterpret_cast<uint32_t*>(codes + (row * K + k) / 2) = w;
        if ((lane & 3) == 0) scales[(row * K + k) / 32] = (uint8_t)(e + 127);
      }
      if (p + 1 < PL) {
        const float up = pow2f(e);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = fmaf(-e2m1_value(w >> (4 * j)), up, f[j]);  // exact
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Product. A tile is 128 tokens (the MMA's M) by BN features (its N), summed
// over all planes in one TMEM accumulator: a weight tile is loaded once and
// multiplied with every plane's token tile. A stage holds 256 k (128-byte rows
// of 4-bit codes, 128-byte swizzle) of all operands and their scale bytes,
// which a warpgroup places in the order that tcgen05.cp copies to TMEM: 4 scale
// bytes (128 k) of row r at byte (r % 32) * 16 + (r / 32) * 4 of a 512-byte
// piece, one piece for 128 rows.
//   warp 0       TMA loads of the codes
//   warp 1       tcgen05.cp of the scales, tcgen05.mma (one thread)
//   warps 4-7    scale bytes into shared memory (4-byte cp.async)
//   warps 8-15   epilogue: TMEM to registers as packed bf16, which frees the
//                accumulator for the next tile, then the stores
// CTAs are persistent and take every gridDim.x-th tile.
// ---------------------------------------------------------------------------
constexpr int kBM = 128;
constexpr int kBKBytes = 128;   // bytes of a stage's row: 256 k
constexpr int kThreads = 512;

template <int BN, int PL>
struct MxCfg {
  static constexpr int kXBytes = PL * kBM * kBKBytes;
  static constexpr int kWBytes = BN * kBKBytes;
  static constexpr int kWPieces = (BN + 127) / 128;           // 128-row scale pieces
  static constexpr int kSfBytes = (PL + kWPieces) * 2 * 512;  // two pieces a row block: 256 k
  static constexpr int kStageBytes = kXBytes + kWBytes + kSfBytes;
  static constexpr int kStages = 212992 / kStageBytes < 8 ? 212992 / kStageBytes : 8;
  static constexpr int kSmem = kStages * kStageBytes + 1024 + 256;
  // TMEM columns: the accumulator, then two sets of scales (4 columns a piece)
  static constexpr int kSfCols = (PL + kWPieces) * 2 * 4;
  static constexpr int kCols = BN + 2 * kSfCols;
  static constexpr int kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
};

// kind::mxf4: E2M1 x E2M1 with UE8M0 scales of blocks of 32, fp32 sums.
//   bits 4-5 B scale id, 7-9 A type (1 = E2M1), 10-11 B type, 17-22 N / 8,
//   23 scale type (1 = UE8M0), 27-28 M / 128, 29-30 A scale id
__host__ __device__ constexpr uint32_t idesc_mxf4(int n, int sf_id) {
  return ((uint32_t)sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
         (1u << 23) | (1u << 27) | ((uint32_t)sf_id << 29);
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// A 512-byte scale piece (32 rows of 16 bytes, no swizzle: groups of 8 rows
// 128 bytes apart) to 4 TMEM columns, the same in all four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t smem) {
  const uint64_t desc = (uint64_t)((smem & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) |
                        ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1 << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
               : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool in) {
  // a size of 0 writes zeros: the scale 2^-127 of an operand that is zero
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 4 : 0)
               : "memory");
}

struct MxArgs {
  const uint8_t* xs;  // [PL][M][K / 32]
  const uint8_t* ws;  // [N][K / 32]
  uint16_t* y;
  int M, N, K;
  int mt, tiles;      // token tiles; all tiles
};

template <int BN, int PL>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x,
                   const __grid_constant__ CUtensorMap tmap_w, const MxArgs a, const WaitCtl wc) {
  using Cfg = MxCfg<BN, PL>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint8_t* sx = smem;                       // [stage][plane][128 rows]
  uint8_t* sw = sx + S * Cfg::kXBytes;      // [stage][BN rows]
  uint8_t* ssf = sw + S * Cfg::kWBytes;     // [stage][plane or weight piece][2][512]
  uint64_t* full = reinterpret_cast<uint64_t*>(ssf + S * Cfg::kSfBytes);
  uint64_t* sffull = full + S;
  uint64_t* empty = sffull + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* mma_done = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KT = (a.K / 2 + kBKBytes - 1) / kBKBytes;

  if (threadIdx.x == 0) {
    sm100::tma_prefetch_desc(&tmap_x);
    sm100::tma_prefetch_desc(&tmap_w);
    for (int s = 0; s < S; ++s) {
      sm100::mbar_init(&full[s], 1);
      sm100::mbar_init(&sffull[s], 128);
      sm100::mbar_init(&empty[s], 1);
    }
    sm100::mbar_init(acc_full, 1);
    sm100::mbar_init(acc_empty, 8);
    sm100::mbar_init(mma_done, 1);
    *abort_flag = 0;
    sm100::fence_mbar_init();
  }
  if (warp == 1) {
    sm100::tmem_alloc(tmem_slot, Cfg::kTmemCols);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_sf = tmem + BN;

  int last_issued = -1;
  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
        const int m0 = (t % a.mt) * kBM, n0 = (t / a.mt) * BN;
        for (int kt = 0; kt < KT; ++kt, ++it) {
          const int s = it % S;
          if (it >= S && !sm100::mbar_wait(&empty[s], (uint32_t)(it / S - 1) & 1u,
                                           &g_mx_gemm_error, 0x3101u, abort_flag, wc.limit_ns)) {
            ok = false;
            break;
          }
          if (wc.stall && it == 0) continue;  // test hook: the first k-tile never arrives
          last_issued = it;
          sm100::mbar_arrive_expect_tx(&full[s], Cfg::kXBytes + Cfg::kWBytes);
#pragma unroll
          for (int p = 0; p < PL; ++p)
            sm100::tma_load_2d(sx + s * Cfg::kXBytes + p * kBM * kBKBytes, &tmap_x, &full[s],
                               kt * kBKBytes, p * a.M + m0);
          sm100::tma_load_2d(sw + s * Cfg::kWBytes, &tmap_w, &full[s], kt * kBKBytes, n0);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0, n = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x, ++n) {
        if (n > 0) {
          if (!sm100::mbar_wait(acc_empty, (uint32_t)(n - 1) & 1u, &g_mx_gemm_error, 0x3201u,
                                abort_flag, wc.limit_ns)) {
            ok = false;
            break;
          }
          sm100::tc_fence_after();
        }
        for (int kt = 0; kt < KT; ++kt, ++it) {
          const int s = it % S;
          const uint32_t ph = (uint32_t)(it / S) & 1u;
          if (!sm100::mbar_wait(&full[s], ph, &g_mx_gemm_error, 0x3202u, abort_flag,
                                wc.limit_ns) ||
              !sm100::mbar_wait(&sffull[s], ph, &g_mx_gemm_error, 0x3203u, abort_flag,
                                wc.limit_ns)) {
            ok = false;
            break;
          }
          sm100::tc_fence_after();
          // scales of the stage: two sets of TMEM columns in turn, so that a
          // copy never meets the MMAs of the stage before
          const uint32_t sf = tmem_sf + (uint32_t)(it & 1) * Cfg::kSfCols;
          const uint32_t sf_smem = smem_u32(ssf + s * Cfg::kSfBytes);
#pragma unroll
          for (int i = 0; i < PL + Cfg::kWPieces; ++i)
#pragma unroll
            for (int kg = 0; kg < 2; ++kg) {
              // weights: the two pieces of 128 rows of one kg side by side
              const uint32_t col =
                  i < PL ? (i * 2 + kg) * 4
                         : PL * 8 + kg * 4 * Cfg::kWPieces + (i - PL) * 4;
              copy_scales(sf + col, sf_smem + (uint32_t)(i * 2 + kg) * 512);
            }
          const uint32_t xb = smem_u32(sx + s * Cfg::kXBytes);
          const uint32_t wb = smem_u32(sw + s * Cfg::kWBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // 64 k each: 32 bytes, 2 scale bytes
            const int kg = kk >> 1;
            const uint32_t idesc =
                (kk & 1) ? idesc_mxf4(BN, 2) : idesc_mxf4(BN, 0);
            const uint64_t bdesc = sm100::sdesc_sw128_kmajor(wb + kk * 32);
            const uint32_t sfb = sf + PL * 8 + kg * 4 * Cfg::kWPieces;
#pragma unroll
            for (int p = 0; p < PL; ++p)
              mma_mxf4(tmem, sm100::sdesc_sw128_kmajor(xb + p * kBM * kBKBytes + kk * 32), bdesc,
                       idesc, sf + (p * 2 + kg) * 4, sfb, (kt | kk | p) != 0 ? 1u : 0u);
          }
          sm100::mma_commit(&empty[s]);
        }
        if (ok) sm100::mma_commit(acc_full);
      }
      sm100::mma_commit(mma_done);
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------- scale bytes: thread = row of a 128-row block ----------------
    const int r = threadIdx.x - 128;
    const int K32 = a.K / 32;
    const uint32_t dst0 = smem_u32(ssf) + (uint32_t)((r & 31) * 16 + (r >> 5) * 4);
    int it = 0;
    bool ok = true;
    auto publish = [&](int i) {  // the writes of stage i are complete
      sm100::fence_proxy_async_smem();
      sm100::mbar_arrive(&sffull[i % S]);
    };
    for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
      const int m0 = (t % a.mt) * kBM, n0 = (t / a.mt) * BN;
      for (int kt = 0; kt < KT; ++kt, ++it) {
        const int s = it % S;
        if (it >= S && !sm100::mbar_wait(&empty[s], (uint32_t)(it / S - 1) & 1u, &g_mx_gemm_error,
                                         0x3301u, abort_flag, wc.limit_ns)) {
          ok = false;
          break;
        }
        const uint32_t dst = dst0 + (uint32_t)s * Cfg::kSfBytes;
#pragma unroll
        for (int i = 0; i < PL + Cfg::kWPieces; ++i) {
          bool in = i < PL ? m0 + r < a.M : n0 + (i - PL) * 128 + r < a.N;
          if (BN < 128 && i >= PL) in = in && r < BN;
          const int64_t row = !in ? 0
                              : i < PL ? (int64_t)i * a.M + m0 + r
                                       : (int64_t)n0 + (i - PL) * 128 + r;
          const uint8_t* src = (i < PL ? a.xs : a.ws) + row * K32 + kt * 8;
#pragma unroll
          for (int kg = 0; kg < 2; ++kg) {
            const bool have = in && kt * 8 + kg * 4 < K32;
            cp_async4(dst + (uint32_t)(i * 2 + kg) * 512, have ? src + kg * 4 : a.ws, have);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (it > 0) {
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          publish(it - 1);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (ok && it > 0) publish(it - 1);
  } else if (warp >= 8) {
    // ---------------- epilogue: thread = token, half of the tile's features ----------------
    const int q = warp & 3, part = (warp - 8) >> 2;
    constexpr int kCols = BN / 2;
    int n = 0;
    for (int t = blockIdx.x; t < a.tiles; t += gridDim.x, ++n) {
      const int m = (t % a.mt) * kBM + 32 * q + lane;
      const int col0 = (t / a.mt) * BN + part * kCols;
      const bool got = sm100::mbar_wait(acc_full, (uint32_t)n & 1u, &g_mx_gemm_error, 0x3401u,
                                        abort_flag, wc.limit_ns);
      if (!__all_sync(0xffffffffu, got)) break;
      sm100::tc_fence_after();
      uint32_t out[kCols / 2];
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c) {
        uint32_t v[32];
        sm100::tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + part * kCols + 32 * c, v);
        sm100::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          out[16 * c + j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
      }
      sm100::tc_fence_before();
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(acc_empty);
      if (m < a.M) {
        uint16_t* dst = a.y + (int64_t)m * a.N + col0;
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i)
          if (col0 + 8 * i < a.N)
            *reinterpret_cast<uint4*>(dst + 8 * i) =
                make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
      }
    }
  }

  // After an abort: wait (bounded) for the loads and MMAs still in flight.
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) {
      for (int i = max(0, last_issued - S + 1); i <= last_issued; ++i)
        if (!(wc.stall && i == 0))
          sm100::mbar_wait_drain(&full[i % S], (uint32_t)(i / S) & 1u, wc.limit_ns);
      sm100::mbar_wait_drain(mma_done, 0, wc.limit_ns);
    }
    __syncthreads();
  }
  sm100::tc_fence_after();
  if (warp == 1) sm100::tmem_dealloc(tmem, Cfg::kTmemCols);
}

template <int BN, int PL>
wq_status launch_gemm_t(const CUtensorMap& tx, const void* wcodes, const MxArgs& a0,
                        cudaStream_t st) {
  using Cfg = MxCfg<BN, PL>;
  CUtensorMap tw;
  if (!make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, wcodes, (uint64_t)a0.K / 2,
                    (uint64_t)a0.N, (uint64_t)a0.K / 2, kBKBytes, BN, CU_TENSOR_MAP_SWIZZLE_128B))
    return WQ_ERR_CUDA;
  static bool attr_set = [] {
    return cudaFuncSetAttribute(mx_gemm_kernel<BN, PL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg::kSmem) == cudaSuccess;
  }();
  if (!attr_set) return WQ_ERR_CUDA;
  MxArgs a = a0;
  a.mt = (a.M + kBM - 1) / kBM;
  a.tiles = a.mt * ((a.N + BN - 1) / BN);
  mx_gemm_kernel<BN, PL><<<std::min(a.tiles, num_sms()), kThreads, Cfg::kSmem, st>>>(tx, tw, a,
                                                                                    wait_ctl());
  return launch_status();
}

template <int PL>
wq_status launch_gemm(const CUtensorMap& tx, const void* wcodes, const MxArgs& a,
                      cudaStream_t st) {
  // the tile width with the least time for the slowest CTA: whole tiles an SM
  // takes, times a tile's cost
  const int64_t mt = (a.M + kBM - 1) / kBM, sms = num_sms();
  auto cost = [&](int bn, int64_t tile) {
    const int64_t tiles = mt * ((a.N + bn - 1) / bn);
    return (tiles + sms - 1) / sms * tile;
  };
  const int64_t c64 = cost(64, 90), c128 = cost(128, 140), c256 = cost(256, 256);
  if (c256 <= c128 && c256 <= c64) return launch_gemm_t<256, PL>(tx, wcodes, a, st);
  if (c128 <= c64) return launch_gemm_t<128, PL>(tx, wcodes, a, st);
  return launch_gemm_t<64, PL>(tx, wcodes, a, st);
}

template <typename T>
void planes(const void* x, int64_t ldx, int M, int K, int P, uint8_t* codes, uint8_t* scales,
            cudaStream_t st) {
  const int64_t total = (int64_t)M * ((K + 255) / 256);
  const unsigned grid = (unsigned)std::min<int64_t>((total + 7) / 8, (int64_t)num_sms() * 64);
  if (P == 1)
    mx_planes_kernel<T, 1><<<grid, 256, 0, st>>>(static_cast<const T*>(x), ldx, M, K, codes, scales);
  else
    mx_planes_kernel<T, 2><<<grid, 256, 0, st>>>(static_cast<const T*>(x), ldx, M, K, codes, scales);
}

}  // namespace

wq_status launch_mx_planes(const void* x, wq_dtype dt, int64_t ldx, int64_t M, int64_t K, int32_t P,
                           uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  if (dt == WQ_BF16)
    planes<__nv_bfloat16>(x, ldx, (int)M, (int)K, P, codes, scales, st);
  else if (dt == WQ_FP16)
    planes<__half>(x, ldx, (int)M, (int)K, P, codes, scales, st);
  else
    planes<float>(x, ldx, (int)M, (int)K, P, codes, scales, st);
  return launch_status();
}

size_t mx_gemm_workspace_bytes(int64_t, int64_t, int64_t, int32_t) { return 0; }

wq_status launch_mx_gemm(const uint8_t* xc, const uint8_t* xs, int64_t M, int64_t N, int64_t K,
                         int32_t P, const uint8_t* wc, const uint8_t* ws, void* y, void*,
                         cudaStream_t st) {
  CUtensorMap tx;
  if (!make_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, xc, (uint64_t)K / 2, (uint64_t)(P * M),
                    (uint64_t)K / 2, kBKBytes, kBM, CU_TENSOR_MAP_SWIZZLE_128B))
    return WQ_ERR_CUDA;
  MxArgs a;
  a.xs = xs;
  a.ws = ws;
  a.y = static_cast<uint16_t*>(y);
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.mt = a.tiles = 0;
  return P == 1 ? launch_gemm<1>(tx, wc, a, st) : launch_gemm<2>(tx, wc, a, st);
}

wq_status read_mx_gemm_error(bool clear, uint32_t* v) {
  uint32_t h = 0;
  if (cudaMemcpyFromSymbol(&h, g_mx_gemm_error, sizeof(h)) != cudaSuccess) return WQ_ERR_CUDA;
  if (clear && h) {
    const uint32_t z = 0;
    if (cudaMemcpyToSymbol(g_mx_gemm_error, &z, sizeof(z)) != cudaSuccess) return WQ_ERR_CUDA;
  }
  *v = h;
  return WQ_OK;
}

}  // namespace wq
