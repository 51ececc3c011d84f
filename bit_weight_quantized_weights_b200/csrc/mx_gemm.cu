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
#include <type_traits>
#include <utility>

#include "sm100.cuh"
#include "splitk_common.cuh"

namespace wq {

__device__ unsigned int g_mx_gemm_error;

namespace {

// ---------------------------------------------------------------------------
// Quantization of activations: one warp takes 512 consecutive elements of a
// row, 16 elements a lane, so a block of 32 is two lanes (one shuffle for its
// largest magnitude) and a lane's codes are one 64-bit store. 8192 x 4096 bf16: two
// planes 24.7 us (104 MB; a copy's rate would be 16), one 14.7; its instructions
// (320 a warp and 512 elements for two planes) hold it, issue 66%.
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

// Eight E2M1 codes of f[i] * scale, element i in nibble i (a negative value
// that rounds to zero has code 8 here).
__device__ __forceinline__ uint32_t e2m1_x8(const float* f, float scale) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(f[0] * scale), "f"(f[1] * scale), "f"(f[2] * scale), "f"(f[3] * scale),
        "f"(f[4] * scale), "f"(f[5] * scale), "f"(f[6] * scale), "f"(f[7] * scale));
  return w;
}

// Code 8 to code 0: zeros are +0.
__device__ __forceinline__ uint32_t plus_zero(uint32_t w) {
  const uint32_t some = (w | (w >> 1) | (w >> 2)) & 0x11111111u;  // magnitude above 0
  return w & (0x77777777u | (some << 3));
}

// The values of eight codes. (The conversion is given bytes of a word's low half
// only: from the third and fourth byte of an unpacked word, nvcc 12.9 returned
// zeros.)
__device__ __forceinline__ void e2m1_values(uint32_t w, float (&v)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
        : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
        : "r"(w >> (16 * i)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = t.x;
    v[2 * i + 1] = t.y;
  }
}

// 16 consecutive elements.
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&f)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 v = ld_stream_u4(p + 8 * h);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2 && __is_same(T, __nv_bfloat16)) {
        f[8 * h + 2 * i] = bf16_lo_to_f32(w[i]);
        f[8 * h + 2 * i + 1] = bf16_hi_to_f32(w[i]);
      } else {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[8 * h + 2 * i] = t.x;
        f[8 * h + 2 * i + 1] = t.y;
      }
    }
  }
}
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&f)[16]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint4 v = ld_stream_u4(p + 4 * h);
    f[4 * h] = __uint_as_float(v.x);
    f[4 * h + 1] = __uint_as_float(v.y);
    f[4 * h + 2] = __uint_as_float(v.z);
    f[4 * h + 3] = __uint_as_float(v.w);
  }
}

template <typename T, int PL>
__global__ void __launch_bounds__(256)
    mx_planes_kernel(const T* __restrict__ x, int64_t ldx, int M, int K,
                     uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  follow_previous();
  const int lane = threadIdx.x & 31;
  const uint32_t chunks = (uint32_t)(K + 511) / 512;
  const uint32_t total = (uint32_t)M * chunks;  // below 2^31
  for (uint32_t i = blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += gridDim.x * 8) {
    const uint32_t m = i / chunks;
    const int k = (int)(i - m * chunks) * 512 + 16 * lane;
    const bool in = k < K;  // whole blocks: K is a multiple of 32
    float f[16];
    if (in) {
      load16(x + (int64_t)m * ldx + k, f);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = 0.0f;
    }
#pragma unroll
    for (int p = 0; p < PL; ++p) {
      float a = 0.0f, b = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a = fmaxf(a, fabsf(f[j]));
        b = fmaxf(b, fabsf(f[8 + j]));
      }
      a = fmaxf(a, b);
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
      const int e = e2m1_exponent(a);
      const float down = pow2f(-e);
      const uint32_t w[2] = {e2m1_x8(f, down), e2m1_x8(f + 8, down)};
      if (in) {
        const int64_t row = (int64_t)p * M + m;
        *reinterpret_cast<uint2*>(codes + (row * K + k) / 2) =
            make_uint2(plus_zero(w[0]), plus_zero(w[1]));
        if ((lane & 1) == 0) scales[(row * K + k) / 32] = (uint8_t)(e + 127);
      }
      if (p + 1 < PL) {
        const float up = pow2f(e);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[8];
          e2m1_values(w[h], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[8 * h + j] = fmaf(-v[j], up, f[8 * h + j]);  // exact
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Scale bytes [rows][K / 32] to the order the MMA takes them in, a 512-byte
// piece for 128 rows x 4 scales (128 k): the 4 bytes of row r at byte
// (r % 32) * 16 + (r / 32) * 4, i.e. lane r % 32, column r / 32 of 4 TMEM
// columns. Pieces are ordered [row block][k / 256][2], zeros (the scale 2^-127)
// where there is no row or block. Loading the bytes a row at a time inside the
// product cost it as much as its MMAs (one 4-byte request a row and 128 k);
// this pass moves K N / 32 bytes once (7 us with cold caches at M = 8192, N = 14336,
// K = 4096, bound by latency).
// ---------------------------------------------------------------------------
struct ScaleArgs {
  const uint8_t* xs;  // [P][M][K / 32]
  const uint8_t* ws;  // [N][K / 32]
  uint8_t* out;       // pieces of x's row blocks (by plane), then w's
  int M, N, K, P;
  int xblocks;        // ceil(M / 128)
  int kt;             // ceil(K / 256)
  int chunks;         // CTAs along k: ceil(2 kt / 8)
};

__global__ void __launch_bounds__(256) mx_scales_kernel(const ScaleArgs a) {
  __shared__ __align__(16) uint32_t sm[8][128];  // piece, then word (r % 32) * 4 + r / 32
  follow_previous();  // (the product reads codes as soon as it starts)
  const int chunk = blockIdx.x % a.chunks, block = blockIdx.x / a.chunks;
  const int words = a.K / 128;  // 4-byte groups of a row
  const bool is_x = block < a.P * a.xblocks;
  const int p = is_x ? block / a.xblocks : 0;
  const int rb = is_x ? block - p * a.xblocks : block - a.P * a.xblocks;
  const int nrows = is_x ? a.M : a.N;
  const uint8_t* base = is_x ? a.xs + (int64_t)p * a.M * (a.K / 32) : a.ws;
  const int r = threadIdx.x >> 1, g0 = (threadIdx.x & 1) * 4;  // row, first of 4 groups
  const int row = rb * 128 + r;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(base + (int64_t)row * (a.K / 32));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int g = chunk * 8 + g0 + i;
    sm[g0 + i][(r & 31) * 4 + (r >> 5)] = row < nrows && g < words ? src[g] : 0u;
  }
  __syncthreads();
  const int piece = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (chunk * 8 + piece < 2 * a.kt)
    *reinterpret_cast<uint4*>(a.out + (((int64_t)block * 2 * a.kt + chunk * 8 + piece) * 512) +
                              16 * lane) = *reinterpret_cast<const uint4*>(&sm[piece][4 * lane]);
}

// ---------------------------------------------------------------------------
// Product. A tile is 128 tokens (the MMA's M) by BN features (its N), summed
// over all planes in one TMEM accumulator: a weight tile is loaded once and
// multiplied with every plane's token tile. A stage holds 256 k (128-byte rows
// of 4-bit codes, 128-byte swizzle) of all operands.
//   warp 0       TMA loads of the codes
//   warps 1, 2   tcgen05.mma: the whole warp runs the loop and one elected lane
//                issues, so that the operands' addresses are warp-uniform (a
//                loop of one lane spent 90 cycles an MMA moving them to the
//                uniform registers the instruction takes: 1100 cycles a stage)
//   warps 4-7    scales: one 16-byte load a lane and piece, tcgen05.st to a ring
//                of TMEM columns (every warp writes its lane quarter: the MMA
//                reads the scales from all four). tcgen05.cp from shared memory
//                by the MMA's thread took a fifth of the MMAs' time.
//                Small products load the bytes as given, a row a thread.
//   warps 8-15   epilogue: TMEM to registers as packed bf16, which frees the
//                accumulator for the next tile, then through shared memory to
//                TMA stores (rows of 128 bytes; one 16-byte store a token cost
//                70 us of 350 at 8192 x 14336 x 4096)
// CTAs are persistent and take every gridDim.x-th tile; where there are few tiles and
// a long K, the 2 or 4 CTAs of a cluster share a tile's K. 8192 x 14336 x 4096 with two
// planes: 325 us with the scale pass, 5.9 POP/s, the tensor cores busy 81% of the
// cycles (bare MMAs: 6.7 POP/s at the same power); with one plane 197 us, bound by
// the operands' way from L2; 33 x 4096 x 4096 6.8 us, bound by latency.
// ---------------------------------------------------------------------------
constexpr int kBM = 128;
constexpr int kBKBytes = 128;   // bytes of a stage's row: 256 k
constexpr int kThreads = 512;

template <int BN, int PL>
struct MxCfg {
  static constexpr int kXBytes = PL * kBM * kBKBytes;
  static constexpr int kWBytes = BN * kBKBytes;
  static constexpr int kStageBytes = kXBytes + kWBytes;
  static constexpr int kEpiWarps = BN >= 128 ? 8 : 4;
  static constexpr int kEpiCols = BN / (kEpiWarps / 4);       // features a warp takes
  static constexpr int kChunk = BN < 64 ? BN : 64;            // features of one store
  static constexpr int kStageOut = 32 * kChunk * 2;           // a warp's 32 tokens x kChunk
  static constexpr int kOutBytes = kEpiWarps * kStageOut;
  static constexpr int kMaxStages = (232448 - 1024 - 512 - kOutBytes) / kStageBytes;
  static constexpr int kStages = kMaxStages < 8 ? kMaxStages : 8;
  static constexpr int kSmem = kStages * kStageBytes + kOutBytes + 1024 + 512;
  // TMEM columns: the accumulator, then the ring of scales (4 columns a piece)
  static constexpr int kWPieces = (BN + 127) / 128;
  static constexpr int kSfCols = (PL + kWPieces) * 2 * 4;
  // stages whose scales are on their way in registers (32 registers a stage at
  // most): one stage ahead cost 0.55 us a stage, the latency of the loads
  static constexpr int kSfAhead = BN >= 256 ? 2 : 3;
  // Warps that issue MMAs. Issuing a stage (the wait, 4 or 8 MMAs, the commit)
  // takes 650 cycles, more than the MMAs of tiles up to 128 wide: two warps
  // then take the stages in turn, each with an accumulator of its own, which
  // the epilogue adds.
  static constexpr int kIssuers = BN <= 128 ? 2 : 1;
  static constexpr int kAccCols = kIssuers * BN;
  static constexpr int kCols = kAccCols + kStages * kSfCols;
  static constexpr int kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512, "TMEM columns");
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

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint4& a, const uint4& b) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
      : "memory");
}

struct MxArgs {
  const uint8_t* sf;  // scale pieces of the token blocks (by plane), then of the weights
  const uint8_t *xs, *ws;  // the scales as given (kDirect)
  int M, N, K;
  int mt, tiles;      // token tiles; all tiles
  int xrows;          // token rows a TMA load brings: 128, or M rounded up to 8
  int split;          // log2 of the CTAs that share a tile's K (above 0: one tile a CTA)
  uint16_t* y;
};

template <int BN, int PL, bool kDirect>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x,
                   const __grid_constant__ CUtensorMap tmap_w,
                   const __grid_constant__ CUtensorMap tmap_y, const MxArgs a, const WaitCtl wc) {
  using Cfg = MxCfg<BN, PL>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint8_t* sx = smem;                       // [stage][plane][128 rows]
  uint8_t* sw = sx + S * Cfg::kXBytes;      // [stage][BN rows]
  uint8_t* sout = sw + S * Cfg::kWBytes;    // [epilogue warp][32 rows of 128 bytes]
  uint64_t* full = reinterpret_cast<uint64_t*>(sout + Cfg::kOutBytes);
  uint64_t* empty = full + S;
  uint64_t* sffull = empty + S;
  uint64_t* acc_full = sffull + S;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* mma_done = acc_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KT = (a.K / 2 + kBKBytes - 1) / kBKBytes;
  // this CTA's first tile, and its stages [k0, k0 + KL) of every tile
  constexpr bool kSplits = BN == 64 || BN == 128;  // the widths that share K
  const int split = kSplits ? a.split : 0;
  const int rank = (int)blockIdx.x & ((1 << split) - 1);  // (clusters start at multiples)
  const int tile0 = (int)blockIdx.x >> split, tstep = (int)gridDim.x >> split;
  const int k0 = rank * KT >> split, KL = ((rank + 1) * KT >> split) - k0;

  if (threadIdx.x == 0) {
    sm100::tma_prefetch_desc(&tmap_x);
    sm100::tma_prefetch_desc(&tmap_w);
    sm100::tma_prefetch_desc(&tmap_y);
    for (int s = 0; s < S; ++s) {
      sm100::mbar_init(&full[s], 1);
      sm100::mbar_init(&empty[s], 1);
      sm100::mbar_init(&sffull[s], 4);
    }
    sm100::mbar_init(acc_full, Cfg::kIssuers);
    sm100::mbar_init(acc_empty, Cfg::kEpiWarps);
    sm100::mbar_init(mma_done, Cfg::kIssuers);
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
  const uint32_t tmem_sf = tmem + Cfg::kAccCols;
  // With the scale pass before it, this kernel starts when everything older is
  // complete (and a next call's pass set up early took 1 to 2 us from it).
  if (kDirect) follow_previous();

  int last_issued = -1;
  if (warp == 0) {
    int it = 0;
    bool ok = true;
    const uint32_t bytes = (uint32_t)(PL * a.xrows * kBKBytes) + Cfg::kWBytes;
    for (int t = tile0; t < a.tiles && ok; t += tstep) {
      const int m0 = (t % a.mt) * kBM, n0 = (t / a.mt) * BN;
      for (int kt = k0; kt < k0 + KL; ++kt, ++it) {
        const int s = it % S;
        if (it >= S) {
          ok = __all_sync(0xffffffffu,
                          sm100::mbar_wait(&empty[s], (uint32_t)(it / S - 1) & 1u,
                                           &g_mx_gemm_error, 0x3101u, abort_flag, wc.limit_ns));
          if (!ok) break;
        }
        if (wc.stall && it == 0) continue;  // test hook: the first k-tile never arrives
        last_issued = it;
        if (sm100::elect_one()) {
          sm100::mbar_arrive_expect_tx(&full[s], bytes);
#pragma unroll
          for (int p = 0; p < PL; ++p)
            sm100::tma_load_2d(sx + s * Cfg::kXBytes + p * kBM * kBKBytes, &tmap_x, &full[s],
                               kt * kBKBytes, p * a.M + m0);
          sm100::tma_load_2d(sw + s * Cfg::kWBytes, &tmap_w, &full[s], kt * kBKBytes, n0);
        }
        __syncwarp();
      }
    }
  } else if (warp <= Cfg::kIssuers) {
    const int who = warp - 1;
    const uint32_t xlo0 = sm100::uniform(sm100::sdesc_lo(smem_u32(sx)));
    const uint32_t wlo0 = sm100::uniform(sm100::sdesc_lo(smem_u32(sw)));
    const uint32_t tm = sm100::uniform(tmem), acc = tm + (uint32_t)(who * BN);
    int it0 = 0, n = 0;  // the tile's first stage; the tile
    bool ok = true;
    for (int t = tile0; t < a.tiles && ok; t += tstep, ++n, it0 += KL) {
      if (n > 0) {
        ok = __all_sync(0xffffffffu,
                        sm100::mbar_wait(acc_empty, (uint32_t)(n - 1) & 1u, &g_mx_gemm_error,
                                         0x3201u, abort_flag, wc.limit_ns));
        if (!ok) break;
        sm100::tc_fence_after();
      }
      for (int kt = who; kt < KL; kt += Cfg::kIssuers) {
        const int it = it0 + kt, s = it % S;
        const uint32_t ph = (uint32_t)(it / S) & 1u;
        ok = __all_sync(0xffffffffu, sm100::mbar_wait(&full[s], ph, &g_mx_gemm_error, 0x3202u,
                                                      abort_flag, wc.limit_ns) &&
                                         sm100::mbar_wait(&sffull[s], ph, &g_mx_gemm_error,
                                                          0x3203u, abort_flag, wc.limit_ns));
        if (!ok) break;
        sm100::tc_fence_after();
        const uint32_t sf = tm + Cfg::kAccCols + (uint32_t)(s * Cfg::kSfCols);
        const uint32_t xlo = xlo0 + (uint32_t)(s * (Cfg::kXBytes >> 4));
        const uint32_t wlo = wlo0 + (uint32_t)(s * (Cfg::kWBytes >> 4));
        if (sm100::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // 64 k each: 32 bytes, 2 scale bytes
            const int kg = kk >> 1;
            const uint32_t idesc = (kk & 1) ? idesc_mxf4(BN, 2) : idesc_mxf4(BN, 0);
            const uint32_t sfb = sf + PL * 8 + kg * 4 * Cfg::kWPieces;
#pragma unroll
            for (int p = 0; p < PL; ++p)
              mma_mxf4(acc, sm100::sdesc_at(xlo + p * (kBM * kBKBytes >> 4) + kk * 2),
                       sm100::sdesc_at(wlo + kk * 2), idesc, sf + (p * 2 + kg) * 4, sfb,
                       (kk | p) != 0 || kt != who ? 1u : 0u);
          }
          sm100::mma_commit(&empty[s]);
        }
        __syncwarp();
      }
      if (ok && sm100::elect_one()) sm100::mma_commit(acc_full);
      __syncwarp();
    }
    if (sm100::elect_one()) sm100::mma_commit(mma_done);
    __syncwarp();
  } else if (kDirect && warp >= 4 && warp < 8) {
    // ---------------- scales as they are given: one tile a CTA ----------------
    // Thread = row of every operand; the rows' words meet in shared memory (the
    // epilogue's buffers, which are free until the tile is complete).
    constexpr int D = Cfg::kSfAhead, kOps = PL + 1;
    static_assert(!kDirect || (Cfg::kWPieces == 1 && 2 * kOps * 1024 <= Cfg::kOutBytes),
                  "one block of features, two stages of pieces");
    const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
    const int r = 32 * (warp & 3) + lane, words = a.K / 128;
    const uint32_t* src[kOps];  // null: no such row, or features past the tile
#pragma unroll
    for (int o = 0; o < kOps; ++o) {
      const int row = o < PL ? (tile0 % a.mt) * kBM + r : tile0 / a.mt * BN + r;
      const bool in = o < PL ? row < a.M : row < a.N && r < BN;
      const uint8_t* base = o < PL ? a.xs + (int64_t)o * a.M * (a.K / 32) : a.ws;
      src[o] = in ? reinterpret_cast<const uint32_t*>(base + (int64_t)row * (a.K / 32)) : nullptr;
    }
    const bool pairs = (words & 1) == 0;  // K % 256 == 0: a stage's two words are aligned
    auto load = [&](uint32_t (&v)[kOps][2], int it) {
      const int kt = k0 + it;
#pragma unroll
      for (int o = 0; o < kOps; ++o) {
        if (pairs) {
          const uint2 w = src[o] ? *reinterpret_cast<const uint2*>(src[o] + 2 * kt)
                                 : make_uint2(0u, 0u);
          v[o][0] = w.x, v[o][1] = w.y;
        } else {
          v[o][0] = src[o] ? src[o][2 * kt] : 0u;
          v[o][1] = src[o] && 2 * kt + 1 < words ? src[o][2 * kt + 1] : 0u;
        }
      }
    };
    uint32_t v[D][kOps][2];
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (d < KL) load(v[d], d);
    bool ok = true;  // (after an abort the warps still meet at every stage's barrier)
    for (int base = 0; base < KL; base += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int it = base + d;
        if (it >= KL) break;
        uint32_t* buf = reinterpret_cast<uint32_t*>(sout + (it & 1) * kOps * 1024);
#pragma unroll
        for (int o = 0; o < kOps; ++o)
#pragma unroll
          for (int g = 0; g < 2; ++g) buf[(2 * o + g) * 128 + 4 * lane + (warp & 3)] = v[d][o][g];
        if (it + D < KL) load(v[d], it + D);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int f = it % S;
        if (ok && it >= S)
          ok = __all_sync(0xffffffffu,
                          sm100::mbar_wait(&empty[f], (uint32_t)(it / S - 1) & 1u,
                                           &g_mx_gemm_error, 0x3301u, abort_flag, wc.limit_ns));
        if (ok) {
          sm100::tc_fence_after();
          const uint4* piece = reinterpret_cast<const uint4*>(buf) + lane;
#pragma unroll
          for (int o = 0; o < kOps; ++o)
            tmem_st8(tmem_sf + quarter + (uint32_t)(f * Cfg::kSfCols + 8 * o), piece[64 * o],
                     piece[64 * o + 32]);
          sm100::tmem_st_wait();
          sm100::tc_fence_before();
          __syncwarp();
          if (lane == 0) sm100::mbar_arrive(&sffull[f]);
        }
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------- scales ----------------
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the pieces are complete
    constexpr int kPieces = Cfg::kSfCols / 4;
    const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
    // the pieces of one stage in column order: planes (2 of k each), then the
    // weights' by k. They are 1024 bytes (2 pieces) after the stage before's.
    constexpr int D = Cfg::kSfAhead;
    const int mine = tile0 < a.tiles ? (a.tiles - 1 - tile0) / tstep + 1 : 0;
    const int total = mine * KL;  // stages of this CTA
    const uint8_t *px[PL], *pw[Cfg::kWPieces];
    int lt = tile0, lk = 0;  // the next stage to load
    auto next = [&](uint4 (&v)[kPieces]) {
      if (lk == 0) {
        const int mb = lt % a.mt, n0 = (lt / a.mt) * BN;
#pragma unroll
        for (int p = 0; p < PL; ++p)
          px[p] = a.sf + ((int64_t)(p * a.mt + mb) * KT + k0) * 1024 + 16 * lane;
#pragma unroll
        for (int w = 0; w < Cfg::kWPieces; ++w)
          // a block of 128 features past N has no pieces: its columns are not stored
          pw[w] = a.sf +
                  ((int64_t)(PL * a.mt + min(n0 / 128 + w, (a.N - 1) / 128)) * KT + k0) * 1024 +
                  16 * lane;
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int j = i - 2 * PL;
        v[i] = *reinterpret_cast<const uint4*>(
            i < 2 * PL ? px[i >> 1] + 512 * (i & 1)
                       : pw[j % Cfg::kWPieces] + 512 * (j / Cfg::kWPieces));
      }
#pragma unroll
      for (int p = 0; p < PL; ++p) px[p] += 1024;
#pragma unroll
      for (int w = 0; w < Cfg::kWPieces; ++w) pw[w] += 1024;
      if (++lk == KL) {
        lk = 0;
        lt += tstep;
      }
    };
    uint4 v[D][kPieces];
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (d < total) next(v[d]);
    bool ok = true;
    int st = tile0, sk = 0, c = 0;  // the stage being stored
    for (int base = 0; base < total && ok; base += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int it = base + d;
        if (it >= total || !ok) break;
        const int f = it % S;
        if (it >= S) {
          const bool got = sm100::mbar_wait(&empty[f], (uint32_t)(it / S - 1) & 1u,
                                            &g_mx_gemm_error, 0x3301u, abort_flag, wc.limit_ns);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          sm100::tc_fence_after();
        }
        if (BN < 128) {
          // a tile inside a block of 128 features: rows 32 c .. are column c
          if (sk == 0) c = ((st / a.mt) * BN & 127) / 32;
#pragma unroll
          for (int i = 2 * PL; i < kPieces; ++i) {
            if (c & 2) v[d][i] = make_uint4(v[d][i].z, v[d][i].w, 0u, 0u);
            if (c & 1) v[d][i].x = v[d][i].y;
          }
          if (++sk == KL) {
            sk = 0;
            st += tstep;
          }
        }
#pragma unroll
        for (int i = 0; i < kPieces; i += 2)
          tmem_st8(tmem_sf + quarter + (uint32_t)(f * Cfg::kSfCols + 4 * i), v[d][i], v[d][i + 1]);
        if (it + D < total) next(v[d]);
        sm100::tmem_st_wait();
        sm100::tc_fence_before();
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&sffull[f]);
      }
    }
  } else if (split == 0 && warp >= 8 && warp < 8 + Cfg::kEpiWarps) {
    // ---------------- epilogue: thread = token, kEpiCols of the tile's features ----------------
    const int q = warp & 3, part = (warp - 8) >> 2;
    constexpr int kCols = Cfg::kEpiCols;
    uint8_t* buf = sout + (warp - 8) * Cfg::kStageOut;
    int n = 0;
    for (int t = tile0; t < a.tiles; t += tstep, ++n) {
      const int m0 = (t % a.mt) * kBM + 32 * q;
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
        if (Cfg::kIssuers == 2 && KL > 1) {
          uint32_t u[32];
          sm100::tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + BN + part * kCols + 32 * c, u);
          sm100::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
          out[16 * c + j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
      }
      sm100::tc_fence_before();
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(acc_empty);
      constexpr int kChunk = Cfg::kChunk;
#pragma unroll
      for (int c = 0; c < kCols / kChunk; ++c) {
        // 16-byte piece i of token row `lane`, in the store's swizzle: rows of
        // 128 bytes have piece i at i ^ (row % 8), of 64 bytes at i ^ (row / 2 % 4)
        const int sw = kChunk == 64 ? lane & 7 : (lane >> 1) & 3;
        if (lane == 0) sm100::bulk_wait_read_all();  // the store before has left the buffer
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kChunk / 8; ++i) {
          const uint32_t* o = out + kChunk / 2 * c + 4 * i;
          *reinterpret_cast<uint4*>(buf + lane * kChunk * 2 + ((i ^ sw) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        sm100::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && m0 < a.M && col0 + kChunk * c < a.N) {
          sm100::tma_store_2d(&tmap_y, buf, col0 + kChunk * c, m0);  // clipped at M and N
          sm100::bulk_commit();
        }
      }
    }
    if (lane == 0) sm100::bulk_wait_all();
  }

  // ---------------- a tile's K over the cluster ----------------
  // Every rank leaves its sums in its own stages (free by then), [row][BN] fp32 with
  // 16-byte piece i of a row at i ^ (row % 8) within 128 bytes; rank r adds the tile's
  // columns [r BN / C, (r + 1) BN / C) of all C ranks, in their order, and stores them.
  if (kSplits && split > 0) {
    const int m0 = (tile0 % a.mt) * kBM, n0 = tile0 / a.mt * BN;
    const int rows = min(kBM, a.M - m0);
    auto place = [](int row, int piece) {
      return (uint32_t)(row * BN * 4 + ((piece ^ (row & 7)) << 4));
    };
    if (warp >= 8 && warp < 8 + Cfg::kEpiWarps) {
      const int q = warp & 3, part = (warp - 8) >> 2, row = 32 * q + lane;
      const bool got = __all_sync(
          0xffffffffu, sm100::mbar_wait(acc_full, 0u, &g_mx_gemm_error, 0x3402u, abort_flag,
                                        wc.limit_ns));
      sm100::tc_fence_after();
      if (got && 32 * q < rows) {
#pragma unroll
        for (int c = 0; c < Cfg::kEpiCols / 32; ++c) {
          const int col = part * Cfg::kEpiCols + 32 * c;
          const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)col;
          uint32_t v[32];
          sm100::tmem_ld32(at, v);
          sm100::tmem_ld_wait();
          if (Cfg::kIssuers == 2 && KL > 1) {
            uint32_t u[32];
            sm100::tmem_ld32(at + BN, u);
            sm100::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(u[j]));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(smem + place(row, col / 4 + i)) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
    }
    __syncwarp();
    splitk::cluster_sync_all();
    auto finish = [&](auto ranks) {
      constexpr int C = decltype(ranks)::value;
      constexpr int kGroups = BN / C / 8;  // of 8 columns, a thread each
      uint32_t src[C];
#pragma unroll
      for (int r = 0; r < C; ++r) src[r] = splitk::map_rank(smem, (uint32_t)r);
      for (int u = threadIdx.x; u < rows * kGroups; u += kThreads) {
        const int row = u / kGroups, col = rank * (BN / C) + u % kGroups * 8;
        if (n0 + col >= a.N) continue;
        float4 x[C][2];
#pragma unroll
        for (int r = 0; r < C; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[r][h].x), "=f"(x[r][h].y), "=f"(x[r][h].z), "=f"(x[r][h].w)
                         : "r"(src[r] + place(row, col / 4 + h)));
#pragma unroll
        for (int r = 1; r < C; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            x[0][h] = make_float4(x[0][h].x + x[r][h].x, x[0][h].y + x[r][h].y,
                                  x[0][h].z + x[r][h].z, x[0][h].w + x[r][h].w);
        *reinterpret_cast<uint4*>(a.y + (int64_t)(m0 + row) * a.N + n0 + col) =
            make_uint4(pack_bf16x2(x[0][0].x, x[0][0].y), pack_bf16x2(x[0][0].z, x[0][0].w),
                       pack_bf16x2(x[0][1].x, x[0][1].y), pack_bf16x2(x[0][1].z, x[0][1].w));
      }
    };
    if (BN == 64 || split == 1)
      finish(std::integral_constant<int, 2>{});
    else
      finish(std::integral_constant<int, 4>{});
    __syncwarp();
    splitk::cluster_sync_all();  // nobody leaves while its sums are read
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

template <int BN, int PL, bool kDirect>
wq_status launch_gemm_t(const CUtensorMap& tx, const void* wcodes, void* y, const MxArgs& a0,
                        cudaStream_t st) {
  using Cfg = MxCfg<BN, PL>;
  CUtensorMap tw, ty;
  if (!make_tmap_2d(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, (uint64_t)a0.N, (uint64_t)a0.M,
                    (uint64_t)a0.N * 2, Cfg::kChunk, 32,
                    Cfg::kChunk == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return WQ_ERR_CUDA;
  if (!make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, wcodes, (uint64_t)a0.K / 2,
                    (uint64_t)a0.N, (uint64_t)a0.K / 2, kBKBytes, BN, CU_TENSOR_MAP_SWIZZLE_128B))
    return WQ_ERR_CUDA;
  static std::atomic<uint64_t> smem_set{0};
  if (!allow_smem(mx_gemm_kernel<BN, PL, kDirect>, Cfg::kSmem, smem_set)) return WQ_ERR_CUDA;
  MxArgs a = a0;
  a.tiles = a.mt * ((a.N + BN - 1) / BN);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (a.split > 0) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = 1u << a.split;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  cfg.stream = st;
  cfg.gridDim = dim3((unsigned)(a.split > 0 ? a.tiles << a.split : std::min(a.tiles, num_sms())), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  if (cudaLaunchKernelEx(&cfg, mx_gemm_kernel<BN, PL, kDirect>, tx, tw, ty, a, wait_ctl()) != cudaSuccess)
    return WQ_ERR_CUDA;
  return launch_status();
}

template <int BN, int PL>
wq_status launch_width(const CUtensorMap& tx, const void* wcodes, void* y, const MxArgs& a,
                       const ScaleArgs& sa, cudaStream_t st) {
  // Few rows of scales, and a tile a CTA: the product takes them as they are and the
  // pass is saved. Two planes, K = 4096, with the pass and without, K not split: 33
  // tokens x 4096 features 9.8 and 9.2 us, 64 9.5 and 9.5, 96 9.6 and 10.5, 64 x 14336
  // 11.7 and 12.6; one plane: 33 x 4096 8.7 and 7.3, 128 8.9 and 8.3, 128 x 14336 10.4
  // and 11.3. A CTA with few stages may have more rows for the same saving: where K is
  // shared (1 to 200 tokens, 1024 to 4608 features, K to 14336, one and two planes: 193
  // shapes) the pass takes 1.5 to 1.0 of the direct form's time up to 2300 row-stages
  // and 1.14 to 0.73 of it beyond; the rule's choice is at most 7% from the faster one.
  if constexpr (BN <= 128) {
    const int64_t tiles = (int64_t)a.mt * ((a.N + BN - 1) / BN);
    const int rows = PL * std::min(a.M, kBM) + BN;
    if (tiles <= num_sms() && (rows <= 176 || rows * (sa.kt >> a.split) <= 2300))
      return launch_gemm_t<BN, PL, true>(tx, wcodes, y, a, st);
  }
  const int64_t blocks = (int64_t)PL * a.mt + (a.N + 127) / 128;
  wq_status s =
      launch_following(mx_scales_kernel, (unsigned)(blocks * sa.chunks), 256, 0, st, sa);
  return s != WQ_OK ? s : launch_gemm_t<BN, PL, false>(tx, wcodes, y, a, st);
}

template <int PL>
wq_status launch_gemm(const CUtensorMap& tx, const void* wcodes, void* y, const MxArgs& a0,
                      const ScaleArgs& sa, cudaStream_t st) {
  // The tile width with the least time for the slowest CTA: whole tiles an SM takes,
  // times a tile's cost.
  const int64_t mt = a0.mt, sms = num_sms();
  auto tiles = [&](int bn) { return mt * (((int64_t)a0.N + bn - 1) / bn); };
  int bn = 32, split = 0;
  int64_t least = INT64_MAX;
  for (auto [width, tile] : {std::pair(256, 256), {128, 140}, {64, 90}, {32, 70}}) {
    const int64_t cost = (tiles(width) + sms - 1) / sms * tile;
    if (cost < least) least = cost, bn = width;
  }
  // A tile a CTA: its stages, one after the other, are the time (ns a stage; the product
  // of 33 x 4096 x 11008, two planes, took 18.1 us). Wider tiles whose K is shared by
  // the CTAs of a cluster have fewer, for the sums' way through shared memory (two
  // cluster barriers, and BN floats a row): 128 wide and 4 CTAs 11.0 us, 64 and 2 13.3.
  // With 128 rows and K = 4096 it does not pay: 9.9 us with 32 wide tiles, 12.5 with
  // 128 and 4; with K = 14336 it does: 23.4 and 15.7.
  // At most 128 CTAs: 33 clusters of 4 are resident at once, and one more takes a second
  // wave (36 tiles in clusters of 4 instead of 2, 1 x 4608 x 4096: 5.4 and 8.3 us). Of 2
  // there are 74; 72 tiles in clusters of 2 are not taken yet (1 x 9216 x 11008: 14.5 us
  // as it is, 10.3).
  if (tiles(bn) <= sms) {
    auto time = [&](int width, int s) {
      const int64_t stage = PL == 1 ? (width == 32 ? 280 : width == 64 ? 330 : 320)
                                    : (width == 32 ? 340 : width == 64 ? 370 : 390);
      const int64_t sums = s > 0 ? 1200 + width * std::min(a0.M, kBM) / 4 : 0;
      return ((sa.kt + (1 << s) - 1) >> s) * stage + sums;
    };
    int64_t best = bn <= 128 ? time(bn, 0) : 0;
    for (auto [width, s] : {std::pair(64, 1), {128, 1}, {128, 2}})
      if (2 << s <= sa.kt && tiles(width) << s <= 128 && time(width, s) < best)
        best = time(width, s), bn = width, split = s;
  }
  MxArgs a = a0;
  a.split = split;
  switch (bn) {
    case 32: return launch_width<32, PL>(tx, wcodes, y, a, sa, st);
    case 64: return launch_width<64, PL>(tx, wcodes, y, a, sa, st);
    case 128: return launch_width<128, PL>(tx, wcodes, y, a, sa, st);
    default: return launch_width<256, PL>(tx, wcodes, y, a, sa, st);
  }
}

template <typename T>
wq_status planes(const void* x, int64_t ldx, int M, int K, int P, uint8_t* codes, uint8_t* scales,
            cudaStream_t st) {
  const int64_t total = (int64_t)M * ((K + 511) / 512);
  const unsigned grid = (unsigned)std::min<int64_t>((total + 7) / 8, (int64_t)num_sms() * 64);
  return launch_following(P == 1 ? mx_planes_kernel<T, 1> : mx_planes_kernel<T, 2>, grid, 256, 0,
                          st, static_cast<const T*>(x), ldx, M, K, codes, scales);
}

}  // namespace

wq_status launch_mx_planes(const void* x, wq_dtype dt, int64_t ldx, int64_t M, int64_t K, int32_t P,
                           uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  if (dt == WQ_BF16)
    return planes<__nv_bfloat16>(x, ldx, (int)M, (int)K, P, codes, scales, st);
  if (dt == WQ_FP16) return planes<__half>(x, ldx, (int)M, (int)K, P, codes, scales, st);
  return planes<float>(x, ldx, (int)M, (int)K, P, codes, scales, st);
}

// Workspace: the scale pieces of all planes' token blocks and of the weights'
// feature blocks.
size_t mx_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t P) {
  return (size_t)(P * ((M + 127) / 128) + (N + 127) / 128) * ((K + 255) / 256) * 1024;
}

wq_status launch_mx_gemm(const uint8_t* xc, const uint8_t* xs, int64_t M, int64_t N, int64_t K,
                         int32_t P, const uint8_t* wc, const uint8_t* ws, void* y, void* workspace,
                         cudaStream_t st) {
  // with fewer than 128 tokens the rest of the tile's rows is not loaded: an
  // MMA row depends on its own operand row only, and rows past M are not stored
  const int xrows = (int)std::min<int64_t>(kBM, (M + 7) / 8 * 8);
  CUtensorMap tx;
  if (!make_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, xc, (uint64_t)K / 2, (uint64_t)(P * M),
                    (uint64_t)K / 2, kBKBytes, (uint32_t)xrows, CU_TENSOR_MAP_SWIZZLE_128B))
    return WQ_ERR_CUDA;
  ScaleArgs sa;
  sa.xs = xs;
  sa.ws = ws;
  sa.out = static_cast<uint8_t*>(workspace);
  sa.M = (int)M;
  sa.N = (int)N;
  sa.K = (int)K;
  sa.P = P;
  sa.xblocks = (int)((M + 127) / 128);
  sa.kt = (int)((K + 255) / 256);
  sa.chunks = (2 * sa.kt + 7) / 8;
  MxArgs a;
  a.sf = sa.out;
  a.xs = xs;
  a.ws = ws;
  a.y = static_cast<uint16_t*>(y);
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.mt = sa.xblocks;
  a.tiles = 0;
  a.xrows = xrows;
  return P == 1 ? launch_gemm<1>(tx, wc, y, a, sa, st) : launch_gemm<2>(tx, wc, y, a, sa, st);
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
