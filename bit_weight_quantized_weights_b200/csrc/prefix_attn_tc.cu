// The prefix part of the shared-prefix attention on the tcgen05 tensor cores,
// for batches whose query rows fill their tiles (the mathematics is in
// prefix_attn.cu; a row's result over a range of keys goes to a slot of the
// partial results that the merge kernel combines).
//
// A CTA runs two streams of 128 query rows x 128-key tiles, so that the
// products of one overlap the softmax of the other:
//   MT = 2  two row tiles against the same keys: a key tile is dequantized once
//           for 256 rows;
//   MT = 1  one row tile against the even and the odd key tiles of the range
//           (two independent partial results).
// Tensor memory holds both streams' scores (128 columns each, overwritten by
// their fp16 weights) and outputs. Per stream and tile:
//   S = Q K^T      A, B in shared memory (fp16, 128-byte swizzle, K-major)
//   softmax        a warp takes 16 rows
//   O += P V       A = the weights in tensor memory
// Roles: warps 0-7 and 8-15 softmax of stream 0 and 1, warps 16-23 dequantize
// keys and values into shared memory (two stages each; 16 keys a warp), warp 24
// issues (25-27 fill its warpgroup).
// The operands are the dequantized values themselves, (q - z) s rounded once to
// fp16 (2^-11), up to a power of two common to 32 keys: a score's scale and the
// exponent's offset are then one multiply-add. Exact integers with the scales in
// a table per key cost 12 bytes of shared memory a column and row, beside the
// MMAs' operands, and two more operations a weight.
// Outputs in fp16 (kExact) are eight times finer than in bf16, and there those
// two roundings would more than double the error: the operands take the leading
// 7 bits of the scales, which makes them exact, and the rest multiplies the
// score and the weight, two operations a weight.
//
// What bounds it: a tile of 256 rows x 128 keys takes about 4700 cycles, its MMAs
// and its exponentials 2050 each, its 11200 warp instructions 2800 (softmax 5600,
// dequantization 3100); a stream's scores, softmax and values follow one another and
// two streams cover each other in part. 1024 rows x 8 heads x 65537 keys, with the
// own tokens and the merge: 306 us with bf16 queries (898 TFLOP/s), 388 with fp16;
// 512 x 8 x 32768: 98 and 118 us.
//
// MMAs of one issuing thread execute in order, so S of a tile completes after
// the O += P V issued before it: when a softmax warp sees its scores it may
// rescale its rows of O, and the next S may overwrite P.
#include <algorithm>

#include "prefix_attn.cuh"
#include "sm100.cuh"

namespace wq {

__device__ unsigned int g_prefix_error;

namespace {

using namespace prefix;

constexpr int kTile = 128;                 // keys of a tile, rows of a row tile
constexpr int kSoftWarps = 16;             // 8 a stream
constexpr int kDeqWarps = 8;
constexpr int kIssueWarp = kSoftWarps + kDeqWarps;
constexpr int kThreads = 28 * 32;
// Registers a thread of each warpgroup (72 the softmax): 4 * 72 + 2 * 88 + 40 = 7 * 72, what the
// block is launched with; the dequantization keeps the next tile's codes.
constexpr int kRegsDequant = 88, kRegsIssue = 40;
constexpr int kOpBytes = kTile * kD * 2;   // an operand tile: two 64-element atoms of 16 KB
constexpr int kAtomBytes = kOpBytes / 2;
// A row's bound is put 2^6 below its largest weight, and moves before a lane's sum of 4
// weights passes 2^15 (with the scales' rest, at most 2^-4 of it, still in fp16): keys of
// 2^-19 of the largest weight keep all bits of theirs.
constexpr float kLiftTc = 6.0f, kSumMax = 32768.0f;
constexpr int kTabs = 4;                   // key-table stages
constexpr int kColO = 256;                 // TMEM columns of the outputs (scores: 0 and 128)

template <int MT>
constexpr int smem_bytes() {
  return 1024 + (MT + 4) * kOpBytes + kTabs * (4 * 16 + kTile / 2 * 8) + 256;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  return h2(__hmul2(as_h2(a), as_h2(b)));
}

__device__ __forceinline__ float pow2(int x) { return __uint_as_float((uint32_t)(127 + x) << 23); }

// The scale's leading 7 bits, whose product with q - z (4 bits) is exact in
// fp16, and what is left of it: s / head - 1 < 2^-6 (2^-15 as bf16). Subnormal
// scales have 10 bits at most and no leading one of their own: from 2^7 units on
// the lowest 3 go (s / head - 1 < 2^-4, 2^-13 as bf16), below that none.
__device__ __forceinline__ uint32_t scale_head(uint32_t bits) {
  return bits & (bits >= 0x400u ? 0xFFF0u : bits >= 0x80u ? 0xFFF8u : 0xFFFFu);
}
__device__ __forceinline__ float scale_rest(uint32_t bits) {
  const float h = __half2float(__ushort_as_half((unsigned short)scale_head(bits)));
  const float s = __half2float(__ushort_as_half((unsigned short)bits));
  return h > 0.0f ? __fdividef(s - h, h) : 0.0f;
}

// fp16 bits of a lane's scale (kExact: of its head) / 2^x, with x (returned)
// such that the largest of the warp's scales becomes [2^10, 2^11) (a largest
// below fp16's normal range counts as 2^-14).
template <bool kExact>
__device__ __forceinline__ uint32_t norm_scale(uint32_t bits, int& x) {
  const uint32_t top = __reduce_max_sync(0xffffffffu, bits & 0x7FFFu);
  x = max((int)(top >> 10), 1) - 25;
  const uint32_t b = kExact ? scale_head(bits) : bits;
  const float s = __half2float(__ushort_as_half((unsigned short)b)) * pow2(-x);
  return __half_as_ushort(__float2half_rn(s));
}

// 32 columns of 16 TMEM lanes: registers 4 j .. 4 j + 3 hold columns 8 j +
// 2 t4, + 1 of row g, then of row g + 8 (lane = 4 g + t4).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_16x256b_x2(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                   taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
               "r"(r[7])
               : "memory");
}
// 16 columns of 16 lanes, one 32-bit column a lane: registers 2 j, 2 j + 1 hold
// column 4 j + t4 of rows g and g + 8.
__device__ __forceinline__ void tmem_ld_16x128b_x4(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                   taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
               "r"(r[7])
               : "memory");
}

template <int MT, bool kExact>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ PrefixArgs p, const WaitCtl wc) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint8_t* sq = smem;                          // [row tile]
  uint8_t* sk = sq + MT * kOpBytes;            // [stage]
  uint8_t* sv = sk + 2 * kOpBytes;             // [stage]
  // [stage][32 keys]: 2^x of the keys' scales, y of the values', 2^-y
  float4* tab = reinterpret_cast<float4*>(sv + 2 * kOpBytes);
  // kExact, [stage][pair of columns]: what the keys' scores and the weights are to
  // be multiplied with, less 1, as two bf16 each
  uint2* fac = reinterpret_cast<uint2*>(tab + kTabs * 4);
  uint64_t* bars = reinterpret_cast<uint64_t*>(fac + kTabs * (kTile / 2));
  uint64_t* q_full = bars;
  uint64_t* k_full = bars + 1;    // [2]
  uint64_t* k_empty = bars + 3;   // [2]
  uint64_t* v_full = bars + 5;    // [2]
  uint64_t* v_empty = bars + 7;   // [2]
  uint64_t* s_full = bars + 9;    // [stream]
  uint64_t* p_full = bars + 11;   // [stream]
  uint64_t* o_full = bars + 13;   // [stream]
  uint64_t* t_empty = bars + 15;  // [kTabs]
  uint64_t* mma_done = bars + 19;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 20);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's KV head, row tiles and keys
  const int splits = MT == 2 ? p.nsp : p.nsp / 2;
  const int split = blockIdx.x % splits;
  const int rg = (blockIdx.x / splits) % p.nrt;  // group of MT row tiles
  const int kh = blockIdx.x / (splits * p.nrt);
  const int begin = split * p.chunk_p;
  const int end = min(begin + p.chunk_p, p.P);
  const int T = (end - begin + kTile - 1) / kTile;

  if (threadIdx.x == 0) {
    sm100::mbar_init(q_full, 8 * MT);
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&k_full[i], kDeqWarps);
      sm100::mbar_init(&k_empty[i], 1);
      sm100::mbar_init(&v_full[i], kDeqWarps);
      sm100::mbar_init(&v_empty[i], 1);
      sm100::mbar_init(&s_full[i], 1);
      sm100::mbar_init(&p_full[i], 8);
      sm100::mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < kTabs; ++i) sm100::mbar_init(&t_empty[i], 8 * MT);
    sm100::mbar_init(mma_done, 1);
    *abort_flag = 0;
    sm100::fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    sm100::tmem_alloc(tmem_slot, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  follow_previous();  // (the kernel of the own tokens reads as soon as it starts)

  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
    // one suspended poll of up to 20 us covers the waits of a running pipeline
    return __all_sync(0xffffffffu,
                      sm100::mbar_try_wait_hint(bar, parity & 1u, 20000) ||
                          sm100::mbar_wait(bar, parity & 1u, &g_prefix_error, site, abort_flag,
                                           wc.limit_ns));
  };

  if (warp < kSoftWarps) {
    // ---------------- softmax: warp = 16 rows ----------------
    const int s = warp >> 3;                               // stream
    const int r0 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);  // first row: half a TMEM lane quarter
    const int base = (MT == 2 ? 2 * rg + s : rg) * kTile + r0;
    const uint32_t lanes = (uint32_t)r0 << 16;
    const int nrows = p.B * p.R;
    float cr;
    {
      // two lanes a row of Q: fp16 times a power of two; rows past the batch are zeros
      const int r = r0 + (lane >> 1), part = lane & 1;
      const int row = base + (lane >> 1);
      const bool have = row < nrows;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(p.q) +
          (have ? (int64_t)(row / p.R) * p.q_stride + (int64_t)(kh * p.R + row % p.R) * kD : 0));
      // (one round of loads: this latency starts the whole pipeline)
      uint4 v[kD / 16];
#pragma unroll
      for (int j = 0; j < kD / 16; ++j)
        v[j] = have ? src[8 * part + j] : make_uint4(0, 0, 0, 0);
      auto values = [&](const uint4& x, float (&f)[8]) {
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (p.fp16) {
            const float2 t = __half22float2(as_h2(u[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
          } else {
            f[2 * i] = bf16_lo_to_f32(u[i]);
            f[2 * i + 1] = bf16_hi_to_f32(u[i]);
          }
        }
      };
      float amax = 0.0f, up, down;
#pragma unroll
      for (int j = 0; j < kD / 16; ++j) {
        float f[8];
        values(v[j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      row_scale(amax, up, down);
      cr = down * kScoreScale;
      if (MT == 2 || s == 0) {
        uint8_t* dst = sq + s * kOpBytes + part * kAtomBytes + r * 128;
#pragma unroll
        for (int j = 0; j < kD / 16; ++j) {
          float f[8];
          values(v[j], f);
          *reinterpret_cast<uint4*>(dst + ((j ^ (r & 7)) << 4)) =
              make_uint4(pack_f16x2(f[0] * up, f[4] * up), pack_f16x2(f[1] * up, f[5] * up),
                         pack_f16x2(f[2] * up, f[6] * up), pack_f16x2(f[3] * up, f[7] * up));
        }
        sm100::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(q_full);
      }
    }
    const uint32_t ts = tmem + lanes + (uint32_t)(s * kTile);
    const uint32_t to = tmem + lanes + (uint32_t)(kColO + s * kD);
    // Scores come in the layout of 16-lane, 8-column accumulator fragments:
    // lane (g, t4) holds columns 8 j + 2 t4 and + 1 (tokens 8 j + t4 and + 4) of
    // rows g and g + 8. Eight warps a stream, 16 rows each, keep the exponentials
    // busy while others of them wait for their scores or store: four warps of 32
    // rows took 2850 cycles a tile, 1024 of them exponentials.
    const int g = lane >> 2, t4 = lane & 3;
    float crow[2], m[2], E[2];  // row factors, bounds, sums
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      crow[n] = __shfl_sync(0xffffffffu, cr, 16 * n + 2 * g);
      E[n] = 0.0f;
      m[n] = 0.0f;
    }
    // a warp whose 16 rows are all past the batch leaves its weights as they are
    const bool idle = base >= nrows;
    bool ok = true;
    int i = 0;
    for (int tile = MT == 2 ? 0 : s; tile < T; tile += MT == 2 ? 1 : 2, ++i) {
      ok = wait(&s_full[s], (uint32_t)i, 0x4101u);
      if (!ok) break;
      if (idle) {
        if (lane == 0) {
          sm100::mbar_arrive(&p_full[s]);
          sm100::mbar_arrive(&t_empty[tile % kTabs]);
        }
        continue;
      }
      sm100::tc_fence_after();
      const int key_left = end - begin - tile * kTile;
      const float4* tb = tab + (tile % kTabs) * 4;
      const uint2* fb = fac + (tile % kTabs) * (kTile / 2) + t4;
      uint32_t v[16];
      tmem_ld_16x256b_x4(ts, v);
#pragma unroll
      for (int c = 0; c < kTile / 32; ++c) {
        // 32 keys share the powers of two 2^x (scale of the keys), 2^y (of the
        // values): t - m = S cr 2^x + (y - m), and E takes 2^(t - m) 2^-y
        const float4 sc = tb[c];
        // (scalar operations: the packed f32x2 forms run on one of the two FMA
        // pipes only, which the fp16 products of the dequantization need as well;
        // with them the largest batch took 342 us instead of 308)
        float2 t[2][4];  // [row][8 columns: this lane's pair]
        uint2 d[4];
        if (kExact)
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = fb[16 * c + 4 * j];
        sm100::tmem_ld_wait();
        if (kExact)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float x = __uint_as_float(v[j]);
            v[j] = __float_as_uint(fmaf(
                x, (j & 1) ? bf16_hi_to_f32(d[j >> 2].x) : bf16_lo_to_f32(d[j >> 2].x), x));
          }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float cf = crow[n] * sc.x, cm = sc.y - m[n];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            t[n][j] = make_float2(fmaf(__uint_as_float(v[4 * j + 2 * n]), cf, cm),
                                  fmaf(__uint_as_float(v[4 * j + 2 * n + 1]), cf, cm));
        }
        if (c + 1 < kTile / 32) tmem_ld_16x256b_x4(ts + 32 * (c + 1), v);
        if (key_left < kTile) {  // the last tile of the prefix: columns without a key
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = 32 * c + 8 * j + t4;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              if (key >= key_left) t[n][j].x = -INFINITY;
              if (key + 4 >= key_left) t[n][j].y = -INFINITY;
            }
          }
        }
        uint32_t w[8];
        float2 e[2];  // [row] sums of even and odd columns
        auto weigh = [&]() {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            e[n] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float w0 = ex2(t[n][j].x), w1 = ex2(t[n][j].y);
              e[n].x += w0;
              e[n].y += w1;
              w[2 * j + n] = kExact ? pack_f16x2(fmaf(w0, bf16_lo_to_f32(d[j].y), w0),
                                                 fmaf(w1, bf16_hi_to_f32(d[j].y), w1))
                                    : pack_f16x2(w0, w1);
            }
          }
        };
        weigh();
        // No weight is above a lane's sums of 4: while those stay below 2^15 they
        // all fit fp16, and no maximum is needed. The first columns set the
        // bound, whatever their scores.
        const bool first = i == 0 && c == 0;
        const float top = fmaxf(fmaxf(e[0].x, e[0].y), fmaxf(e[1].x, e[1].y));
        if (__any_sync(0xffffffffu, first || top > kSumMax)) {
          // a bound moves (in a row's first columns, rarely later): what was
          // summed against the old one is brought down, the weights of this
          // tile's columns before these among it
          float f[2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float mx = kNone, sum = fmaxf(e[n].x, e[n].y);
#pragma unroll
            for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(t[n][j].x, t[n][j].y));
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              sum = fmaxf(sum, __shfl_xor_sync(0xffffffffu, sum, o));
            }
            // a row moves by its own scores only; t is relative to the old bound.
            // Bounds are integers: 2^-up is exact, and so are the products with it
            const float up = first || sum > kSumMax ? rintf(mx) - kLiftTc : 0.0f;
            f[n] = first ? 1.0f : up < 126.0f ? pow2(-(int)up) : 0.0f;
            m[n] += up;
            E[n] *= f[n];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              t[n][j].x -= up;
              t[n][j].y -= up;
            }
          }
          if (i > 0) {
#pragma unroll 1
            for (int k = 0; k < kD / 16; ++k) {
              uint32_t o[8];
              tmem_ld_16x256b_x2(to + 16 * k, o);
              sm100::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 8; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * f[(j >> 1) & 1]);
              tmem_st_16x256b_x2(to + 16 * k, o);
            }
          }
          if (c > 0) {
            sm100::tmem_st_wait();
#pragma unroll 1
            for (int k = 0; k < c; ++k) {
              uint32_t o[8];
              tmem_ld_16x128b_x4(ts + 16 * k, o);
              sm100::tmem_ld_wait();
              // (in fp32: 2^-up is below fp16's range from 2^-25 on, a weight times it not yet)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float2 x = __half22float2(as_h2(o[j]));
                o[j] = pack_f16x2(x.x * f[j & 1], x.y * f[j & 1]);
              }
              tmem_st_16x128b_x4(ts + 16 * k, o);
            }
          }
          weigh();
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) E[n] = fmaf(e[n].x + e[n].y, sc.z, E[n]);
        tmem_st_16x128b_x4(ts + 16 * c, w);  // over columns whose scores were read
      }
      sm100::tmem_st_wait();
      sm100::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        sm100::mbar_arrive(&p_full[s]);
        sm100::mbar_arrive(&t_empty[tile % kTabs]);
      }
    }
    // ---- the rows' partial results
    const int nslot = p.nsp + p.nso;
    const int slot = MT == 2 ? split : 2 * split + s;
    if (ok && i > 0) ok = wait(&o_full[s], 0, 0x4102u);
    if (ok) {
      sm100::tc_fence_after();
      int64_t at[2];
      bool have[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int row = base + 8 * n + g;
        have[n] = row < nrows;
        at[n] = ((int64_t)(row / p.R) * p.Hq + kh * p.R + row % p.R) * nslot + slot;
        float e = E[n];
        e += __shfl_xor_sync(0xffffffffu, e, 1);
        e += __shfl_xor_sync(0xffffffffu, e, 2);
        if (t4 == 0 && have[n]) p.stat[at[n]] = make_float2(i > 0 ? m[n] : kNone, e);
      }
      if (i > 0) {
#pragma unroll
        for (int c = 0; c < kD / 32; ++c) {
          uint32_t v[16];
          tmem_ld_16x256b_x4(to + 32 * c, v);
          sm100::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < 2; ++n)
              if (have[n])
                *reinterpret_cast<uint2*>(p.part + at[n] * kD + 32 * c + 8 * j + 2 * t4) =
                    make_uint2(v[4 * j + 2 * n], v[4 * j + 2 * n + 1]);
        }
      }
    }
  } else if (warp < kSoftWarps + kDeqWarps) {
    // ---------------- keys and values to fp16 ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsDequant));
    const int w = (warp - kSoftWarps) >> 1;       // group of 32 keys
    const int half = (warp - kSoftWarps) & 1;     // of its 16-key halves, this warp's
    const int64_t crow = (int64_t)kh * p.pre.cap, vrow = (int64_t)kh * p.pre.nblk;
    // K: lane = 16-byte piece `piece` of token 8 i + kt of the warp's 16
    const int kt = lane >> 2, piece = lane & 3;
    // token t of 8 sits at row ((t & 3) << 1) | (t >> 2)
    const int krow = ((kt & 3) << 1) | (kt >> 2);
    uint4 kr[2];
    uint32_t vr[8];
    uint32_t cur[4], nxt[4];  // fp16 bits of the group's token `lane`: sk, zk, sv, zv
    // running pointers to this lane's pieces of the tile
    const int key0 = begin + 32 * w;
    const uint32_t* kp = p.pre.kc + (crow + key0 + 16 * half + kt) * (kD / 8) + 4 * piece;
    const uint32_t* vp = p.pre.vc + (vrow + key0 / 8 + 2 * half) * kD + lane;
    const uint16_t* sp4[4];
    {
      const __half* t[4] = {p.pre.ks, p.pre.kz, p.pre.vs, p.pre.vz};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sp4[i] = reinterpret_cast<const uint16_t*>(t[i]) + crow + key0 + lane;
    }
    int left_k = end - key0, left_v = left_k;  // keys from the group's first on
    auto load_k = [&](uint32_t (&sc)[4]) {
      if (left_k >= 32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) kr[i] = ld_stream_u4(kp + 8 * i * (kD / 8));
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = *sp4[i];
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          kr[i] = 16 * half + 8 * i + kt < left_k ? ld_stream_u4(kp + 8 * i * (kD / 8))
                                                  : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = lane < left_k ? *sp4[i] : 0u;
      }
      kp += kTile * (kD / 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) sp4[i] += kTile;
      left_k -= kTile;
    };
    auto load_v = [&]() {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bool in = 16 * half + 8 * j < left_v;
#pragma unroll
        for (int i = 0; i < 4; ++i) vr[4 * j + i] = in ? __ldg(vp + j * kD + 32 * i) : 0u;
      }
      vp += kTile / 8 * kD;
      left_v -= kTile;
    };
    // where this lane's 16-byte pieces go: K's word j of a row (words of the
    // second 64 dimensions in the order 1 0 3 2, so that the 8 lanes of a store
    // phase hit distinct banks), V's block j (row d = 32 i + lane)
    const bool sw = piece >= 2;
    uint32_t koff[4], voff[2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      koff[j] = (uint32_t)((piece >> 1) * kAtomBytes + (32 * w + 16 * half + krow) * 128 +
                           (((4 * (piece & 1) + (j ^ (sw ? 1 : 0))) ^ krow) << 4));
#pragma unroll
    for (int j = 0; j < 2; ++j)
      voff[j] = (uint32_t)((w >> 1) * kAtomBytes + lane * 128 +
                           (((4 * (w & 1) + 2 * half + j) ^ (lane & 7)) << 4));
    if (T > 0) {
      load_k(cur);
      load_v();
    }
    for (int tile = 0; tile < T; ++tile) {
      const int st = tile & 1;
      const uint32_t use = (uint32_t)(tile >> 1);
      if (tile >= 2 && !wait(&k_empty[st], use - 1u, 0x4201u)) break;
      if (tile >= kTabs && !wait(&t_empty[tile % kTabs], (uint32_t)(tile / kTabs) - 1u, 0x4202u))
        break;
      // the 32 keys' scales, K's and V's, times a power of two that brings the
      // largest to [2^10, 2^11): a product with q - z is at most 30705, and stays
      // a normal fp16 number down to scales 2^-24 of the largest
      int kx, vx;
      const uint32_t ks = norm_scale<kExact>(cur[0], kx), vs = norm_scale<kExact>(cur[2], vx);
      if (kExact && half == 0) {
        // token 8 j + t is column pair 4 j + t % 4, its first for t < 4
        uint16_t* at = reinterpret_cast<uint16_t*>(fac + (tile % kTabs) * (kTile / 2) + 16 * w +
                                                   4 * (lane >> 3) + (lane & 3)) +
                       ((lane >> 2) & 1);
        at[0] = bf16_bits(scale_rest(cur[0]));
        at[2] = bf16_bits(scale_rest(cur[2]));
      }
      if (lane == 0 && half == 0)
        tab[(tile % kTabs) * 4 + w] = make_float4(pow2(kx), (float)vx, pow2(-vx), 0.0f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int token = 16 * half + 8 * i + kt;
        const uint32_t s2 = __shfl_sync(0xffffffffu, ks, token) * 0x10001u;
        const uint32_t z = __shfl_sync(0xffffffffu, cur[1], token) * 0x10001u;
        const uint32_t z1 = h2(__hadd2(as_h2(z), as_h2(0x64006400u)));
        const uint32_t z64 = h2(__hneg2(__hadd2(as_h2(z), as_h2(0x54005400u))));
        uint8_t* dst = sk + st * kOpBytes + 8 * i * 128;
        const uint32_t u[4] = {sw ? kr[i].y : kr[i].x, sw ? kr[i].x : kr[i].y,
                               sw ? kr[i].w : kr[i].z, sw ? kr[i].z : kr[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a0, a1, a2, a3;
          codes_f16(u[j], z1, z64, a0, a1);
          codes_f16(u[j] >> 8, z1, z64, a2, a3);
          a0 = mul_f16x2(a0, s2), a1 = mul_f16x2(a1, s2);
          a2 = mul_f16x2(a2, s2), a3 = mul_f16x2(a3, s2);
          *reinterpret_cast<uint4*>(dst + koff[j]) = make_uint4(a0, a1, a2, a3);
        }
      }
      sm100::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && !(wc.stall && tile == 0)) sm100::mbar_arrive(&k_full[st]);
      if (tile + 1 < T) load_k(nxt);
      if (tile >= 2 && !wait(&v_empty[st], use - 1u, 0x4203u)) break;
      // zeros and scales of 8 tokens as the pairs (0, 4), (1, 5), (2, 6), (3, 7):
      // lane 8 j + t holds pair t of block j
      const uint32_t zp =
          prmt(cur[3], __shfl_down_sync(0xffffffffu, cur[3], 4), 0x5410);
      const uint32_t sp = prmt(vs, __shfl_down_sync(0xffffffffu, vs, 4), 0x5410);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = 2 * half + j;  // block of the group
        uint32_t y1[2], y64[2], s2[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) s2[t] = __shfl_sync(0xffffffffu, sp, 8 * b + t);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          y1[t] = h2(__hadd2(as_h2(__shfl_sync(0xffffffffu, zp, 8 * b + 2 * t)),
                             as_h2(0x64006400u)));
          y64[t] = h2(__hneg2(__hadd2(as_h2(__shfl_sync(0xffffffffu, zp, 8 * b + 2 * t + 1)),
                                      as_h2(0x54005400u))));
        }
        uint8_t* dst = sv + st * kOpBytes + voff[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a0, a1, a2, a3;
          codes_f16(vr[4 * j + i], y1[0], y64[0], a0, a1);
          codes_f16(vr[4 * j + i] >> 8, y1[1], y64[1], a2, a3);
          a0 = mul_f16x2(a0, s2[0]), a1 = mul_f16x2(a1, s2[1]);
          a2 = mul_f16x2(a2, s2[2]), a3 = mul_f16x2(a3, s2[3]);
          *reinterpret_cast<uint4*>(dst + 32 * i * 128) = make_uint4(a0, a1, a2, a3);
        }
      }
      sm100::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&v_full[st]);
      if (tile + 1 < T) load_v();
#pragma unroll
      for (int i = 0; i < 4; ++i) cur[i] = nxt[i];
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
  }
  if (warp == kIssueWarp) {
    // ---------------- MMA issue ----------------
    constexpr uint32_t idesc = sm100::idesc_f16_f32(kTile, kTile);
    const uint32_t tm = sm100::uniform(tmem);
    const uint32_t qlo = sm100::uniform(sm100::sdesc_lo(smem_u32(sq)));
    const uint32_t klo = sm100::uniform(sm100::sdesc_lo(smem_u32(sk)));
    const uint32_t vlo = sm100::uniform(sm100::sdesc_lo(smem_u32(sv)));
    auto scores = [&](int s, int st, bool release) {
      if (sm100::elect_one()) {
        const uint32_t a = qlo + (MT == 2 ? s : 0) * (kOpBytes >> 4), b = klo + st * (kOpBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t o = (kk >> 2) * (kAtomBytes >> 4) + (kk & 3) * 2;
          sm100::mma_f16(tm + s * kTile, sm100::sdesc_at(a + o), sm100::sdesc_at(b + o), idesc,
                         kk > 0);
        }
        sm100::mma_commit(&s_full[s]);
        if (release) sm100::mma_commit(&k_empty[st]);
      }
      __syncwarp();
    };
    auto values = [&](int s, int st, bool first, bool release, bool last) {
      if (sm100::elect_one()) {
        const uint32_t b = vlo + st * (kOpBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk) {
          const uint32_t o = (kk >> 2) * (kAtomBytes >> 4) + (kk & 3) * 2;
          sm100::mma_f16_tmem_a(tm + kColO + s * kD, tm + s * kTile + 8 * kk,
                                sm100::sdesc_at(b + o), idesc, !first || kk > 0);
        }
        if (release) sm100::mma_commit(&v_empty[st]);
        if (last) sm100::mma_commit(&o_full[s]);
      }
      __syncwarp();
    };
    bool ok = T > 0 && wait(q_full, 0, 0x4301u);
    if (ok) sm100::tc_fence_after();
    if (MT == 2) {
      if (ok && (ok = wait(&k_full[0], 0, 0x4302u))) {
        sm100::tc_fence_after();
        scores(0, 0, false);
        scores(1, 0, true);
      }
      for (int n = 0; n < T && ok; ++n) {
        const int st = n & 1, st1 = (n + 1) & 1;
        if (!(ok = wait(&v_full[st], (uint32_t)(n >> 1), 0x4303u))) break;
        if (n + 1 < T && !(ok = wait(&k_full[st1], (uint32_t)((n + 1) >> 1), 0x4304u))) break;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!(ok = wait(&p_full[s], (uint32_t)n, 0x4305u))) break;
          sm100::tc_fence_after();
          values(s, st, n == 0, s == 1, n + 1 == T);
          if (n + 1 < T) scores(s, st1, s == 1);
        }
      }
    } else {
      for (int t = 0; t < 2 && t < T && ok; ++t) {
        if (!(ok = wait(&k_full[t], 0, 0x4302u))) break;
        sm100::tc_fence_after();
        scores(t, t, true);
      }
      for (int n = 0; n < T && ok; ++n) {
        const int st = n & 1, s = n & 1;
        if (!(ok = wait(&v_full[st], (uint32_t)(n >> 1), 0x4303u))) break;
        if (!(ok = wait(&p_full[s], (uint32_t)(n >> 1), 0x4305u))) break;
        sm100::tc_fence_after();
        values(s, st, n < 2, true, n + 2 >= T);
        if (n + 2 < T) {
          if (!(ok = wait(&k_full[st], (uint32_t)((n + 2) >> 1), 0x4304u))) break;
          sm100::tc_fence_after();
          scores(s, st, true);
        }
      }
    }
    if (sm100::elect_one()) sm100::mma_commit(mma_done);
    __syncwarp();
  }

  // After an abort: wait (bounded) for the MMAs still in flight.
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) sm100::mbar_wait_drain(mma_done, 0, wc.limit_ns);
    __syncthreads();
  }
  sm100::tc_fence_after();
  if (warp == kIssueWarp) sm100::tmem_dealloc(tmem, 512);
}

template <int MT, bool kExact>
wq_status launch(const PrefixArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> smem_set{0};
  if (!allow_smem(prefix_tc_kernel<MT, kExact>, smem_bytes<MT>(), smem_set)) return WQ_ERR_CUDA;
  return launch_following(prefix_tc_kernel<MT, kExact>, (unsigned)a.nprefix, kThreads,
                          smem_bytes<MT>(), st, a, wait_ctl());
}

}  // namespace

wq_status launch_prefix_tc(const PrefixArgs& a, int row_tiles, cudaStream_t st) {
  if (a.fp16) return row_tiles == 2 ? launch<2, true>(a, st) : launch<1, true>(a, st);
  return row_tiles == 2 ? launch<2, false>(a, st) : launch<1, false>(a, st);
}

wq_status read_prefix_error(bool clear, uint32_t* v) {
  uint32_t h = 0;
  if (cudaMemcpyFromSymbol(&h, g_prefix_error, sizeof(h)) != cudaSuccess) return WQ_ERR_CUDA;
  if (clear && h) {
    const uint32_t z = 0;
    if (cudaMemcpyToSymbol(g_prefix_error, &z, sizeof(z)) != cudaSuccess) return WQ_ERR_CUDA;
  }
  *v = h;
  return WQ_OK;
}

}  // namespace wq
