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
//   softmax        a warp takes 32 rows
//   O += P V       A = the weights in tensor memory
// Roles: warps 0-3 and 4-7 softmax of stream 0 and 1, warps 8-11 dequantize
// keys and values into shared memory (two stages each), warp 12 issues.
// Within a group of 8 dimensions (K) or keys (V) the nibbles of a code word
// come out as pairs (0, 4), (1, 5), (2, 6), (3, 7): Q's dimensions and the rows
// of K (hence the columns of S and P) are stored in that order, 0 4 1 5 2 6 3 7.
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
constexpr int kThreads = 13 * 32;
constexpr int kOpBytes = kTile * kD * 2;   // an operand tile: two 64-element atoms of 16 KB
constexpr int kAtomBytes = kOpBytes / 2;
constexpr int kTabs = 4;                   // key-table stages
constexpr uint32_t kHalf = 16u << 16;      // the upper 16 lanes of a warp's quarter of TMEM
constexpr int kColO = 256;                 // TMEM columns of the outputs (scores: 0 and 128)

template <int MT>
constexpr int smem_bytes() {
  return 1024 + (MT + 4) * kOpBytes + kTabs * 3 * kTile * 4 + 256;
}

__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_get(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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

template <int MT>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ PrefixArgs p, const WaitCtl wc) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint8_t* sq = smem;                          // [row tile]
  uint8_t* sk = sq + MT * kOpBytes;            // [stage]
  uint8_t* sv = sk + 2 * kOpBytes;             // [stage]
  // [stage] per column pair (sk, sk, log2 sv, log2 sv), then 1 / sv per column
  float* tab = reinterpret_cast<float*>(sv + 2 * kOpBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(tab + kTabs * 3 * kTile);
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this CTA's KV head, row tiles and keys
  const int splits = MT == 2 ? p.nsp : p.nsp / 2;
  const int split = blockIdx.x % splits;
  const int rg = (blockIdx.x / splits) % p.nrt;  // group of MT row tiles
  const int kh = blockIdx.x / (splits * p.nrt);
  const int begin = split * p.chunk_p;
  const int end = min(begin + p.chunk_p, p.P);
  const int T = (end - begin + kTile - 1) / kTile;

  if (threadIdx.x == 0) {
    sm100::mbar_init(q_full, 4 * MT);
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&k_full[i], 4);
      sm100::mbar_init(&k_empty[i], 1);
      sm100::mbar_init(&v_full[i], 4);
      sm100::mbar_init(&v_empty[i], 1);
      sm100::mbar_init(&s_full[i], 1);
      sm100::mbar_init(&p_full[i], 4);
      sm100::mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < kTabs; ++i) sm100::mbar_init(&t_empty[i], 4 * MT);
    sm100::mbar_init(mma_done, 1);
    *abort_flag = 0;
    sm100::fence_mbar_init();
  }
  if (warp == 12) {
    sm100::tmem_alloc(tmem_slot, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
    return __all_sync(0xffffffffu, sm100::mbar_wait(bar, parity & 1u, &g_prefix_error, site,
                                                    abort_flag, wc.limit_ns));
  };

  if (warp < 8) {
    // ---------------- softmax: warp = 32 rows ----------------
    const int s = warp >> 2, q = warp & 3;
    const int r = 32 * q + lane;
    const int row = (MT == 2 ? 2 * rg + s : rg) * kTile + r;
    const bool have = row < p.B * p.R;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    float up = 1.0f, cr = 0.0f;
    {
      // the row of Q as fp16 times a power of two; rows past the batch are zeros
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(p.q) +
          (have ? (int64_t)(row / p.R) * p.q_stride + (int64_t)(kh * p.R + row % p.R) * kD : 0));
      auto values = [&](int j, float (&f)[8]) {
        const uint4 v = have ? src[j] : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
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
      float amax = 0.0f, down;
#pragma unroll 4
      for (int j = 0; j < kD / 8; ++j) {
        float f[8];
        values(j, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
      }
      row_scale(amax, up, down);
      cr = down * kScoreScale;
      if (MT == 2 || s == 0) {
        uint8_t* dst = sq + s * kOpBytes + r * 128;
#pragma unroll 4
        for (int j = 0; j < kD / 8; ++j) {
          float f[8];
          values(j, f);
          *reinterpret_cast<uint4*>(dst + (j >> 3) * kAtomBytes + (((j & 7) ^ (r & 7)) << 4)) =
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
    // lane (g, t4) holds columns 8 j + 2 t4 and + 1 of rows 8 n + g, n = 0 .. 3.
    // A thread meets a quarter of the columns and takes their table entries for
    // 4 rows at once: read by one row a thread, 12 bytes a column and lane
    // filled the shared-memory pipe twice as long as the MMAs run.
    const int g = lane >> 2, t4 = lane & 3;
    uint64_t cr2[4], E2[4], mm[4];  // row factors, sums of even and odd columns, minus the bounds
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float c = __shfl_sync(0xffffffffu, cr, 8 * n + g);
      cr2[n] = f2(c, c);
      E2[n] = 0;
      mm[n] = f2(-kNone, -kNone);
    }
    bool ok = true;
    int i = 0;
    for (int tile = MT == 2 ? 0 : s; tile < T; tile += MT == 2 ? 1 : 2, ++i) {
      ok = wait(&s_full[s], (uint32_t)i, 0x4101u);
      if (!ok) break;
      sm100::tc_fence_after();
      const float* tb = tab + (tile % kTabs) * 3 * kTile + 4 * t4;
      const float* rb = tab + (tile % kTabs) * 3 * kTile + 2 * kTile + 2 * t4;
#pragma unroll
      for (int c = 0; c < kTile / 32; ++c) {
        uint32_t v[2][16];
        tmem_ld_16x256b_x4(ts + 32 * c, v[0]);
        tmem_ld_16x256b_x4(ts + kHalf + 32 * c, v[1]);
        sm100::tmem_ld_wait();
        uint64_t t[4][4];  // [row][8 columns: this lane's pair]
        float mx[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(tb + 64 * c + 16 * j);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint32_t* u = v[n >> 1] + 4 * j + 2 * (n & 1);
            t[n][j] = f2_fma(f2_mul(f2(__uint_as_float(u[0]), __uint_as_float(u[1])), cr2[n]), a.x,
                             a.y);
            const float2 x = f2_get(t[n][j]);
            mx[n] = fmaxf(mx[n], fmaxf(x.x, x.y));
          }
        }
        bool grow = false;
#pragma unroll
        for (int n = 0; n < 4; ++n) grow |= mx[n] > kSlack - f2_get(mm[n]).x;
        if (__any_sync(0xffffffffu, grow)) {
          // a bound moves (in a row's first columns, rarely later): what was
          // summed against the old one is brought down, the weights of this
          // tile's columns before these among it
          float f[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xffffffffu, mx[n], 1));
            mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xffffffffu, mx[n], 2));
            const float m = -f2_get(mm[n]).x;
            // a row moves by its own scores only
            const float nm = mx[n] > m + kSlack ? mx[n] : m;
            f[n] = ex2(m - nm);
            mm[n] = f2(-nm, -nm);
            E2[n] = f2_mul(E2[n], f2(f[n], f[n]));
          }
          if (i > 0) {
#pragma unroll 1
            for (int k = 0; k < 2 * (kD / 32); ++k) {
              const int h = k & 1;
              uint32_t o[16];
              tmem_ld_16x256b_x4(to + (h ? kHalf : 0) + 32 * (k >> 1), o);
              sm100::tmem_ld_wait();
              const float f0 = h ? f[2] : f[0], f1 = h ? f[3] : f[1];
#pragma unroll
              for (int j = 0; j < 16; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * (((j >> 1) & 1) ? f1 : f0));
              tmem_st_16x256b_x4(to + (h ? kHalf : 0) + 32 * (k >> 1), o);
            }
          }
          if (c > 0) {
            sm100::tmem_st_wait();
#pragma unroll 1
            for (int k = 0; k < 2 * c; ++k) {
              const int h = k & 1;
              const uint32_t at = ts + (h ? kHalf : 0) + 16 * (k >> 1);
              uint32_t o[8];
              tmem_ld_16x128b_x4(at, o);
              sm100::tmem_ld_wait();
              const __half2 f0 = __float2half2_rn(h ? f[2] : f[0]);
              const __half2 f1 = __float2half2_rn(h ? f[3] : f[1]);
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] = h2(__hmul2(as_h2(o[j]), (j & 1) ? f1 : f0));
              tmem_st_16x128b_x4(at, o);
            }
          }
        }
        uint32_t w[2][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t d = *reinterpret_cast<const uint64_t*>(rb + 32 * c + 8 * j);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float2 y = f2_get(f2_add(t[n][j], mm[n]));
            const float w0 = ex2(y.x), w1 = ex2(y.y);
            E2[n] = f2_fma(f2(w0, w1), d, E2[n]);
            w[n >> 1][2 * j + (n & 1)] = pack_f16x2(w0, w1);
          }
        }
        // over columns whose scores were read
        tmem_st_16x128b_x4(ts + 16 * c, w[0]);
        tmem_st_16x128b_x4(ts + kHalf + 16 * c, w[1]);
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
      auto place = [&](int rr) {
        return ((int64_t)(rr / p.R) * p.Hq + kh * p.R + rr % p.R) * nslot + slot;
      };
      const int64_t at = have ? place(row) : 0;
      if (i > 0) {
#pragma unroll
        for (int c = 0; c < kD / 32; ++c) {
          uint32_t v[32];
          sm100::tmem_ld32(to + 32 * c, v);
          sm100::tmem_ld_wait();
          if (have)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(p.part + at * kD + 32 * c + 4 * j) =
                  make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float2 x = f2_get(E2[n]);
        float e = x.x + x.y;
        e += __shfl_xor_sync(0xffffffffu, e, 1);
        e += __shfl_xor_sync(0xffffffffu, e, 2);
        const int rr = row - lane + 8 * n + g;
        if (t4 == 0 && rr < p.B * p.R) p.stat[place(rr)] = make_float2(-f2_get(mm[n]).x, e);
      }
    }
  } else if (warp < 12) {
    // ---------------- keys and values to fp16 integers ----------------
    const int w = warp - 8;
    const int64_t crow = (int64_t)kh * p.pre.cap, vrow = (int64_t)kh * p.pre.nblk;
    // K: lane = 16-byte piece `piece` of token 8 i + kt of the warp's 32
    const int kt = lane >> 2, piece = lane & 3;
    // token t of 8 sits at row ((t & 3) << 1) | (t >> 2)
    const int krow = ((kt & 3) << 1) | (kt >> 2);
    const int pos = 32 * w + (lane & 24) + (((lane & 3) << 1) | ((lane >> 2) & 1));
    uint4 kr[4];
    uint32_t vr[16];
    uint32_t cur[4], nxt[4];  // fp16 bits of this lane's token: sk, zk, sv, zv
    auto load_k = [&](int tile, uint32_t (&sc)[4]) {
      const int key0 = begin + tile * kTile + 32 * w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + 8 * i + kt;
        kr[i] = key < end ? ld_stream_u4(p.pre.kc + (crow + key) * (kD / 8) + 4 * piece)
                          : make_uint4(0, 0, 0, 0);
      }
      const int key = key0 + lane;
      const bool in = key < end;
      const __half* t[4] = {p.pre.ks, p.pre.kz, p.pre.vs, p.pre.vz};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sc[i] = in ? reinterpret_cast<const uint16_t*>(t[i])[crow + key] : 0u;
    };
    auto load_v = [&](int tile) {
      const int blk0 = (begin + tile * kTile) / 8 + 4 * w;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vr[4 * j + i] =
              8 * (blk0 + j) < end
                  ? __ldg(p.pre.vc + (vrow + blk0 + j) * kD + 32 * i + lane)
                  : 0u;
    };
    if (T > 0) {
      load_k(0, cur);
      load_v(0);
    }
    for (int tile = 0; tile < T; ++tile) {
      const int st = tile & 1;
      const uint32_t use = (uint32_t)(tile >> 1);
      if (tile >= 2 && !wait(&k_empty[st], use - 1u, 0x4201u)) break;
      if (tile >= kTabs && !wait(&t_empty[tile % kTabs], (uint32_t)(tile / kTabs) - 1u, 0x4202u))
        break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t z = __shfl_sync(0xffffffffu, cur[1], 8 * i + kt) * 0x10001u;
        const uint32_t z1 = h2(__hadd2(as_h2(z), as_h2(0x64006400u)));
        const uint32_t z64 = h2(__hneg2(__hadd2(as_h2(z), as_h2(0x54005400u))));
        const int row = 32 * w + 8 * i + krow;
        uint8_t* dst = sk + st * kOpBytes + (piece >> 1) * kAtomBytes + row * 128;
        // pieces of the second 64 dimensions take their words in the order
        // 1 0 3 2: the 8 lanes of a store phase then hit distinct banks
        const bool sw = piece >= 2;
        const uint32_t u[4] = {sw ? kr[i].y : kr[i].x, sw ? kr[i].x : kr[i].y,
                               sw ? kr[i].w : kr[i].z, sw ? kr[i].z : kr[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a0, a1, a2, a3;
          codes_f16(u[j], z1, z64, a0, a1);
          codes_f16(u[j] >> 8, z1, z64, a2, a3);
          const int chunk = 4 * (piece & 1) + (j ^ (sw ? 1 : 0));
          *reinterpret_cast<uint4*>(dst + ((chunk ^ (row & 7)) << 4)) = make_uint4(a0, a1, a2, a3);
        }
      }
      {
        // per key: sk, log2 sv, 1 / sv; keys past the end weigh 2^-inf
        const bool in = begin + tile * kTile + 32 * w + lane < end;
        float* tb = tab + (tile % kTabs) * 3 * kTile;
        const float x = fmaxf(__half2float(__ushort_as_half((unsigned short)cur[2])),
                              5.9604645e-8f);  // fp16's smallest: a scale of 0 has no log
        const float l = __log2f(x);
        tb[4 * (pos >> 1) + (pos & 1)] = __half2float(__ushort_as_half((unsigned short)cur[0]));
        tb[4 * (pos >> 1) + 2 + (pos & 1)] = in ? l : -INFINITY;
        tb[2 * kTile + pos] = in ? ex2(-l) : 0.0f;
      }
      sm100::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && !(wc.stall && tile == 0)) sm100::mbar_arrive(&k_full[st]);
      if (tile + 1 < T) load_k(tile + 1, nxt);
      if (tile >= 2 && !wait(&v_empty[st], use - 1u, 0x4203u)) break;
      // zeros of 8 tokens as the pairs (0, 4), (1, 5), (2, 6), (3, 7): lane
      // 8 j + t holds pair t of block j
      const uint32_t zp =
          prmt(cur[3], __shfl_down_sync(0xffffffffu, cur[3], 4), 0x5410);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t y1[2], y64[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          y1[t] = h2(__hadd2(as_h2(__shfl_sync(0xffffffffu, zp, 8 * j + 2 * t)),
                             as_h2(0x64006400u)));
          y64[t] = h2(__hneg2(__hadd2(as_h2(__shfl_sync(0xffffffffu, zp, 8 * j + 2 * t + 1)),
                                      as_h2(0x54005400u))));
        }
        const int chunk = 4 * (w & 1) + j;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = 32 * i + lane;
          uint32_t a0, a1, a2, a3;
          codes_f16(vr[4 * j + i], y1[0], y64[0], a0, a1);
          codes_f16(vr[4 * j + i] >> 8, y1[1], y64[1], a2, a3);
          *reinterpret_cast<uint4*>(sv + st * kOpBytes + (w >> 1) * kAtomBytes + d * 128 +
                                    ((chunk ^ (d & 7)) << 4)) = make_uint4(a0, a1, a2, a3);
        }
      }
      sm100::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&v_full[st]);
      if (tile + 1 < T) load_v(tile + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) cur[i] = nxt[i];
    }
  } else {
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
  if (warp == 12) sm100::tmem_dealloc(tmem, 512);
}

template <int MT>
wq_status launch(const PrefixArgs& a, cudaStream_t st) {
  static bool attr_set = [] {
    return cudaFuncSetAttribute(prefix_tc_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                smem_bytes<MT>()) == cudaSuccess;
  }();
  if (!attr_set) return WQ_ERR_CUDA;
  prefix_tc_kernel<MT><<<(unsigned)a.nprefix, kThreads, smem_bytes<MT>(), st>>>(a, wait_ctl());
  return launch_status();
}

}  // namespace

wq_status launch_prefix_tc(const PrefixArgs& a, int row_tiles, cudaStream_t st) {
  return row_tiles == 2 ? launch<2>(a, st) : launch<1>(a, st);
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
