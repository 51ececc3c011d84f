// Decode attention of a batch whose sequences share a cached prefix: the
// prefix is read once for all of them, and every sequence attends its own
// cached tokens too. Both caches are INT4 (one group per token row).
//
// Per KV head the B * R query rows (R query heads share it) meet the same P
// prefix keys: a dense product whose keys are loaded and dequantized once for
// a tile of rows. Each sequence's own tokens meet its R rows only. Both are
// cut into key ranges that are computed independently (flash decoding), and a
// second kernel merges the partial results of a row.
//
// Mathematics of one range, for a row r and key l:
//   s_l = log2(e) / sqrt(D) sk_l sum_d q_d (qk_ld - zk_l)
//   t_l = s_l + log2(sv_l),  w_l = 2^(t_l - m),  m = a running bound of max t
//   O_d = sum_l w_l (qv_ld - zv_l),  E = sum_l w_l / sv_l
//   out_d = sum_j 2^(m_j - M) O_jd / sum_j 2^(m_j - M) E_j over the ranges j.
// The integers q - z are exact in fp16 and enter the MMAs as they are; the
// key's scale multiplies the fp32 score, the value's scale goes into the
// exponent, so that the fp16 weight w_l <= 2^15 carries it whatever its
// magnitude. q is scaled per row by a power of two into fp16's range (exact
// for elements down to 2^-28 of the row's largest). The only roundings below
// fp32 are w's (2^-11 of w, where w >= 2^-21 of the largest) and the output's.
#include <algorithm>
#include <cmath>

#include "prefix_attn.cuh"

namespace wq {

wq_status launch_prefix_tc(const PrefixArgs& a, int row_tiles, cudaStream_t st);

std::atomic<int> g_prefix_path{0};  // 0: chosen per call, 1: mma.sync, 2: tcgen05

namespace {

using namespace prefix;

constexpr int kWarps = 4;            // warps of a CTA; each takes every 4th step of a range
constexpr int kStep = 32;            // keys of a warp's step
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// A warp's steps (32 keys each) go through a ring of its own in shared memory:
// two steps are in flight by cp.async while one is computed, and nothing but the
// warp itself waits for them. A stage holds 32 K rows of 64 bytes and 4 V blocks
// of 512. Lane (g, t4) reads the K rows of tokens 4 g .. 4 g + 3 (16 bytes of
// each: dimensions 32 t4 ..) and the V words of block t4 (dimensions 32 j + 4 g
// ..): row r is kept at place r ^ (r / 4 % 2), piece q of block t4 at q ^ 2 t4,
// so that the 8 lanes of a phase read distinct banks. The step's scales and
// zeros, which may lie at any 2-byte address, are loaded a step ahead in
// registers (a token a lane) and put beside, V's scale as its logarithm and its
// inverse: worked out once a token instead of by the 4 lanes that use it.
constexpr int kStages = 3;
constexpr int kStageBytes = kStep * kD;                    // codes of 32 keys, K and V
constexpr int kScaleBytes = kStep * 16;  // sk, log2(sv), 1 / sv in fp32, zk, zv in fp16
constexpr int kRingBytes = kWarps * kStages * kStageBytes;

template <int NT>
constexpr int attn_smem() {  // ring, scales (two steps), query fragments, statistics
  return kRingBytes + kWarps * 2 * kScaleBytes + (NT > 1 ? NT * 2048 : 0) + 2 * kWarps * 8 * NT * 4;
}
// the warps' output rows use the ring's space at the end
constexpr int kOutPitch = kD + 4;
static_assert(kWarps * 2 * 8 * kOutPitch * 4 <= kRingBytes, "two groups of 8 rows");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}

// Codes of the step at token l0 < end into a stage (tokens from `end` on: zeros).
// kp and vp are this lane's pieces of the step's first rows and of its first block.
__device__ __forceinline__ void load_codes(uint32_t stage, const uint32_t* kp, const uint32_t* vp,
                                           int l0, int end, int lane) {
  const int r = lane >> 2;
  const uint32_t kd = stage + (uint32_t)((r ^ (r >> 2)) * 64 + 16 * (lane & 3));
  const uint32_t vd = stage + kStep * 64;
  if (l0 + kStep <= end) {
#pragma unroll
    for (int i = 0; i < 4; ++i) cp_async16(kd + 512 * i, kp + 8 * i * (kD / 8), true);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      cp_async16(vd + i * 512 + ((lane ^ (2 * i)) << 4), vp + i * kD, true);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = l0 + 8 * i + r < end;
      cp_async16(kd + 512 * i, in ? kp + 8 * i * (kD / 8) : kp - r * (kD / 8), in);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = l0 + 8 * i < end;
      cp_async16(vd + i * 512 + ((lane ^ (2 * i)) << 4), in ? vp + i * kD : vp, in);
    }
  }
}

// The lane's token of the step at l0: sk, zk, sv, zv as bits (from `end` on: 1 and 0);
// and the same put into shared memory.
__device__ __forceinline__ void load_scales(uint16_t (&s)[4], const Cache& c, int64_t crow0, int l0,
                                            int end, int lane) {
  const bool in = l0 + lane < end;
  const int64_t at = crow0 + l0 + lane;
  s[0] = in ? reinterpret_cast<const uint16_t*>(c.ks)[at] : (uint16_t)0x3C00u;
  s[1] = in ? reinterpret_cast<const uint16_t*>(c.kz)[at] : (uint16_t)0;
  s[2] = in ? reinterpret_cast<const uint16_t*>(c.vs)[at] : (uint16_t)0x3C00u;
  s[3] = in ? reinterpret_cast<const uint16_t*>(c.vz)[at] : (uint16_t)0;
}

__device__ __forceinline__ void store_scales(uint8_t* dst, const uint16_t (&s)[4], int lane) {
  auto value = [](uint16_t b) { return __half2float(__ushort_as_half(b)); };
  float* f = reinterpret_cast<float*>(dst) + lane;
  const float l = __log2f(fmaxf(value(s[2]), 5.9604645e-8f));  // fp16's smallest: 0 has no log
  f[0] = value(s[0]);
  f[kStep] = l;
  f[2 * kStep] = ex2(-l);
  uint16_t* z = reinterpret_cast<uint16_t*>(dst + 12 * kStep) + lane;
  z[0] = s[1];
  z[kStep] = s[3];
}

// The query rows row0 + n (n < nrows, at most 8 NT) of KV head kh against keys
// [begin, end) of one cache; the result goes to each row's slot.
template <int NT>
__device__ __forceinline__ void attend(const PrefixArgs& p, const Cache& c, int64_t crow0,
                                       int64_t vrow0, int kh, int row0, int nrows, int begin,
                                       int end, int slot, uint8_t* sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = smem_u32(sm) + (uint32_t)(warp * kStages * kStageBytes);
  const uint8_t* ring_p = sm + warp * kStages * kStageBytes;
  uint8_t* scl = sm + kRingBytes + warp * 2 * kScaleBytes;
  uint2* qsm = reinterpret_cast<uint2*>(sm + kRingBytes + kWarps * 2 * kScaleBytes);
  float* msm = reinterpret_cast<float*>(sm + kRingBytes + kWarps * 2 * kScaleBytes +
                                        (NT > 1 ? NT * 2048 : 0));  // [warps][8 NT] m, then E
  constexpr int kStride = kWarps * kStep;
  int l0 = begin + warp * kStep;
  uint16_t sc4[4];
  // (a piece of the next step to load: in the cache, or where no step is left not used)
  const uint32_t* kp = c.kc + (crow0 + l0 + (lane >> 2)) * (kD / 8) + 4 * (lane & 3);
  const uint32_t* vp = c.vc + (vrow0 + (l0 >> 3)) * kD + 4 * lane;
  auto next_codes = [&](int stage, int at) {
    load_codes(ring + (uint32_t)stage * kStageBytes, kp, vp, at, end, lane);
    kp += kStride * (kD / 8);
    vp += kStride / 8 * kD;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (l0 + s * kStride < end) next_codes(s, l0 + s * kStride);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  if (l0 < end) {
    load_scales(sc4, c, crow0, l0, end, lane);
    store_scales(scl, sc4, lane);
    if (l0 + kStride < end) load_scales(sc4, c, crow0, l0 + kStride, end, lane);
  }

  // Query fragments (B operand, column n = row): dimensions 32 t4 + 8 j + ..
  // in the order of the code words' nibbles. The row's power of two goes to
  // the score factor of rows 2 t4 and 2 t4 + 1, the accumulator's columns.
  // Eight rows stay in registers; more are read again at every step.
  constexpr bool kQSmem = NT > 1;
  uint32_t bq[kQSmem ? 1 : 8][2];
  float cr[NT][2];
  for (int nt = 0; nt < NT; ++nt) {
    const int n = 8 * nt + g;
    float f[32];
    float amax = 0.0f;
    if (n < nrows) {
      const int row = row0 + n;
      const int64_t off = (int64_t)(row / p.R) * p.q_stride +
                          (int64_t)(kh * p.R + row % p.R) * kD + 32 * t4;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + off);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = src[i];
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (p.fp16) {
            const float2 t = __half22float2(as_h2(u[j]));
            f[8 * i + 2 * j] = t.x;
            f[8 * i + 2 * j + 1] = t.y;
          } else {
            f[8 * i + 2 * j] = bf16_lo_to_f32(u[j]);
            f[8 * i + 2 * j + 1] = bf16_hi_to_f32(u[j]);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) f[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(f[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    float up, down;
    row_scale(amax, up, down);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t b[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          b[h] = pack_f16x2(f[8 * j + 2 * e + h] * up, f[8 * j + 2 * e + h + 4] * up);
        if (kQSmem) {
          // every warp has the same fragments: one of them writes
          if (warp == nt % kWarps) qsm[(nt * 8 + 2 * j + e) * 32 + lane] = make_uint2(b[0], b[1]);
        } else {
          bq[kQSmem ? 0 : 2 * j + e][0] = b[0];
          bq[kQSmem ? 0 : 2 * j + e][1] = b[1];
        }
      }
    const float fac = down * kScoreScale;
    const float c0 = __shfl_sync(0xffffffffu, fac, (2 * t4) * 4);
    const float c1 = __shfl_sync(0xffffffffu, fac, (2 * t4 + 1) * 4);
#pragma unroll
    for (int i = 0; i < NT; ++i)
      if (i == nt) cr[i][0] = c0, cr[i][1] = c1;
  }
  if (kQSmem) __syncthreads();

  float O[NT][8][4];
  float m[NT][2], E[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) O[nt][i][r] = 0.0f;
    m[nt][0] = m[nt][1] = kNone;
    E[nt][0] = E[nt][1] = 0.0f;
  }

  for (int k = 0; l0 < end; l0 += kStride, ++k) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();  // the step is complete, and the stage of the step before is read
    if (l0 + (kStages - 1) * kStride < end)
      next_codes((k + kStages - 1) % kStages, l0 + (kStages - 1) * kStride);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (l0 + kStride < end) {
      store_scales(scl + ((k + 1) & 1) * kScaleBytes, sc4, lane);
      if (l0 + 2 * kStride < end) load_scales(sc4, c, crow0, l0 + 2 * kStride, end, lane);
    }
    const uint8_t* stage = ring_p + (k % kStages) * kStageBytes;
    const uint8_t* sp = scl + (k & 1) * kScaleBytes;
    const uint2 szk = *reinterpret_cast<const uint2*>(sp + 12 * kStep + 8 * g);
    const uint4 szv = *reinterpret_cast<const uint4*>(sp + 14 * kStep + 16 * t4);
    // ---- scores: S^T tile s holds tokens 4 g + 2 s (rows g) and + 1 (rows
    // g + 8) against the query rows 2 t4, 2 t4 + 1
    float sc[NT][2][4];
    const uint32_t zk2[4] = {prmt(szk.x, 0, 0x1010), prmt(szk.x, 0, 0x3232),
                             prmt(szk.y, 0, 0x1010), prmt(szk.y, 0, 0x3232)};
    uint32_t z1[4], z64[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z1[i] = h2(__hadd2(as_h2(zk2[i]), as_h2(0x64006400u)));
      z64[i] = h2(__hneg2(__hadd2(as_h2(zk2[i]), as_h2(0x54005400u))));
    }
    const float4 skf = *reinterpret_cast<const float4*>(sp + 16 * g);
    const float4 lsv = *reinterpret_cast<const float4*>(sp + 4 * kStep + 16 * g);
    const float4 rsv = *reinterpret_cast<const float4*>(sp + 8 * kStep + 16 * g);
    const float sk4[4] = {skf.x, skf.y, skf.z, skf.w}, lv4[4] = {lsv.x, lsv.y, lsv.z, lsv.w},
                rv4[4] = {rsv.x, rsv.y, rsv.z, rsv.w};
    uint32_t y1[2], y64[2];  // k-step s: zeros of tokens (2s, 2s + 4), and (2s + 1, 2s + 5)
    y1[0] = h2(__hadd2(as_h2(prmt(szv.x, szv.z, 0x5410)), as_h2(0x64006400u)));
    y1[1] = h2(__hadd2(as_h2(prmt(szv.y, szv.w, 0x5410)), as_h2(0x64006400u)));
    y64[0] = h2(__hneg2(__hadd2(as_h2(prmt(szv.x, szv.z, 0x7632)), as_h2(0x54005400u))));
    y64[1] = h2(__hneg2(__hadd2(as_h2(prmt(szv.y, szv.w, 0x7632)), as_h2(0x54005400u))));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) sc[nt][s][r] = 0.0f;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint4 ra = *reinterpret_cast<const uint4*>(
          stage + ((4 * g + 2 * s) ^ (g & 1)) * 64 + 16 * t4);
      const uint4 rb = *reinterpret_cast<const uint4*>(
          stage + ((4 * g + 2 * s + 1) ^ (g & 1)) * 64 + 16 * t4);
      const uint32_t ka[4] = {ra.x, ra.y, ra.z, ra.w}, kb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t a0, a1, a2, a3;
          codes_f16(e ? ka[j] >> 8 : ka[j], z1[2 * s], z64[2 * s], a0, a2);
          codes_f16(e ? kb[j] >> 8 : kb[j], z1[2 * s + 1], z64[2 * s + 1], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint2 q;
            if (kQSmem)
              q = qsm[(nt * 8 + 2 * j + e) * 32 + lane];
            else
              q = make_uint2(bq[kQSmem ? 0 : 2 * j + e][0], bq[kQSmem ? 0 : 2 * j + e][1]);
            mma16816(sc[nt][s], a0, a1, a2, a3, q.x, q.y);
          }
        }
    }
    // ---- weights
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 2 * s + (r >> 1);  // token 4 g + i
          sc[nt][s][r] = fmaf(sc[nt][s][r] * cr[nt][r & 1], sk4[i], lv4[i]);
        }
    if (l0 + kStep > end) {
      const int left = end - (l0 + 4 * g);  // this lane's tokens i < left exist
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (2 * s + (r >> 1) >= left) sc[nt][s][r] = -INFINITY;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float top = fmaxf(fmaxf(sc[nt][0][x], sc[nt][0][2 + x]),
                                fmaxf(sc[nt][1][x], sc[nt][1][2 + x]));
        grow |= top > m[nt][x] + kSlack;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = fmaxf(fmaxf(sc[nt][0][x], sc[nt][0][2 + x]),
                           fmaxf(sc[nt][1][x], sc[nt][1][2 + x]));
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          // a row moves by its own scores only, whatever rows share its tile
          const float nm = mx > m[nt][x] + kSlack ? mx - kLift : m[nt][x];
          const float f = ex2(m[nt][x] - nm);
          m[nt][x] = nm;
          E[nt][x] *= f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            O[nt][i][x] *= f;
            O[nt][i][2 + x] *= f;
          }
        }
    }
    uint32_t bp[NT][2][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          w[r] = ex2(sc[nt][s][r] - m[nt][r & 1]);
          E[nt][r & 1] = fmaf(w[r], rv4[2 * s + (r >> 1)], E[nt][r & 1]);
        }
        bp[nt][s][0] = transpose8x8(pack_f16x2(w[0], w[1]));
        bp[nt][s][1] = transpose8x8(pack_f16x2(w[2], w[3]));
      }
    // ---- values
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 rv = *reinterpret_cast<const uint4*>(
          stage + kStep * 64 + t4 * 512 + (((8 * j + g) ^ (2 * t4)) << 4));
      const uint32_t vw[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t a0, a1, a2, a3;
          codes_f16(s ? vw[2 * e] >> 8 : vw[2 * e], y1[s], y64[s], a0, a2);
          codes_f16(s ? vw[2 * e + 1] >> 8 : vw[2 * e + 1], y1[s], y64[s], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(O[nt][2 * j + e], a0, a1, a2, a3, bp[nt][s][0], bp[nt][s][1]);
        }
    }
  }

  // ---- the warps' results: E over the lanes of a column, then O and E over
  // the warps against their common bound
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();                                  // the rings are read: their space is free
  float* osm = reinterpret_cast<float*>(sm);        // [warps][8 NT rows][kOutPitch]
  float* esm = msm + kWarps * 8 * NT;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1)
        E[nt][x] += __shfl_xor_sync(0xffffffffu, E[nt][x], o);
      if (g == 0) {
        msm[warp * 8 * NT + 8 * nt + 2 * t4 + x] = m[nt][x];
        esm[warp * 8 * NT + 8 * nt + 2 * t4 + x] = E[nt][x];
      }
    }
  __syncthreads();
  float f[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float big = kNone;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) big = fmaxf(big, msm[w * 8 * NT + 8 * nt + 2 * t4 + x]);
      f[nt][x] = ex2(m[nt][x] - big);
    }
  // each warp puts its rows down, then the warps' parts are added in order
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = 32 * (i >> 1) + 4 * g + 2 * (i & 1) + (r >> 1);
        osm[(warp * 8 * NT + 8 * nt + 2 * t4 + (r & 1)) * kOutPitch + d] =
            O[nt][i][r] * f[nt][r & 1];
      }
  __syncthreads();
  const int nslot = p.nsp + p.nso;
  for (int n = warp; n < nrows; n += kWarps) {
    const int row = row0 + n;
    const int64_t at = ((int64_t)(row / p.R) * p.Hq + kh * p.R + row % p.R) * nslot + slot;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x =
          *reinterpret_cast<const float4*>(osm + (w * 8 * NT + n) * kOutPitch + 4 * lane);
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    *reinterpret_cast<float4*>(p.part + at * kD + 4 * lane) = v;
    if (lane == 0) {
      float big = kNone, e = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) big = fmaxf(big, msm[w * 8 * NT + n]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        e = fmaf(ex2(msm[w * 8 * NT + n] - big), esm[w * 8 * NT + n], e);
      p.stat[at] = make_float2(big, e);
    }
  }
}

__device__ __forceinline__ int own_length(const PrefixArgs& p, int b) {
  return min(max(p.lengths[b], 0), (int)p.own.cap);
}

// CTAs 0 .. nprefix - 1: key range x row tile x KV head of the prefix (none
// where the tcgen05 kernel takes it: nprefix is 0 here); the rest: key range x
// KV head x sequence of the own tokens. Bound by its instructions, about 640 a
// warp's step of 32 keys, half of them dequantization: 64 sequences x 8 heads x 8
// rows on 2000 to 2048 own tokens take 43 us (141 MB of cache, issue 51%, HBM 42%).
// With few keys its latency is what counts: 4 chats on 1021 shared keys 7.8 us with
// the merge. Launched while the tcgen05 kernel still runs, whose results the merge
// needs too: every CTA ends by waiting for it. Without that kernel it is the call's
// first and waits at once (ends_waiting false).
template <int NTP, int NTO>
__global__ void __launch_bounds__(32 * kWarps, NTP * NTO == 1 ? 4 : 2)
    prefix_attn_kernel(const __grid_constant__ PrefixArgs p, int nprefix, bool ends_waiting) {
  extern __shared__ __align__(16) uint8_t sm[];
  if (ends_waiting)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  else
    follow_previous();
  int i = blockIdx.x;
  if (i < nprefix) {
    const int ranges = p.nsp;
    const int slot = i % ranges;
    const int rt = (i / ranges) % p.nrt;
    const int kh = i / (ranges * p.nrt);
    const int begin = slot * p.chunk_p;
    attend<NTP>(p, p.pre, kh * p.pre.cap, kh * p.pre.nblk, kh, rt * 8 * NTP,
                min(8 * NTP, p.B * p.R - rt * 8 * NTP), begin, min(begin + p.chunk_p, p.P), slot,
                sm);
  } else {
    i -= nprefix;
    const int range = i % p.nso;
    const int kh = (i / p.nso) % p.Hkv;
    const int b = i / (p.nso * p.Hkv);
    const int len = own_length(p, b);
    const int begin = range * p.chunk_o;
    const int64_t bh = (int64_t)b * p.Hkv + kh;
    if (begin < len)
      attend<NTO>(p, p.own, bh * p.own.cap, bh * p.own.nblk, kh, b * p.R, p.R, begin,
                  min(begin + p.chunk_o, len), p.nsp + range, sm);
  }
  if (ends_waiting) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The ranges' partial results of a row against their common bound. W warps a
// row, each a run of the ranges: 4 where there are many ranges (a single warp
// that walked 30 to 60 of them one by one took 12 us), one where there are few
// and the rows fill the GPU. A lane takes one range's statistics, and four
// partial rows are in flight at once.
constexpr int kMergeWarps = 4;
template <int W>
__global__ void __launch_bounds__(32 * kMergeWarps)
    prefix_merge_kernel(const __grid_constant__ PrefixArgs p) {
  __shared__ float4 acc[kMergeWarps][32];
  __shared__ float2 top[kMergeWarps];  // (bound, E) of each warp's ranges
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * (kMergeWarps / W) + warp / W, part = warp % W;
  const bool have = row < p.B * p.Hq;
  const int n = have ? p.nsp + (own_length(p, row / p.Hq) + p.chunk_o - 1) / p.chunk_o : 0;
  const int64_t base = (int64_t)row * (p.nsp + p.nso);
  const int run = (n + W - 1) / W;
  const int end = min((part + 1) * run, n);
  follow_previous();
  float m = kNone, e = 0.0f;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j0 = part * run; j0 < end; j0 += 32) {
    const int cnt = min(32, end - j0);
    // a range without keys wrote (kNone, 0) and no partial row
    const float2 st = lane < cnt ? p.stat[base + j0 + lane] : make_float2(kNone, 0.0f);
    const float* src = p.part + (base + j0) * kD + 4 * lane;
    float big = fmaxf(m, st.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    const float f = st.y == 0.0f ? 0.0f : ex2(st.x - big);
    const float old = ex2(m - big);
    m = big;
    e = fmaf(e, old, f * st.y);  // per lane, summed at the end
    a.x *= old, a.y *= old, a.z *= old, a.w *= old;
    for (int j = 0; j < cnt; j += 4) {
      float4 v[4];
      float g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = __shfl_sync(0xffffffffu, f, (j + i) & 31);
        g[i] = j + i < cnt ? w : 0.0f;
        v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (g[i] != 0.0f) v[i] = *reinterpret_cast<const float4*>(src + (int64_t)(j + i) * kD);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a.x = fmaf(g[i], v[i].x, a.x);
        a.y = fmaf(g[i], v[i].y, a.y);
        a.z = fmaf(g[i], v[i].z, a.z);
        a.w = fmaf(g[i], v[i].w, a.w);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
  if (W > 1) {
    acc[warp][lane] = a;
    if (lane == 0) top[warp] = make_float2(m, e);
    __syncthreads();
    if (part != 0) return;
    float big = kNone;
#pragma unroll
    for (int w = 0; w < W; ++w) big = fmaxf(big, top[warp + w].x);
    a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    e = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = ex2(top[warp + w].x - big);
      const float4 v = acc[warp + w][lane];
      e = fmaf(f, top[warp + w].y, e);
      a.x = fmaf(f, v.x, a.x);
      a.y = fmaf(f, v.y, a.y);
      a.z = fmaf(f, v.z, a.z);
      a.w = fmaf(f, v.w, a.w);
    }
  }
  if (!have) return;
  const float inv = n > 0 ? 1.0f / e : 0.0f;  // a row with no key at all: zeros
  const float x[4] = {a.x * inv, a.y * inv, a.z * inv, a.w * inv};
  uint2 o;
  if (p.fp16)
    o = make_uint2(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]));
  else
    o = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (int64_t)row * kD + 4 * lane) = o;
}

// Which kernel takes the prefix. On mma.sync the time grows with 16-row groups
// times keys (45 ps each, the GPU full), on tcgen05 with row tiles times keys
// (114 ps a key for 128 rows, 145 for 256) from about 10 us more. 8 KV heads,
// mma.sync against tcgen05: 64 rows 14 and 16 us at 4096 keys, 29 and 27 at
// 16384; 256 rows 21 and 24 us at 2048, 30 and 27 at 4096, 91 and 42 at 16384;
// 32 rows 19 and 26 us at 16384, 48 and 69 at 65536, never the other way.
bool prefix_on_tc(int64_t Hkv, int64_t rows, int64_t P, int tiles, int groups_of_tiles) {
  const int64_t gain = 45 * ((rows + 15) / 16) - (tiles == 2 ? 145 : 114) * groups_of_tiles;
  return gain > 0 && Hkv * P > 10000000 / gain;
}

// How a problem is cut: the same for the workspace query and the launch.
struct Plan {
  int tc;   // row tiles of a tcgen05 CTA (1 or 2), or 0: the prefix on mma.sync
  int ntp;  // 8-row groups of a prefix row tile on mma.sync
  int nto;  // of a sequence's own rows
  int nrt, chunk_p, ranges, nsp, chunk_o, nso;
};

Plan make_plan(int64_t B, int64_t Hq, int64_t Hkv, int64_t P, int64_t cap) {
  Plan pl;
  const int64_t R = Hq / Hkv, rows = B * R, sms = num_sms();
  const int64_t step = kWarps * kStep;
  auto cut = [&](int64_t keys, int64_t others, int64_t want, int& chunk, int& n) {
    const int64_t ranges =
        std::max<int64_t>(1, std::min<int64_t>((keys + step - 1) / step, want / others));
    chunk = (int)(((keys + ranges - 1) / ranges + step - 1) / step * step);
    n = (int)((keys + chunk - 1) / chunk);
  };
  pl.nto = R <= 8 ? 1 : 2;
  pl.ntp = 1;
  int64_t wave = pl.nto == 1 ? 4 * sms : 2 * sms;  // CTAs that fit at once
  pl.tc = 0;
  pl.nsp = pl.ranges = 0;
  pl.nrt = 0;
  pl.chunk_p = 128;
  const int64_t rt = (rows + 127) / 128;
  const int per = rt >= 2 ? 2 : 1;
  const int64_t rg = (rt + per - 1) / per;
  const int path = g_prefix_path.load(std::memory_order_relaxed);
  if (P > 0 && (path == 2 || (path == 0 && prefix_on_tc(Hkv, rows, P, per, (int)rg)))) {
    // tcgen05: the ranges that give the slowest SM the least work, a CTA's
    // start and end counted as 4 tiles
    const int64_t tiles = (P + 127) / 128;
    pl.tc = per;
    pl.nrt = (int)rg;
    // (about two waves at most; 2^24 units fill any number of SMs with one range)
    const uint32_t units = (uint32_t)std::min<int64_t>(Hkv * pl.nrt, 1 << 24);
    uint64_t best = UINT64_MAX;
    const uint32_t most = (uint32_t)std::min<int64_t>(
        tiles, std::max<uint32_t>(8, 2 * (uint32_t)sms / units + 1));
    for (uint32_t n = 1; n <= most; ++n) {
      const uint32_t waves = (units * n + (uint32_t)sms - 1) / (uint32_t)sms;
      const uint32_t run = ((uint32_t)tiles + n - 1) / n;
      const uint64_t cost = (uint64_t)waves * (run + 4);
      if (cost < best) {
        best = cost;
        pl.chunk_p = (int)run * 128;
      }
    }
    pl.ranges = (int)((P + pl.chunk_p - 1) / pl.chunk_p);
    pl.nsp = pl.tc == 1 ? 2 * pl.ranges : pl.ranges;
  } else if (P > 0) {
    // 16 rows share a key's loads, at half the warps; where the sequences' own
    // tokens are most of the work they run better beside 8 rows (64 sequences
    // x 8 heads, 512 own tokens, 128 shared: 18.4 us, 21.4 with 16 rows; 128
    // own, 1024 shared: 23.7 with 16 rows)
    pl.ntp = rows <= 8 || (R <= 8 && B * cap > (rows + 15) / 16 * P) ? 1 : 2;
    wave = pl.ntp * pl.nto == 1 ? 4 * sms : 2 * sms;
    pl.nrt = (int)((rows + 8 * pl.ntp - 1) / (8 * pl.ntp));
    cut(P, std::max<int64_t>(1, Hkv * pl.nrt), wave, pl.chunk_p, pl.ranges);
    pl.nsp = pl.ranges;
  }
  // own tokens: two waves, as lengths differ, unless a row then has more than 20
  // ranges to merge (8 KV heads: 64 sequences of 10 to 2048 tokens 36 us with one
  // wave, 32 with two, 32 with three; of 2000 to 2048 44, 44 and 48; two of 8192
  // tokens 12 us with 37 ranges, 15 with 64)
  const int64_t own = std::max<int64_t>(1, B * Hkv);
  cut(cap, own, std::max(wave, std::min(2 * wave, 20 * own)), pl.chunk_o, pl.nso);
  return pl;
}

template <int NTP, int NTO>
wq_status launch(const PrefixArgs& a, int tc, cudaStream_t st) {
  if (tc) {
    const wq_status s = launch_prefix_tc(a, tc, st);
    if (s != WQ_OK) return s;
  }
  const int nprefix = tc ? 0 : a.nprefix;
  constexpr int kSmem = attn_smem<(NTP > NTO ? NTP : NTO)>();
  static std::atomic<uint64_t> smem_set{0};
  if (!allow_smem(prefix_attn_kernel<NTP, NTO>, kSmem, smem_set)) return WQ_ERR_CUDA;
  const wq_status s = launch_following(prefix_attn_kernel<NTP, NTO>,
                                       (unsigned)(nprefix + (int64_t)a.nso * a.Hkv * a.B),
                                       32 * kWarps, kSmem, st, a, nprefix, tc != 0);
  if (s != WQ_OK) return s;
  const int64_t rows = (int64_t)a.B * a.Hq;
  const int warps = a.nsp + a.nso <= 12 ? 1 : kMergeWarps;
  return launch_following(warps == 1 ? prefix_merge_kernel<1> : prefix_merge_kernel<kMergeWarps>,
                          (unsigned)((rows * warps + kMergeWarps - 1) / kMergeWarps),
                          32 * kMergeWarps, 0, st, a);
}

template <int NTO>
wq_status launch_o(const PrefixArgs& a, const Plan& pl, cudaStream_t st) {
  // (R > 8 has more than 8 rows: a prefix on mma.sync then takes two groups)
  if (NTO == 1 && pl.ntp == 1) return launch<1, 1>(a, pl.tc, st);
  return launch<2, NTO>(a, pl.tc, st);
}

}  // namespace

static size_t plan_bytes(const Plan& pl, int64_t B, int64_t Hq) {
  return (size_t)B * Hq * (pl.nsp + pl.nso) * (kD * 4 + 8);
}

size_t prefix_attn_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t P, int64_t cap) {
  return plan_bytes(make_plan(B, Hq, Hkv, P, cap), B, Hq);
}

wq_status launch_prefix_attn(const void* q, wq_dtype dt, int64_t q_stride, int64_t B, int64_t Hq,
                             int64_t Hkv, int64_t P, int64_t pre_cap, const void* const* pre,
                             int64_t cap, const void* const* own, const int32_t* lengths,
                             void* out, void* workspace, size_t ws_bytes, cudaStream_t st) {
  const Plan pl = make_plan(B, Hq, Hkv, P, cap);
  if (!workspace || ws_bytes < plan_bytes(pl, B, Hq)) return WQ_ERR_WORKSPACE;
  if (!aligned16(workspace)) return WQ_ERR_ALIGNMENT;
  PrefixArgs a;
  a.q = q;
  a.q_stride = q_stride;
  a.fp16 = dt == WQ_FP16;
  a.B = (int)B;
  a.Hq = (int)Hq;
  a.Hkv = (int)Hkv;
  a.R = (int)(Hq / Hkv);
  auto cache = [](const void* const* c, int64_t n) {
    return Cache{static_cast<const uint32_t*>(c[0]), static_cast<const __half*>(c[1]),
                 static_cast<const __half*>(c[2]),   static_cast<const uint32_t*>(c[3]),
                 static_cast<const __half*>(c[4]),   static_cast<const __half*>(c[5]),
                 n,                                  (n + 7) / 8};
  };
  a.pre = cache(pre, pre_cap);
  a.own = cache(own, cap);
  a.P = (int)P;
  a.lengths = lengths;
  a.chunk_p = pl.chunk_p;
  a.nsp = pl.nsp;
  a.chunk_o = pl.chunk_o;
  a.nso = pl.nso;
  a.nrt = pl.nrt;
  a.nprefix = (int)(Hkv * pl.nrt * pl.ranges);
  a.part = static_cast<float*>(workspace);
  a.stat = reinterpret_cast<float2*>(a.part + (size_t)B * Hq * (pl.nsp + pl.nso) * kD);
  a.out = out;
  return pl.nto == 1 ? launch_o<1>(a, pl, st) : launch_o<2>(a, pl, st);
}

}  // namespace wq
