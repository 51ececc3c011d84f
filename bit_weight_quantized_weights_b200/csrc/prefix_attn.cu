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
// exponent, so that the fp16 weight w_l <= 2^8 carries it whatever its
// magnitude. q is scaled per row by a power of two into fp16's range (exact
// for elements down to 2^-28 of the row's largest). The only roundings below
// fp32 are w's (2^-11 of w, where w >= 2^-14 of the largest) and the output's.
#include <algorithm>
#include <cmath>

#include "prefix_attn.cuh"

namespace wq {

wq_status launch_prefix_tc(const PrefixArgs& a, int row_tiles, cudaStream_t st);

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

// One step's 32 keys as they come from memory. Lane (g, t4) holds the K rows
// of tokens 4 g .. 4 g + 3 (16 bytes of each: dimensions 32 t4 ..), the V
// words of block t4 (dimensions 32 j + 4 g ..), and the scales of its tokens.
struct Raw {
  uint4 k[4], v[4];
  uint2 sk, zk, sv, zv;  // 4 fp16 each
};

__device__ __forceinline__ uint2 load4(const __half* p, int64_t at, int n, bool vec, uint32_t pad) {
  if (vec) return *reinterpret_cast<const uint2*>(p + at);
  const uint16_t* u = reinterpret_cast<const uint16_t*>(p) + at;
  const uint32_t a = n > 0 ? u[0] : pad, b = n > 1 ? u[1] : pad;
  const uint32_t c = n > 2 ? u[2] : pad, d = n > 3 ? u[3] : pad;
  return make_uint2(a | (b << 16), c | (d << 16));
}

// Step at token l0 of the cache row block that starts at row0 (V: vrow0);
// tokens from `end` on give zero codes, scale 1 and zero 0.
__device__ __forceinline__ void load_step(Raw& w, const Cache& c, int64_t row0, int64_t vrow0,
                                          int l0, int end, int g, int t4, bool vec4) {
  const int tok = l0 + 4 * g;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w.k[i] = tok + i < end ? ld_stream_u4(c.kc + (row0 + tok + i) * (kD / 8) + 4 * t4)
                           : make_uint4(0, 0, 0, 0);
  const int blk = (l0 >> 3) + t4;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w.v[j] = 8 * blk < end ? ld_stream_u4(c.vc + (vrow0 + blk) * kD + 32 * j + 4 * g)
                           : make_uint4(0, 0, 0, 0);
  const bool vec = vec4 && l0 + kStep <= end;
  const int n = end - tok;
  w.sk = load4(c.ks, row0 + tok, n, vec, 0x3C00u);
  w.zk = load4(c.kz, row0 + tok, n, vec, 0u);
  w.sv = load4(c.vs, row0 + tok, n, vec, 0x3C00u);
  w.zv = load4(c.vz, row0 + tok, n, vec, 0u);
}

// The query rows row0 + n (n < nrows, at most 8 NT) of KV head kh against keys
// [begin, end) of one cache; the result goes to each row's slot.
template <int NT>
__device__ __forceinline__ void attend(const PrefixArgs& p, const Cache& c, int64_t crow0,
                                       int64_t vrow0, int kh, int row0, int nrows, int begin,
                                       int end, int slot, float* sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const bool vec4 = (crow0 & 3) == 0;

  Raw cur;
  int l0 = begin + warp * kStep;
  if (l0 < end) load_step(cur, c, crow0, vrow0, l0, end, g, t4, vec4);

  // Query fragments (B operand, column n = row): dimensions 32 t4 + 8 j + ..
  // in the order of the code words' nibbles. The row's power of two goes to
  // the score factor of rows 2 t4 and 2 t4 + 1, the accumulator's columns.
  uint32_t bq[NT][8][2];
  float cr[NT][2];
#pragma unroll
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
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          bq[nt][2 * j + e][b] = pack_f16x2(f[8 * j + 2 * e + b] * up, f[8 * j + 2 * e + b + 4] * up);
    const float fac = down * kScoreScale;
    cr[nt][0] = __shfl_sync(0xffffffffu, fac, (2 * t4) * 4);
    cr[nt][1] = __shfl_sync(0xffffffffu, fac, (2 * t4 + 1) * 4);
  }

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

  for (; l0 < end; l0 += kWarps * kStep) {
    // ---- scores: S^T tile s holds tokens 4 g + 2 s (rows g) and + 1 (rows
    // g + 8) against the query rows 2 t4, 2 t4 + 1
    float sc[NT][2][4];
    const uint32_t zk2[4] = {prmt(cur.zk.x, 0, 0x1010), prmt(cur.zk.x, 0, 0x3232),
                             prmt(cur.zk.y, 0, 0x1010), prmt(cur.zk.y, 0, 0x3232)};
    uint32_t z1[4], z64[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z1[i] = h2(__hadd2(as_h2(zk2[i]), as_h2(0x64006400u)));
      z64[i] = h2(__hneg2(__hadd2(as_h2(zk2[i]), as_h2(0x54005400u))));
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) sc[nt][s][r] = 0.0f;
      const uint32_t ka[4] = {cur.k[2 * s].x, cur.k[2 * s].y, cur.k[2 * s].z, cur.k[2 * s].w};
      const uint32_t kb[4] = {cur.k[2 * s + 1].x, cur.k[2 * s + 1].y, cur.k[2 * s + 1].z,
                              cur.k[2 * s + 1].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t a0, a1, a2, a3;
          codes_f16(e ? ka[j] >> 8 : ka[j], z1[2 * s], z64[2 * s], a0, a2);
          codes_f16(e ? kb[j] >> 8 : kb[j], z1[2 * s + 1], z64[2 * s + 1], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(sc[nt][s], a0, a1, a2, a3, bq[nt][2 * j + e][0], bq[nt][2 * j + e][1]);
        }
    }
    // ---- weights
    float skf[4], lsv[4], rsv[4];
    {
      const float2 s01 = __half22float2(as_h2(cur.sk.x)), s23 = __half22float2(as_h2(cur.sk.y));
      const float2 v01 = __half22float2(as_h2(cur.sv.x)), v23 = __half22float2(as_h2(cur.sv.y));
      skf[0] = s01.x, skf[1] = s01.y, skf[2] = s23.x, skf[3] = s23.y;
      const float v[4] = {v01.x, v01.y, v23.x, v23.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = fmaxf(v[i], 5.9604645e-8f);  // fp16's smallest: a scale of 0 has no log
        lsv[i] = __log2f(x);
        rsv[i] = ex2(-lsv[i]);
      }
    }
    const int left = end - (l0 + 4 * g);  // this lane's tokens i < left exist
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 2 * s + (r >> 1);  // token 4 g + i
          const float t = fmaf(sc[nt][s][r] * cr[nt][r & 1], skf[i], lsv[i]);
          sc[nt][s][r] = i < left ? t : -INFINITY;
          grow |= sc[nt][s][r] > m[nt][r & 1] + kSlack;
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
          const float nm = mx > m[nt][x] + kSlack ? mx : m[nt][x];
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
          E[nt][r & 1] = fmaf(w[r], rsv[2 * s + (r >> 1)], E[nt][r & 1]);
        }
        bp[nt][s][0] = transpose8x8(pack_f16x2(w[0], w[1]));
        bp[nt][s][1] = transpose8x8(pack_f16x2(w[2], w[3]));
      }
    // ---- values: zeros of block t4's tokens come from lanes g = 2 t4, 2 t4 + 1
    uint32_t y1[2], y64[2];  // k-step s: tokens (2s, 2s + 4), and (2s + 1, 2s + 5)
    {
      const uint32_t ax = __shfl_sync(0xffffffffu, cur.zv.x, 8 * t4);
      const uint32_t ay = __shfl_sync(0xffffffffu, cur.zv.y, 8 * t4);
      const uint32_t bx = __shfl_sync(0xffffffffu, cur.zv.x, 8 * t4 + 4);
      const uint32_t by = __shfl_sync(0xffffffffu, cur.zv.y, 8 * t4 + 4);
      y1[0] = h2(__hadd2(as_h2(prmt(ax, bx, 0x5410)), as_h2(0x64006400u)));
      y1[1] = h2(__hadd2(as_h2(prmt(ay, by, 0x5410)), as_h2(0x64006400u)));
      y64[0] = h2(__hneg2(__hadd2(as_h2(prmt(ax, bx, 0x7632)), as_h2(0x54005400u))));
      y64[1] = h2(__hneg2(__hadd2(as_h2(prmt(ay, by, 0x7632)), as_h2(0x54005400u))));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t vw[4] = {cur.v[j].x, cur.v[j].y, cur.v[j].z, cur.v[j].w};
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
    if (l0 + kWarps * kStep < end)
      load_step(cur, c, crow0, vrow0, l0 + kWarps * kStep, end, g, t4, vec4);
  }

  // ---- the warps' results: E over the lanes of a column, then O and E over
  // the warps against their common bound
  float* osm = sm;                                  // [8 NT rows][128 + 4]
  float* msm = sm + 8 * NT * (kD + 4);              // [warps][8 NT] m, then E
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
  // the warps add up in order, so that the sum does not depend on their timing
  for (int w = 0; w < kWarps; ++w) {
    if (warp == w) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = 32 * (i >> 1) + 4 * g + 2 * (i & 1) + (r >> 1);
            float* at = osm + (8 * nt + 2 * t4 + (r & 1)) * (kD + 4) + d;
            const float v = O[nt][i][r] * f[nt][r & 1];
            *at = w == 0 ? v : *at + v;
          }
    }
    __syncthreads();
  }
  const int nslot = p.nsp + p.nso;
  for (int n = warp; n < nrows; n += kWarps) {
    const int row = row0 + n;
    const int64_t at = ((int64_t)(row / p.R) * p.Hq + kh * p.R + row % p.R) * nslot + slot;
    *reinterpret_cast<float4*>(p.part + at * kD + 4 * lane) =
        *reinterpret_cast<const float4*>(osm + n * (kD + 4) + 4 * lane);
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
// KV head x sequence of the own tokens. Launched while the tcgen05 kernel still
// runs, whose results the merge needs too: every CTA ends by waiting for it.
template <int NT>
__global__ void __launch_bounds__(32 * kWarps)
    prefix_attn_kernel(const __grid_constant__ PrefixArgs p, int nprefix) {
  __shared__ __align__(16) float sm[8 * NT * (kD + 4) + 2 * kWarps * 8 * NT];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int i = blockIdx.x;
  if (i < nprefix) {
    const int slot = i % p.nsp;
    const int rt = (i / p.nsp) % p.nrt;
    const int kh = i / (p.nsp * p.nrt);
    const int begin = slot * p.chunk_p;
    attend<NT>(p, p.pre, kh * p.pre.cap, kh * p.pre.nblk, kh, rt * 8 * NT,
               min(8 * NT, p.B * p.R - rt * 8 * NT), begin, min(begin + p.chunk_p, p.P), slot, sm);
  } else {
    i -= nprefix;
    const int range = i % p.nso;
    const int kh = (i / p.nso) % p.Hkv;
    const int b = i / (p.nso * p.Hkv);
    const int len = own_length(p, b);
    const int begin = range * p.chunk_o;
    const int64_t bh = (int64_t)b * p.Hkv + kh;
    if (begin < len)
      attend<NT>(p, p.own, bh * p.own.cap, bh * p.own.nblk, kh, b * p.R, p.R, begin,
                 min(begin + p.chunk_o, len), p.nsp + range, sm);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One warp a row: the ranges' partial results against their common bound.
__global__ void __launch_bounds__(128) prefix_merge_kernel(const __grid_constant__ PrefixArgs p) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= p.B * p.Hq) return;
  const int b = row / p.Hq;
  const int n = p.nsp + (own_length(p, b) + p.chunk_o - 1) / p.chunk_o;
  const int64_t base = (int64_t)row * (p.nsp + p.nso);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float big = kNone;
  for (int j = lane; j < n; j += 32) big = fmaxf(big, p.stat[base + j].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float e = 0.0f;
  for (int j = 0; j < n; ++j) {
    const float2 st = p.stat[base + j];
    if (st.y == 0.0f) continue;  // a range without keys wrote no partial result
    const float f = ex2(st.x - big);
    const float4 v = *reinterpret_cast<const float4*>(p.part + (base + j) * kD + 4 * lane);
    a.x = fmaf(f, v.x, a.x);
    a.y = fmaf(f, v.y, a.y);
    a.z = fmaf(f, v.z, a.z);
    a.w = fmaf(f, v.w, a.w);
    e = fmaf(f, st.y, e);
  }
  const float inv = n > 0 ? 1.0f / e : 0.0f;  // a row with no key at all: zeros
  const float x[4] = {a.x * inv, a.y * inv, a.z * inv, a.w * inv};
  uint2 o;
  if (p.fp16)
    o = make_uint2(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]));
  else
    o = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (int64_t)row * kD + 4 * lane) = o;
}

// How a problem is cut: the same for the workspace query and the launch.
struct Plan {
  int tc;  // row tiles of a tcgen05 CTA (1 or 2), or 0: the prefix on mma.sync
  int nt, nrt, chunk_p, ranges, nsp, chunk_o, nso;
};

Plan make_plan(int64_t B, int64_t Hq, int64_t Hkv, int64_t P, int64_t cap) {
  Plan pl;
  const int64_t R = Hq / Hkv, rows = B * R, sms = num_sms();
  const int64_t step = kWarps * kStep;
  const int64_t want = sms * 4;  // CTAs: four of a wave's fit an SM
  auto cut = [&](int64_t keys, int64_t others, int& chunk, int& n) {
    const int64_t ranges =
        std::max<int64_t>(1, std::min<int64_t>((keys + step - 1) / step, want / others));
    chunk = (int)(((keys + ranges - 1) / ranges + step - 1) / step * step);
    n = (int)((keys + chunk - 1) / chunk);
  };
  pl.nt = R <= 8 ? 1 : 2;
  pl.tc = 0;
  pl.nsp = pl.ranges = 0;
  pl.nrt = 0;
  pl.chunk_p = 128;
  if (P > 0 && rows > 16) {
    // tcgen05: the ranges that give the slowest SM the least work, a CTA's
    // start and end counted as 4 tiles
    const int64_t tiles = (P + 127) / 128, rt = (rows + 127) / 128;
    pl.tc = rt >= 2 ? 2 : 1;
    pl.nrt = (int)((rt + pl.tc - 1) / pl.tc);
    int64_t best = INT64_MAX;
    for (int64_t n = 1; n <= std::min<int64_t>(tiles, 64); ++n) {
      const int64_t waves = (Hkv * pl.nrt * n + sms - 1) / sms;
      const int64_t cost = waves * ((tiles + n - 1) / n + 4);
      if (cost < best) {
        best = cost;
        pl.chunk_p = (int)((tiles + n - 1) / n) * 128;
      }
    }
    pl.ranges = (int)((P + pl.chunk_p - 1) / pl.chunk_p);
    pl.nsp = pl.tc == 1 ? 2 * pl.ranges : pl.ranges;
  } else if (P > 0) {
    pl.nrt = (int)((rows + 8 * pl.nt - 1) / (8 * pl.nt));
    cut(P, std::max<int64_t>(1, Hkv * pl.nrt), pl.chunk_p, pl.ranges);
    pl.nsp = pl.ranges;
  }
  cut(cap, std::max<int64_t>(1, B * Hkv), pl.chunk_o, pl.nso);
  return pl;
}

template <int NT>
wq_status launch(const PrefixArgs& a, int tc, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.stream = st;
  if (tc) {
    wq_status s = launch_prefix_tc(a, tc, st);
    if (s != WQ_OK) return s;
    cfg.numAttrs = 1;
  }
  const int nprefix = tc ? 0 : a.nprefix;
  cfg.gridDim = dim3((unsigned)(nprefix + (int64_t)a.nso * a.Hkv * a.B), 1, 1);
  cfg.blockDim = dim3(32 * kWarps, 1, 1);
  if (cudaLaunchKernelEx(&cfg, prefix_attn_kernel<NT>, a, nprefix) != cudaSuccess)
    return WQ_ERR_CUDA;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(((int64_t)a.B * a.Hq + 3) / 4), 1, 1);
  cfg.blockDim = dim3(128, 1, 1);
  if (cudaLaunchKernelEx(&cfg, prefix_merge_kernel, a) != cudaSuccess) return WQ_ERR_CUDA;
  return launch_status();
}

}  // namespace

size_t prefix_attn_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t P, int64_t cap) {
  const Plan pl = make_plan(B, Hq, Hkv, P, cap);
  return (size_t)B * Hq * (pl.nsp + pl.nso) * (kD * 4 + 8);
}

wq_status launch_prefix_attn(const void* q, wq_dtype dt, int64_t q_stride, int64_t B, int64_t Hq,
                             int64_t Hkv, int64_t P, int64_t pre_cap, const void* const* pre,
                             int64_t cap, const void* const* own, const int32_t* lengths,
                             void* out, void* workspace, cudaStream_t st) {
  const Plan pl = make_plan(B, Hq, Hkv, P, cap);
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
  return pl.nt == 1 ? launch<1>(a, pl.tc, st) : launch<2>(a, pl.tc, st);
}

}  // namespace wq
