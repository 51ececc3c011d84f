// Writing new tokens into an INT4 KV cache and reading rows of it back.
//
// The cache is the one wq_msd_decode_attention reads, with room for `cap`
// tokens a sequence: one INT4 asymmetric group per (sequence, head, token) row,
//   s = fp16(fp32(max(0, max x) - min(0, min x)) / 15)  ([-1, 1] if that is 0),
//   z = clamp(rint(-min(0, min x) / s), 0, 15), q = clamp(rint(x / s) + z, 0, 15),
// K codes a token a row (uint32 [B, Hkv, cap, 16]), V codes in blocks of 8
// tokens (uint32 [B, Hkv, ceil(cap / 8), 128]: token t of dimension d in
// nibble t % 8). A row read back is RN((q - z) s); (q - z) s is exact in fp32.
//
// Both kernels stream rows once: per row of 128 elements the append reads 256 B
// (16-bit types) and writes 68 B, the read-back the reverse. The read is bound by
// HBM (127315 tokens x 8 heads, bf16: 660 MB in 110 us, 91% of a copy's rate; fp32:
// 1.18 GB in 236 us, 76%), the append by its instructions, about 1020 a warp for 16
// rows, and the latency of its loads (issue 58%, 2.8 waves of CTAs; 12891 tokens x 8
// heads: 67 MB in 16.0 us, 64% of a copy's rate; fp32 rows: 120 MB in 24.0 us, 76%).
// The unit of work is one V block, 8 cache positions of one (sequence, head), taken by
// one warp: 16 lanes hold a row (8 elements a lane, one 16-byte access), the two halves
// of the warp hold two rows, four steps
// cover the block. So a V word has one writer (no atomics; the nibbles of
// positions that are not written are read and put back), a K word is the 8
// elements of one lane, and the group's minimum and maximum take 4 shuffles.
// The warps of a CTA take neighbouring heads, whose rows lie side by side in
// the packed [T, Hkv, D] tensors.
//
// Sequences are packed: offsets[b] .. offsets[b + 1] are sequence b's tokens,
// starts[b] the cache position of the first. A sequence of n tokens touches
// at most floor((n + 14) / 8) blocks, so giving it the unit numbers from
// offsets[b] / 8 + 2 b on never overlaps the next one's, and a warp finds its
// sequence by a 32-way search in `offsets` without any prefix sum. Every
// position is checked against the capacity and every token against T on the
// device, whatever the two arrays hold.
#include "common.cuh"

namespace wq {
namespace {

constexpr int kD = 128;
// Warps of a CTA and CTAs an SM: the warps share nothing, and with small CTAs an
// SM takes new work the sooner (127315 tokens x 8 heads read: 124 us with 8 x 4,
// 114 with 2 x 18). The read runs 2 x 20 (48 registers a thread): 110 us, 118
// with 2 x 18, 111 with 4 x 10; 12891 tokens 13.0 us, 12.8 with 2 x 18, 14.0 with
// 2 x 24. The append needs 64 registers (17.9 us for 12891 tokens with 2 x 16,
// 18.9 with 2 x 18).
constexpr unsigned kWarps = 2;

struct KvRows {            // packed rows and where they belong
  const int32_t* starts;   // [B]
  const int32_t* offsets;  // [B + 1]
  int64_t T;
  int64_t cap;
  int64_t units;           // T / 8 + 2 B
  int64_t kts, khs, vts, vhs;  // token and head strides of the rows (elements)
  int B, H;
  int nblk;                // ceil(cap / 8)
};

// What a warp works on: block `blk` of sequence b and, for its lane's half,
// the token index of each of its 4 rows (-1: not written or read).
struct Unit {
  int b;
  int64_t blk;
  int64_t tok[4];
  bool any;
};

// 32-way search for the last b in [0, B) whose first unit offsets[b] / 8 + 2 b
// is at most u (0 if there is none). The last round loads what the found
// sequence needs with its keys, so that up to 32 sequences take one round of
// loads in all.
__device__ __forceinline__ Unit find_unit(const KvRows& p, int64_t u, int half, int lane,
                                          bool clip) {
  int lo = 0, n = p.B;
  while (n > 32) {
    const int step = (n + 31) >> 5;
    const int i = lane * step;
    const bool in = i < n;
    const int64_t first = in ? (int64_t)(p.offsets[lo + i] >> 3) + 2 * (int64_t)(lo + i) : 0;
    const int cnt = __popc(__ballot_sync(0xffffffffu, in && first <= u));
    const int skip = (cnt > 0 ? cnt - 1 : 0) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  const bool in = lane < n;
  const int32_t o0 = in ? p.offsets[lo + lane] : 0, o1 = in ? p.offsets[lo + lane + 1] : 0;
  const int32_t s0 = in ? p.starts[lo + lane] : 0;
  const int cnt = __popc(__ballot_sync(
      0xffffffffu, in && (int64_t)(o0 >> 3) + 2 * (int64_t)(lo + lane) <= u));
  const int at = cnt > 0 ? cnt - 1 : 0;
  Unit w;
  w.b = lo + at;
  const int64_t t0 = __shfl_sync(0xffffffffu, o0, at), t1 = __shfl_sync(0xffffffffu, o1, at);
  const int64_t first = __shfl_sync(0xffffffffu, s0, at);
  const int64_t local = u - ((t0 >> 3) + 2 * (int64_t)w.b);
  w.blk = (first >> 3) + local;
  w.any = local >= 0 && 8 * w.blk < first + (t1 - t0);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t pos = 8 * w.blk + 2 * r + half;
    const int64_t t = t0 + pos - first;
    const bool ok = w.any && pos >= first && t < t1 && t >= 0 && t < p.T &&
                    (!clip || (pos >= 0 && pos < p.cap));
    w.tok[r] = ok ? t : -1;
  }
  return w;
}

template <typename T>
struct Row;  // 8 consecutive elements of a row
template <>
struct Row<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = ld_stream_u4(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo_to_f32(w[i]);
      f[2 * i + 1] = bf16_hi_to_f32(w[i]);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    st_stream_u4(p, make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
  }
};
template <>
struct Row<__half> {
  uint4 v;
  __device__ __forceinline__ void load(const __half* p) { v = ld_stream_u4(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ void store(__half* p, const float (&f)[8]) {
    st_stream_u4(p, make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]),
                               pack_f16x2(f[4], f[5]), pack_f16x2(f[6], f[7])));
  }
};
template <>
struct Row<float> {
  uint4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = ld_stream_u4(p);
    b = ld_stream_u4(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    st_stream_u4(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                               __float_as_uint(f[2]), __float_as_uint(f[3])));
    st_stream_u4(p + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]),
                                   __float_as_uint(f[6]), __float_as_uint(f[7])));
  }
};

// a / b rounded to nearest from y = RN(1 / b): one correction step on the
// product a y (Markstein's theorem, with the residual a - b q exact in a fused
// multiply-add). Where a quotient underflows the result is still below 1/2 in
// magnitude, which is all its rounding to an integer needs.
__device__ __forceinline__ float div_by(float a, float b, float y) {
  const float q = a * y;
  return __fmaf_rn(__fmaf_rn(-q, b, a), y, q);
}

// min(0, min x) and max(0, max x) of a row: 16 lanes x 8 elements. 16-bit types
// keep (min, -max) packed in one register: a packed minimum and a shuffle a step.
__device__ __forceinline__ void row_range(const Row<float>& r, float& lo, float& hi) {
  float f[8];
  r.get(f);
  lo = hi = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, f[i]);
    hi = fmaxf(hi, f[i]);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
}
template <typename P>  // a packed pair type
__device__ __forceinline__ P min2(P a, P b) { return __hmin2(a, b); }
template <typename P, typename T>
__device__ __forceinline__ uint32_t packed_range(const Row<T>& r) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
  auto as = [](uint32_t u) { return *reinterpret_cast<P*>(&u); };
  auto bits = [](P v) { return *reinterpret_cast<uint32_t*>(&v); };
  constexpr uint32_t kNeg = 0x80008000u;
  const P n = min2(min2(as(w[0]), as(w[1])), min2(as(w[2]), as(w[3])));
  const P x = __hmax2(__hmax2(as(w[0]), as(w[1])), __hmax2(as(w[2]), as(w[3])));
  const uint32_t y = bits(x) ^ kNeg;
  P m = min2(as(prmt(bits(n), y, 0x5410)), as(prmt(bits(n), y, 0x7632)));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
    m = min2(m, as(__shfl_xor_sync(0xffffffffu, bits(m), o)));
  return bits(m);
}
__device__ __forceinline__ void row_range(const Row<__nv_bfloat16>& r, float& lo, float& hi) {
  const uint32_t m = packed_range<__nv_bfloat162>(r);
  lo = fminf(0.0f, bf16_lo_to_f32(m));
  hi = fmaxf(0.0f, -bf16_hi_to_f32(m));
}
__device__ __forceinline__ void row_range(const Row<__half>& r, float& lo, float& hi) {
  const uint32_t m = packed_range<__half2>(r);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
  lo = fminf(0.0f, f.x);
  hi = fmaxf(0.0f, -f.y);
}

// rint(v) + z clamped to 0 .. 15, for |v| far below 2^22 (here at most about
// 30: fp16's smallest scales are off by at most half of themselves): adding
// 1.5 * 2^23 leaves the integer in the low mantissa bits; the integer sum and
// both bounds are one instruction.
__device__ __forceinline__ int code_of(float v, int z) {
  return __viaddmin_s32_relu(__float_as_int(__fadd_rn(v, 12582912.0f)), z - 0x4B400000, 15);
}

// The code of element a of a row with scale s, y = RN(1 / s). A quotient of a
// 16-bit element (11 bits) and s (11 bits) is a half-integer or at least 2^-13
// away from every one, and a y is off by at most 30 * 2^-24: rounded to 2^-16
// (the spacing around 192) it is a tie where a / s is one and on the same side
// of it elsewhere. Two operations instead of the four of the quotient itself.
template <typename T>
__device__ __forceinline__ int code_of(float a, float s, float y, int z) {
  if (sizeof(T) == 4) return code_of(div_by(a, s, y), z);
  return __viaddmin_s32_relu(
      __float_as_int(__fadd_rn(__fmaf_rn(a, y, 192.0f), 12582912.0f - 192.0f)), z - 0x4B400000,
      15);
}

// Scale, its reciprocal and the zero of a row's range. A row of an infinite scale is
// coded with the reciprocal 0 (of s = 1, so that div_by's residual is finite).
__device__ __forceinline__ void row_scale(float lo, float hi, __half& sh, float& s, float& y,
                                          int& z) {
  // (hi - lo) / 15 rounded to nearest
  sh = __float2half_rn(div_by(__fsub_rn(hi, lo), 15.0f, 1.0f / 15.0f));
  if (__half2float(sh) == 0.0f) {  // an all-zero (or vanishing) row: range [-1, 1]
    lo = -1.0f;
    sh = __float2half_rn(2.0f / 15.0f);
  }
  s = __half2float(sh);
  y = __frcp_rn(s);
  z = code_of(div_by(-lo, s, y), 0);
  if (!(s <= 65504.0f)) {  // beyond fp16 (or hi - lo beyond fp32): x / s is 0 for every x
    sh = __ushort_as_half((unsigned short)0x7C00u);
    s = 1.0f;
    y = 0.0f;
    z = 0;
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 4 ? 8 : 16)
    kv_append_kernel(KvRows p, const T* __restrict__ k, const T* __restrict__ v,
                     uint32_t* __restrict__ kc, __half* __restrict__ ks, __half* __restrict__ kz,
                     uint32_t* __restrict__ vc, __half* __restrict__ vs,
                     __half* __restrict__ vz) {
  // no early start of the next kernel: a decode GEMV over the K rows (one head's
  // codes, scales and zeros are INT4 weights of group 128) reads them at once
  wait_previous();
  const int lane = threadIdx.x & 31, half = lane >> 4, col = lane & 15;
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);  // units * H < 2^31 - 8
  if (item >= (uint32_t)(p.units * p.H)) return;
  const int h = (int)(item % (uint32_t)p.H);
  const Unit w = find_unit(p, item / (uint32_t)p.H, half, lane, true);
  if (!w.any) return;
  // bit t: position 8 blk + t is written
  const uint32_t mine = (w.tok[0] >= 0 ? 1u : 0u) | (w.tok[1] >= 0 ? 4u : 0u) |
                        (w.tok[2] >= 0 ? 16u : 0u) | (w.tok[3] >= 0 ? 64u : 0u);
  const uint32_t even = __shfl_sync(0xffffffffu, mine, 0);
  const uint32_t odd = __shfl_sync(0xffffffffu, mine, 16);
  const uint32_t mask = even | (odd << 1);
  if (mask == 0) return;

  Row<T> kr[4], vr[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (w.tok[r] >= 0) {
      kr[r].load(k + w.tok[r] * p.kts + h * p.khs + 8 * col);
      vr[r].load(v + w.tok[r] * p.vts + h * p.vhs + 8 * col);
    } else {
      kr[r].zero();
      vr[r].zero();
    }
  }
  const int64_t row0 = ((int64_t)w.b * p.H + h) * p.cap + 8 * w.blk;  // cache row of the block
  uint4* vword = reinterpret_cast<uint4*>(
      vc + (((int64_t)w.b * p.H + h) * p.nblk + w.blk) * kD + 8 * col + 4 * half);
  uint4 old = make_uint4(0, 0, 0, 0);
  if (mask != 0xFFu) old = *vword;

  // Rows r = 0..3 of this half are block positions 2 r + half. The ranges of its
  // 4 K and 4 V rows first: lane r (K) or 4 + r (V) of the half then works out
  // that row's scale, once for the row instead of once a lane.
  float mylo = 0.0f, myhi = 0.0f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    // bits 2 r and 2 r + 1: either half has a row (the shuffles take both)
    if (((mask >> (2 * r)) & 3u) == 0) continue;
    float lo, hi;
    row_range(kr[r], lo, hi);
    if (col == r) mylo = lo, myhi = hi;
    row_range(vr[r], lo, hi);
    if (col == 4 + r) mylo = lo, myhi = hi;
  }
  __half sh;
  float s, y;
  int z;
  row_scale(mylo, myhi, sh, s, y, z);
  uint32_t words[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (((mask >> (2 * r)) & 3u) == 0) continue;
    float f[8];
    int from = 16 * half + r;
    float sr = __shfl_sync(0xffffffffu, s, from), yr = __shfl_sync(0xffffffffu, y, from);
    int zr = __shfl_sync(0xffffffffu, z, from);
    kr[r].get(f);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      word += (uint32_t)code_of<T>(f[i], sr, yr, zr) << (4 * i);
    if (w.tok[r] >= 0) kc[(row0 + 2 * r + half) * (kD / 8) + col] = word;
    from += 4;
    sr = __shfl_sync(0xffffffffu, s, from);
    yr = __shfl_sync(0xffffffffu, y, from);
    zr = __shfl_sync(0xffffffffu, z, from);
    vr[r].get(f);
    const uint32_t place = half ? 16u << (8 * r) : 1u << (8 * r);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      words[i] += (uint32_t)code_of<T>(f[i], sr, yr, zr) * place;
  }
  {
    const int r = col & 3;
    if (col < 8 && ((mask >> (2 * r + half)) & 1u)) {
      const int64_t at = row0 + 2 * r + half;
      (col < 4 ? ks : vs)[at] = sh;
      (col < 4 ? kz : vz)[at] = __int2half_rn(z);
    }
  }
  // the two halves hold the even and the odd positions of the same 8 words:
  // each keeps 4 of them
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t got =
        __shfl_xor_sync(0xffffffffu, half ? words[j] : words[4 + j], 16);
    o[j] = (half ? words[4 + j] : words[j]) | got;
  }
  if (mask != 0xFFu) {
    // spread the 8 position bits to nibbles: keep the others' codes
    uint32_t m = mask;
    m = (m | (m << 12)) & 0x000F000Fu;
    m = (m | (m << 6)) & 0x03030303u;
    m = (m | (m << 3)) & 0x11111111u;
    m *= 15u;
    o[0] = (o[0] & m) | (old.x & ~m);
    o[1] = (o[1] & m) | (old.y & ~m);
    o[2] = (o[2] & m) | (old.z & ~m);
    o[3] = (o[3] & m) | (old.w & ~m);
  }
  *vword = make_uint4(o[0], o[1], o[2], o[3]);
}

// (q - z) s by one fused multiply-add: a code at mantissa bits 12 - 15 (or 16 - 19)
// of 1.0 is 1 + q / u with u = 2^11 (2^7), and (1 + q / u) (u s) - (u + z) s is
// exact: u + z has 12 bits at most, s has 11.
constexpr uint32_t kOne = 0x3F800000u;
struct Affine {
  float a, b;
  __device__ __forceinline__ Affine(float u, float s, float z) : a(u * s), b(-(u + z) * s) {}
  __device__ __forceinline__ float operator()(uint32_t word, uint32_t mask) const {
    return __fmaf_rn(__uint_as_float(lop3_and_or(word, mask, kOne)), a, b);
  }
};

template <typename T>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 4 ? 8 : 20)
    kv_read_kernel(KvRows p, const uint32_t* __restrict__ kc, const __half* __restrict__ ks,
                   const __half* __restrict__ kz, const uint32_t* __restrict__ vc,
                   const __half* __restrict__ vs, const __half* __restrict__ vz,
                   T* __restrict__ k, T* __restrict__ v) {
  follow_previous();
  const int lane = threadIdx.x & 31, half = lane >> 4, col = lane & 15;
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);  // units * H < 2^31 - 8
  if (item >= (uint32_t)(p.units * p.H)) return;
  const int h = (int)(item % (uint32_t)p.H);
  const Unit w = find_unit(p, item / (uint32_t)p.H, half, lane, false);
  if (!w.any) return;
  const int64_t row0 = ((int64_t)w.b * p.H + h) * p.cap + 8 * w.blk;
  uint4 mine = make_uint4(0, 0, 0, 0);
  if (w.blk >= 0 && w.blk < p.nblk)
    mine = ld_stream_u4(vc + (((int64_t)w.b * p.H + h) * p.nblk + w.blk) * kD + 8 * col +
                        4 * half);
  uint32_t kw[4];
  float sk[4], zk[4], sv[4], zv[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t pos = 8 * w.blk + 2 * r + half;
    const bool ok = w.tok[r] >= 0 && pos >= 0 && pos < p.cap;  // outside: rows of zeros
    const int64_t at = row0 + 2 * r + half;
    kw[r] = ok ? kc[at * (kD / 8) + col] : 0u;
    sk[r] = ok ? __half2float(ks[at]) : 0.0f;
    zk[r] = ok ? __half2float(kz[at]) : 0.0f;
    sv[r] = ok ? __half2float(vs[at]) : 0.0f;
    zv[r] = ok ? __half2float(vz[at]) : 0.0f;
  }
  // all 8 words of this lane's columns: 4 of its own, 4 of the other half's
  const uint32_t own4[4] = {mine.x, mine.y, mine.z, mine.w};
  uint32_t words[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, own4[j], 16);
    words[j] = half ? got : own4[j];
    words[4 + j] = half ? own4[j] : got;
  }
  const uint32_t vmask = half ? 0xF0000u : 0xF000u;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (w.tok[r] < 0) continue;
    float f[8];
    {
      const uint32_t w = kw[r];
      const Affine lo(2048.0f, sk[r], zk[r]), hi(128.0f, sk[r], zk[r]);
      f[0] = lo(w << 12, 0xF000u);
      f[1] = lo(w << 8, 0xF000u), f[2] = hi(w << 8, 0xF0000u);
      f[3] = lo(w, 0xF000u), f[4] = hi(w, 0xF0000u);
      f[5] = lo(w >> 8, 0xF000u), f[6] = hi(w >> 8, 0xF0000u);
      f[7] = lo(w >> 16, 0xF000u);
    }
    Row<T>::store(k + w.tok[r] * p.kts + h * p.khs + 8 * col, f);
    const Affine val(half ? 128.0f : 2048.0f, sv[r], zv[r]);
#pragma unroll
    for (int i = 0; i < 8; ++i)  // nibbles 2 r and 2 r + 1 to bits 12 and 16
      f[i] = val(r == 0 ? words[i] << 12 : r == 1 ? words[i] << 4 : words[i] >> (8 * r - 12),
                 vmask);
    Row<T>::store(v + w.tok[r] * p.vts + h * p.vhs + 8 * col, f);
  }
}

KvRows make_rows(int64_t T, int64_t Hkv, const int64_t* k_strides, const int64_t* v_strides,
                 int64_t B, const int32_t* starts, const int32_t* offsets, int64_t cap) {
  KvRows p;
  p.starts = starts;
  p.offsets = offsets;
  p.T = T;
  p.cap = cap;
  p.units = T / 8 + 2 * B;
  p.kts = k_strides[0];
  p.khs = k_strides[1];
  p.vts = v_strides[0];
  p.vhs = v_strides[1];
  p.B = (int)B;
  p.H = (int)Hkv;
  p.nblk = (int)((cap + 7) / 8);
  return p;
}

template <typename T>
wq_status append(const KvRows& p, const void* k, const void* v, void* const* c, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.units * p.H + kWarps - 1) / kWarps);
  return launch_following(
      kv_append_kernel<T>, grid, 32 * kWarps, 0, st, p, static_cast<const T*>(k),
      static_cast<const T*>(v), static_cast<uint32_t*>(c[0]), static_cast<__half*>(c[1]),
      static_cast<__half*>(c[2]), static_cast<uint32_t*>(c[3]), static_cast<__half*>(c[4]),
      static_cast<__half*>(c[5]));
}

template <typename T>
wq_status read_back(const KvRows& p, void* k, void* v, const void* const* c, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.units * p.H + kWarps - 1) / kWarps);
  return launch_following(
      kv_read_kernel<T>, grid, 32 * kWarps, 0, st, p, static_cast<const uint32_t*>(c[0]),
      static_cast<const __half*>(c[1]), static_cast<const __half*>(c[2]),
      static_cast<const uint32_t*>(c[3]), static_cast<const __half*>(c[4]),
      static_cast<const __half*>(c[5]), static_cast<T*>(k), static_cast<T*>(v));
}

}  // namespace

wq_status launch_kv_append(const void* k, const void* v, wq_dtype dt, int64_t T, int64_t Hkv,
                           const int64_t* k_strides, const int64_t* v_strides, int64_t B,
                           const int32_t* starts, const int32_t* offsets, int64_t cap,
                           void* const* cache, cudaStream_t st) {
  const KvRows p = make_rows(T, Hkv, k_strides, v_strides, B, starts, offsets, cap);
  if (dt == WQ_BF16) return append<__nv_bfloat16>(p, k, v, cache, st);
  if (dt == WQ_FP16) return append<__half>(p, k, v, cache, st);
  return append<float>(p, k, v, cache, st);
}

wq_status launch_kv_read(void* k, void* v, wq_dtype dt, int64_t T, int64_t Hkv,
                         const int64_t* k_strides, const int64_t* v_strides, int64_t B,
                         const int32_t* starts, const int32_t* offsets, int64_t cap,
                         const void* const* cache, cudaStream_t st) {
  const KvRows p = make_rows(T, Hkv, k_strides, v_strides, B, starts, offsets, cap);
  if (dt == WQ_BF16) return read_back<__nv_bfloat16>(p, k, v, cache, st);
  if (dt == WQ_FP16) return read_back<__half>(p, k, v, cache, st);
  return read_back<float>(p, k, v, cache, st);
}

}  // namespace wq
