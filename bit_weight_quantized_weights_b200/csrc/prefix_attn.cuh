// Shared by the kernels of the shared-prefix attention: the caches, the
// problem, and the dequantization of a code word to exact fp16 integers.
#pragma once

#include "common.cuh"

namespace wq {
inline namespace prefix {

constexpr int kD = 128;
constexpr float kNone = -1e30f;      // the running bound before any key
// The bound is put kLift below a row's largest exponent, and moved when one is kSlack
// above it: the fp16 weights w reach from 2^7 to 2^15 at their largest, and keys whose
// weight is 2^-21 of that still have all bits of theirs (where one key has the weight but
// no value, the many far below it are the row's result). 160 sequences x 8 heads x 2000
// keys 2^-18 below one, fp16: the error, over that of rounding each weight and output at
// its type's normal step, is 0.8, and was 2.6 with the bound at the largest.
constexpr float kLift = 7.0f, kSlack = 15.0f;

struct Cache {
  const uint32_t* kc;   // [.., cap, 16]
  const __half* ks;     // [.., cap]
  const __half* kz;
  const uint32_t* vc;   // [.., nblk, 128]
  const __half* vs;
  const __half* vz;
  int64_t cap;
  int64_t nblk;
};

struct PrefixArgs {
  const void* q;         // [B, Hq, 128], rows of a sequence q_stride elements apart
  int64_t q_stride;
  int fp16;              // q and out are fp16 (else bf16)
  int B, Hq, Hkv, R;
  Cache pre, own;
  int P;
  const int32_t* lengths;
  int chunk_p, nsp;      // keys of a prefix range; partial results a row gets of the prefix
  int chunk_o, nso;      // keys of a range of own tokens, ranges
  int nrt;               // prefix row tiles (groups of them on tcgen05)
  int nprefix;           // CTAs of the prefix: Hkv * nrt * ranges
  float* part;           // [B * Hq][nsp + nso][128]
  float2* stat;          // [B * Hq][nsp + nso] (m, E)
  void* out;
};

__device__ __forceinline__ float ex2(float x) {  // ex2.approx: 2^-22 relative; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }

// Codes of nibbles (0, 4) and (1, 5) of a word as exact fp16 integers q - z:
// a nibble placed in the low mantissa bits of 1024 is 1024 + q, one place
// higher 1024 + 16 q. z1024 = (1024 + z) of both keys, zm64 = -(64 + z).
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t z1024, uint32_t zm64, uint32_t& even,
                                          uint32_t& odd) {
  const uint32_t e = lop3_and_or(w, 0x000F000Fu, 0x64006400u);
  const uint32_t o = lop3_and_or(w, 0x00F000F0u, 0x64006400u);
  even = h2(__hsub2(as_h2(e), as_h2(z1024)));
  odd = h2(__hfma2(as_h2(o), as_h2(0x2C002C00u), as_h2(zm64)));  // 0x2C00 = 1/16
}

// The power of two 2^e that brings a row's largest magnitude into
// [2^14, 2^15), and its inverse; 1 for a row of zeros, infinities or
// magnitudes whose power of two is outside fp32's normal range.
__device__ __forceinline__ void row_scale(float amax, float& up, float& down) {
  const int ex = (int)(__float_as_uint(amax) >> 23);
  const bool scaled = ex > 14 && ex < 255;
  up = scaled ? __uint_as_float((uint32_t)(127 + 14 + 127 - ex) << 23) : 1.0f;
  down = scaled ? __uint_as_float((uint32_t)(ex - 14) << 23) : 1.0f;
}
constexpr float kScoreScale = 1.4426950408889634f / 11.313708498984761f;  // log2(e) / sqrt(128)

}  // namespace prefix
}  // namespace wq
