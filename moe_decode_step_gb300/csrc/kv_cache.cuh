// The paged 8-bit KV cache as the kernels see it: E4M3 codes with one E8M0
// scale per (block of tokens, KV head).
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "moe_decode.h"

namespace moe {

constexpr int kKvExpMin = -60, kKvExpMax = 60;   // scale exponents of a block
// Attention's weights carry the values' exponent ev down to this one only; the
// rest of a smaller one multiplies them where they meet the values.  A weight
// relative to M, which a key of exponent 60 may have set, so stays above
// 2^-126 as long as the key counts in the denominator: 60 + 28 + 38 = 126.
constexpr int kKvExpLow = -28;

struct KvView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;
  uint8_t* vs;
  long long bstride, hstride, tstride, sstride;
  int n_blocks, bs_log2, heads;
};

// The scale exponent a stored byte stands for.
__device__ __forceinline__ int kv_exp(uint32_t byte) {
  return min(max((int)byte - 127, kKvExpMin), kKvExpMax);
}

// Smallest e in the cache's range with amax <= 448 * 2^e (448 = 1.75 * 2^8),
// for finite amax >= 0.  The choice keeps the block's largest value from
// saturating, which floor(log2 amax) - 8 would not (up to 12.5% of it).
__device__ __forceinline__ int kv_block_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int be = (int)(b >> 23);
  if (be == 0) return kKvExpMin;   // zero or subnormal
  const int e = be - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kKvExpMin), kKvExpMax);
}

// Four E4M3 codes -> two f16x2 (codes 0, 1 and 2, 3), exact.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Two floats -> two E4M3 codes (a in the low byte): nearest, ties to even,
// magnitudes past 448 to 448, NaN to NaN.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float a, float b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  return c;
}

// Element pair of a bf16 (0) or f16 (1) tensor to floats.
__device__ __forceinline__ float2 unpack16(uint32_t w, int f16) {
  if (f16) return make_float2(f16_lo(w), f16_hi(w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Floats to a bf16 (0) or f16 (1) pair, round to nearest even.
__device__ __forceinline__ uint32_t pack16(float a, float b, int f16) {
  if (f16) return pack_f16x2(a, b);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

}  // namespace moe
