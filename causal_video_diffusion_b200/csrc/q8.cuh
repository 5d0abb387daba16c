// q8.cuh -- the 8-bit cache's number format: e4m3 codes under power-of-two scales, one scale for
// 32 channels.
//
// A block with largest magnitude a has the exponent E = the smallest integer >= -111 with
// a <= 448 * 2^E, held as the byte b = E + 127.  448 = 1.75 * 2^8, so with a = 2^e (1 + f), E is
// e - 8 for f <= 0.75 and e - 7 above: on the bits of a, (bits + 0x1FFFFF) >> 23 carries into the
// exponent field exactly when the 23-bit fraction exceeds 0x600000.  x / 2^E is exact (a power of
// two), so the conversion to e4m3 is the only rounding.  E >= -111 keeps every non-zero stored
// value at 2^-120 or above, a normal bf16 number.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "internal.h"
#include "sm100.cuh"

namespace unstep {

constexpr int kQ8Block = 32;             // channels that share a scale
constexpr int kQ8MinByte = 127 - 111;    // smallest scale byte of a block
constexpr uint32_t kQ8NanByte = 255;     // a block with a NaN or an infinity
constexpr uint32_t kQ8TopByte = 247;     // byte of blocks up to the largest fp32: codes up to 240

// Scale byte of a block whose largest magnitude has the fp32 bits `abs_bits` (NaN and infinity
// compare above every finite value).
__device__ __forceinline__ uint32_t q8_scale_byte(uint32_t abs_bits) {
  if (abs_bits >= 0x7F800000u) return kQ8NanByte;
  const int b = static_cast<int>((abs_bits + 0x1FFFFFu) >> 23) - 8;
  return static_cast<uint32_t>(max(b, kQ8MinByte));
}

// 1 / 2^E of a scale byte (16 .. 247).
__device__ __forceinline__ float q8_inv_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Two values -> two codes (lo in the low byte).  |x * inv| <= 448; under the top scale byte (2^120)
// below 256, as fp32 ends at 2^128.  There the caller clamps to 240 first: a value that rounds up to
// the code 256 would read back as 2^128, which is infinite.
__device__ __forceinline__ uint32_t q8_encode2(float lo, float hi, float inv) {
  const uint64_t inv2 = f2_make(inv, inv);
  float a, b;
  f2_split(fmul2(f2_make(lo, hi), inv2), a, b);
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// bf16 pairs that multiply raw codes (see q8_decode2) up to their values: 2^(E + 120) as the
// product of two, because it exceeds bf16 for E > 7; the second is 1 up to kQ8SplitByte, and NaN for
// a NaN block.
constexpr uint32_t kQ8SplitByte = 134;

__device__ __forceinline__ uint32_t q8_mul1(uint32_t byte) {
  return (min(byte, kQ8SplitByte) + 120u) * 0x00800080u;
}

__device__ __forceinline__ uint32_t q8_mul2(uint32_t byte) {
  return byte == kQ8NanByte ? 0x7FC07FC0u
                            : (max(byte, kQ8SplitByte) - kQ8SplitByte + 127u) * 0x00800080u;
}

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// q8_mul1 of a byte that stands in both halves of b2 and does not exceed kQ8SplitByte.
__device__ __forceinline__ uint32_t q8_mul1_pair(uint32_t b2) { return b2 * 128u + 120u * 0x00800080u; }

// Whether one of a word's four scale bytes exceeds kQ8SplitByte.
__device__ __forceinline__ bool q8_any_split(uint32_t word) {
  return __vmaxu4(word, kQ8SplitByte * 0x01010101u) != kQ8SplitByte * 0x01010101u;
}

// Two sign-extended codes, one in each half of w -> a bf16 pair of their values times 2^-120: sign
// in bit 15, the seven magnitude bits in bits 4-10 (e4m3's exponent bias is 7, bf16's 127; subnormal
// codes become subnormal bf16 numbers of the same value).
__device__ __forceinline__ uint32_t q8_decode2(uint32_t w) { return (w * 16u) & 0x87F087F0u; }

// Four codes -> two bf16 pairs, times 2^-120.  A byte selector of 8 + i replicates byte i's sign.
__device__ __forceinline__ uint2 q8_decode4(uint32_t c) {
  uint32_t lo, hi;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(lo) : "r"(c));
  asm("prmt.b32 %0, %1, 0, 0xB3A2;" : "=r"(hi) : "r"(c));
  return make_uint2(q8_decode2(lo), q8_decode2(hi));
}

}  // namespace unstep
