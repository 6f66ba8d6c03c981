// fp4_format.cuh -- microscaled 4-bit floating point: the formats, their layout
// in memory and the fp32 arithmetic that makes codes and scales.
//
// Codes are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a
// byte, the even element in the low half.  A row's value is
// code * S(block) * s(row):
//   NV16  blocks of 16, S in E4M3; s = 2^k, the smallest power of two (not below
//         2^-126) with max|row| <= 6 * 448 * s; S = E4M3(max|block| / s / 6)
//   MX32  blocks of 32, S = 2^E held as E + 127, the smallest (not below 2^-127)
//         with max|block| <= 6 * S; no row scale
// and code = E2M1(x / s / S), ties to the even code, saturating at 6.
//
// Every step has one right answer that fp32 finds.  Divisions by s and by a power
// of two are exact.  The midpoints between E2M1 values have 3 significant bits
// and S has 4, so x / S meets one only where x is their product, which fp32 holds:
// rounding the IEEE quotient to E2M1 rounds the exact one.
//
// Block scales lie as the tensor core's scale operand wants them: tiles of 128
// rows by 256 elements, each of 4 (NV16) or 2 (MX32) parts of 512 bytes; in a
// part, 16 bytes for each row r of 0..31, made of the four scales of r, r + 32,
// r + 64 and r + 96.  One part goes into four columns of tensor memory by one
// copy.  Scales past K in a tile are 0: E2M1 codes past K read as 0, and 0 times
// NaN would not be.
#pragma once
#include <cstdint>

namespace i8 {

constexpr int kFp4TileK = 256;  // elements of a tile's row: 128 bytes of codes

__host__ __device__ constexpr int fp4_tile_bytes(int block) { return 128 * (kFp4TileK / block); }

// Byte of block `b` of `row` in scales whose tiles are `deep` to a row.
__device__ __forceinline__ int64_t fp4_scale_at(int64_t row, int b, int deep, int block) {
  const int per = kFp4TileK / block;
  const int tile = b / per, in = b % per;
  return ((row >> 7) * deep + tile) * fp4_tile_bytes(block) + (in >> 2) * 512 + (row & 31) * 16 +
         ((row >> 5) & 3) * 4 + (in & 3);
}

// 2^k for k in [-126, 127].
__device__ __forceinline__ float pow2f(int k) { return __int_as_float((k + 127) << 23); }

// NV16: the exponent of a row's scale from the bits of its largest magnitude.
// 6 * 448 = 1.3125 * 2^11.
__device__ __forceinline__ int nv16_row_exponent(uint32_t amax) {
  const int k = static_cast<int>(amax >> 23) - 127 - 11 + ((amax & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return max(k, -126);
}

// MX32: a block's scale byte from the bits of its largest magnitude (255, NaN,
// where that is not finite).  6 = 1.5 * 2^2.
__device__ __forceinline__ uint32_t mx32_scale(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255u;
  const int e = static_cast<int>(amax >> 23) - 2 + ((amax & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));
}

// E4M3 of a value that is not negative, and the value of an E4M3 code.
__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(x));
  return d & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

// Eight E2M1 codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&q)[8]) {
  uint32_t d;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(d)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return d;
}

// About 1 / x.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The codes of 8 elements of one block and the block's scale byte.  top: bits of
// the block's largest magnitude; s and inverse: the row's scale and 1 / s (NV16;
// between 2^-100 and 2^100, where everything below is a normal number).
//
// Quotients t / d come from a = t * y, y about 1 / d, and one correction by the
// residual a * d - t, which an fma gives exactly (P. Markstein, 1990): the result is
// the exact quotient rounded once but for 2^-40 of an ulp, so it meets a midpoint
// of E2M1 or E4M3 where the quotient does, and only there.  With these signs -0
// stays -0.  (In pairs, f32x2, it took 8 % longer.)
template <bool MX>
__device__ __forceinline__ uint32_t fp4_codes8(const float (&t)[8], uint32_t top, float s, float inverse,
                                               uint32_t* scale) {
  float q[8];
  if constexpr (MX) {
    const uint32_t byte = mx32_scale(top);
    const float inv = __int_as_float((254 - min(byte, 253u)) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fmul_rn(t[i], inv);
    *scale = byte;
    return e2m1x8(q);
  } else {
    constexpr float kSixth = 1.0f / 6.0f;
    const float u = __fmul_rn(__uint_as_float(top), inverse), v = __fmul_rn(u, kSixth);
    const uint32_t code = e4m3_of(__fmaf_rn(__fmaf_rn(v, 6.0f, -u), -kSixth, v));
    const float S = e4m3_value(code), y = __fmul_rn(rcp_approx(S), inverse), d = __fmul_rn(S, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = __fmul_rn(t[i], y);
      q[i] = __fmaf_rn(__fmaf_rn(a, d, -t[i]), -y, a);
    }
    *scale = code;
    return code == 0 ? 0u : e2m1x8(q);
  }
}

}  // namespace i8
