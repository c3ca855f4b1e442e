// One page of one KV head in the E4M3 cache: a record of bytes that holds the
// codes in the order in which the tensor-core fragments of a warp want them, so
// that every lane reads 16 bytes at a time, whole 512-byte lines of shared or
// global memory per warp and nothing to transpose, and one bulk copy brings all.
//   K codes  [D / 64][S][64]                       dims of one token, 64 at a time
//   V codes  [S / 16][D / 32][8][4][4][2][2]       [s][i][g][t][c][hi][lo] holds
//            dim 32 i + 4 g + c of token 16 s + 8 hi + 2 t + lo
//   K scales [S], V scales [S]                     exponent bytes (E8M0): 2^(b - 127), 113 to 134
// A code times its token's scale is the value; with exponents in [-14, 7] that is
// always an fp16 number (E4M3 has 4 significant bits, its smallest step is 2^-9).
#pragma once

#include "common.cuh"

namespace quest {

constexpr int kScaleMin = -14, kScaleMax = 7;
constexpr uint32_t kScaleTop = 0x7b00u;       // fp16 bits of 448 * 2^7, the largest value kept

__host__ __device__ constexpr size_t record_bytes(int page_size, int head_dim) {
  return (size_t)2 * page_size * (head_dim + 1);
}
// Byte of a record: K code of (token, dim), V code of (token, dim).
__device__ __forceinline__ int k_code_at(int S, int token, int dim) {
  return (dim >> 6) * S * 64 + token * 64 + (dim & 63);
}

// Two codes as fp16 (exact).
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}
// Two fp16 as codes, to the nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3_codes(uint32_t h2) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h2));
  return c;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 2^e as an fp16 pair, -14 <= e <= 15.
__device__ __forceinline__ uint32_t pow2_h2(int e) { return (uint32_t)(e + 15) * 0x04000400u; }
// Scale bytes of two tokens (bits 0..7 and 16..23) as an fp16 pair.
__device__ __forceinline__ uint32_t scale_h2(uint32_t two) { return (two - 0x00700070u) << 10; }
__device__ __forceinline__ float scale_f(uint32_t byte) { return __uint_as_float(byte << 23); }

// The exponent of a row whose largest magnitude has these fp16 bits: the least
// e with 448 * 2^e = 1.75 * 2^(e + 8) at or above it.
__device__ __forceinline__ int scale_exponent(uint32_t top) {
  return min(kScaleMax, max(kScaleMin, (int)((top + 0xffu) >> 10) - 23));
}
// Largest magnitude bits of two fp16 pairs' halves (not a number: above infinity).
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, uint32_t h2) {
  uint32_t r;
  asm("{\n\t.reg .b32 a;\n\tabs.f16x2 a, %2;\n\tmax.NaN.f16x2 %0, %1, a;\n\t}" : "=r"(r) : "r"(m), "r"(h2));
  return r;
}
// The greatest codes at or below four fp16 numbers (two pairs), as e4m3_floor
// does it, four at a time: round to nearest, and one code down where that is
// above the number.
__device__ __forceinline__ uint32_t e4m3_floor4(uint32_t x01, uint32_t x23, bool& ovf) {
  const uint32_t least = 0xdf00df00u;                   // -448: nothing is kept below
  uint32_t y01, y23;
  asm("max.f16x2 %0, %1, %2;" : "=r"(y01) : "r"(x01), "r"(least));
  asm("max.f16x2 %0, %1, %2;" : "=r"(y23) : "r"(x23), "r"(least));
  ovf = ovf || y01 != x01 || y23 != x23;
  const uint32_t c01 = e4m3_codes(y01), c23 = e4m3_codes(y23);
  const uint32_t d01 = e4m3_pair(c01), d23 = e4m3_pair(c23);
  auto above = [](const uint32_t& d, const uint32_t& y) {
    return __hgt2_mask(*reinterpret_cast<const __half2*>(&d), *reinterpret_cast<const __half2*>(&y));
  };
  uint32_t c = c01 | c23 << 16;
  const uint32_t down = __byte_perm(above(d01, y01), above(d23, y23), 0x6420);
  const uint32_t step = ~((c >> 7 & 0x01010101u) * 0xfeu);      // -1, or +1 below zero
  c = __vadd4(c, step & down);
  return c & ~__vcmpeq4(c, 0x80808080u);                // a zero stays +0
}
// What cannot be kept as it is: not a number becomes 0, more than 448 * 2^7 becomes that.
__device__ __forceinline__ uint32_t keepable(uint32_t h2) {
  const uint32_t m = h2 & 0x7fff7fffu, top = kScaleTop * 0x00010001u;
  const uint32_t num = ~__vcmpgtu2(m, 0x7c007c00u);
  return (__vminu2(m, top) | (h2 & 0x80008000u)) & num;
}

}  // namespace quest
