// Rows held in 4 bits (include/fa.h: fa_append4). A row's d values are groups of 32; a group is a scale s
// (its largest magnitude over 7, rounded up to five significant bits, as bf16) times whole numbers −7 … 7,
// kept plus 8 in four bits. Seven times a five-bit number has eight bits: every value is a bf16 number,
// so codes become tensor-core operands without a rounding.
//
// The order of a row's codes makes a thread's operand fragments out of whole words, eight codes each:
//   keys    word c·(d/32) + w: dimensions 32w + 4c + (0, 2, 16, 18, 1, 3, 17, 19). Thread c of a quad reads
//           its d/32 words in one piece; bits 4i and 16 + 4i of a word are the pairs of the B fragments
//           of two products of 16 dimensions, whose order within the 16 is (4c, 4c + 1 | 4c + 2, 4c + 3)
//           for the thread: any order does, as long as Q's fragments have the same.
//   values  word 8h + n: dimensions 64h + n + 8·(0 … 7): column n of eight 16 × 8 products.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "sm103.cuh"

namespace fa {

// From codes to values: with a code in bits 3 … 6 of a half word, under the exponent of 16, the half is the bf16
// number 16 + code; (16 + code)·s − 24·s = (code − 8)·s in one fused operation, exact since 24·s has
// seven bits. (Not under the exponent of 128, where no shift would be needed: 136·s has ten.)
struct FourScale {
  __nv_bfloat162 s, off;
};
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }
__device__ __forceinline__ FourScale four_scale(uint32_t pair) {
  FourScale f;
  f.s = as_bf162(pair);
  f.off = __hmul2(f.s, as_bf162(0xC1C0C1C0u));  // −24
  return f;
}
// The pair of codes at bits 4i and 16 + 4i of a word, as bf16 values.
template <int I>
__device__ __forceinline__ uint32_t four_pair(uint32_t word, const FourScale& f) {
  const uint32_t at = I == 0 ? word << 3 : word >> (I == 0 ? 0 : 4 * I - 3);
  // (mask and exponent in registers, so that both are one operation, which with two constants in its code
  // they are not: B8 H16 Hkv4 ctx60000 d128 65.8 -> 56.3 µs)
  uint32_t mask, exponent, y;
  asm("mov.b32 %0, 0x00780078;" : "=r"(mask));
  asm("mov.b32 %0, 0x41804180;" : "=r"(exponent));
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(at), "r"(mask), "r"(exponent));  // (at & mask) | exponent
  const __nv_bfloat162 x = __hfma2(as_bf162(y), f.s, f.off);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// A group's scale from the bits of its largest magnitude. Below 2⁻¹⁰⁰: zeros. From 2¹²⁵ on (infinities and NaN
// among them): a NaN, which the whole group then stands for.
__device__ __forceinline__ float four_scale_of(uint32_t top_bits) {
  if (top_bits >= 0x7E000000u) return __uint_as_float(0x7FC00000u);
  if (top_bits < 0x0D800000u) return 0.f;
  // (times a little less than 1/7: a quotient that has five bits stays below itself and is rounded up to it,
  // and an eight-bit number over 7 comes no nearer to any other than 2⁻⁹ of it)
  const uint32_t q = __float_as_uint(__uint_as_float(top_bits) * 0.14285701f);
  return __uint_as_float((q + 0x7FFFFu) & ~0x7FFFFu);
}

// Eight values over a scale s, each the nearest whole number, ties to even, plus 8, as a word (number e at bits
// 4e). The quotient is x·(1/s) with 1/s in two parts, within 2⁻²⁴ of itself before the addition of
// 1.5·2²³ + 8, in whose lowest bits it becomes a whole number: so a quotient half-way between two numbers,
// which fp32 has, is found exactly (an eight-bit over a five-bit number comes no nearer to half-way than
// 2⁻¹¹ otherwise). All on the multiply-add pipe; the bits are gathered there too.
__device__ __forceinline__ uint32_t four_codes(const float* v, float s) {
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const float rest = fmaf(-s, inv, 1.0f) * inv;
  constexpr float kRound = 12582912.0f + 8.0f;  // bits 0x4B400008
  uint32_t w = 0u;
#pragma unroll
  for (int e = 7; e >= 0; --e) w = w * 16u + __float_as_uint(fmaf(v[e], inv, v[e] * rest) + kRound);
  return w - 0x4B400000u * 0x11111111u;  // (0x4B400000 in every place)
}
// The bits of the largest magnitude among eight bf16 values and those of the other three lanes of a group; a
// NaN's where there is one.
__device__ __forceinline__ uint32_t four_top(const uint4& x) {
  auto top = [](__nv_bfloat162 a, __nv_bfloat162 b) { return __hmax2_nan(a, b); };
  __nv_bfloat162 m = top(top(__habs2(as_bf162(x.x)), __habs2(as_bf162(x.y))), top(__habs2(as_bf162(x.z)), __habs2(as_bf162(x.w))));
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) m = top(m, as_bf162(__shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&m), off)));
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
  return max(u << 16, u & 0xFFFF0000u);
}

// Eight lanes' words as an 8 × 8 matrix of codes (lane x, nibble n), transposed.
__device__ __forceinline__ uint32_t four_transpose(uint32_t w, int x) {
  uint32_t y = __shfl_xor_sync(0xffffffffu, w, 4);
  w = (x & 4) ? (w & 0xFFFF0000u) | (y >> 16) : (w & 0x0000FFFFu) | (y << 16);
  y = __shfl_xor_sync(0xffffffffu, w, 2);
  w = (x & 2) ? (w & 0xFF00FF00u) | ((y >> 8) & 0x00FF00FFu) : (w & 0x00FF00FFu) | ((y << 8) & 0xFF00FF00u);
  y = __shfl_xor_sync(0xffffffffu, w, 1);
  return (x & 1) ? (w & 0xF0F0F0F0u) | ((y >> 4) & 0x0F0F0F0Fu) : (w & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
}

// Between eight dimensions in a row (lane x of eight holds 8x … 8x + 7) and the keys' words: lanes x and x ^ 2
// exchange halves, so that lane x holds, of its group of 32, dimensions 4c + (0 … 3) and 16 + 4c +
// (0 … 3), c = four_key_word(x); then nibbles a0 a1 a2 a3 b0 b1 b2 b3 become a0 a2 b0 b2 a1 a3 b1 b3.
__device__ __forceinline__ int four_key_word(int x) { return 2 * (x & 1) + ((x >> 1) & 1); }
__device__ __forceinline__ uint32_t four_halves(uint32_t w, int x) {
  const uint32_t y = __shfl_xor_sync(0xffffffffu, w, 2);
  return (x & 2) ? (w & 0xFFFF0000u) | (y >> 16) : (w & 0x0000FFFFu) | (y << 16);
}
__device__ __forceinline__ uint32_t four_to_key(uint32_t w, int x) {
  w = four_halves(w, x);
  return (w & 0x0000000Fu) | ((w >> 4) & 0x000000F0u) | ((w >> 8) & 0x00000F00u) | ((w >> 12) & 0x0000F000u) |
         ((w << 12) & 0x000F0000u) | ((w << 8) & 0x00F00000u) | ((w << 4) & 0x0F000000u) | (w & 0xF0000000u);
}
__device__ __forceinline__ uint32_t four_from_key(uint32_t w, int x) {
  w = (w & 0x0000000Fu) | ((w & 0x000000F0u) << 4) | ((w & 0x00000F00u) << 8) | ((w & 0x0000F000u) << 12) |
      ((w & 0x000F0000u) >> 12) | ((w & 0x00F00000u) >> 8) | ((w & 0x0F000000u) >> 4) | (w & 0xF0000000u);
  return four_halves(w, x);
}

}  // namespace fa
