// ufp4_expand.hpp -- packed 4-bit codes under E4M3 block scales to fp16, exact,
// for the products on the fp16 MFMA (byte arithmetic described in
// ufp4_gemm.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ufp4_device.hpp"

namespace ufp4 {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t g32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t g32x4 __attribute__((ext_vector_type(4)));

// High bytes of the fp16 encodings of the grid magnitudes by magnitude
// index (low word: indices 0..3, high word: 4..7).
template <int GRID>
__device__ __forceinline__ uint32_t f16_hi_lo() {
  return GRID == kGridINT4 ? 0x42403C00u : 0x3E3C3800u;  // {0, 1, 2, 3} / {0, .5, 1, 1.5}
}
template <int GRID>
__device__ __forceinline__ uint32_t f16_hi_hi() {
  return GRID == kGridE1M2 ? 0x43424140u    // 2, 2.5, 3, 3.5
         : GRID == kGridINT4 ? 0x47464544u  // 4, 5, 6, 7
                             : 0x46444240u; // 2, 3, 4, 6 (E2M1; the clamped grid uses 0..4)
}

// Two's-complement nibbles -> sign-magnitude nibbles, eight at a time (for
// a negative nibble n, |n| = (n ^ 7) + 1 with the sign bit kept).
__device__ __forceinline__ uint32_t signmag8(uint32_t P) {
  const uint32_t A = P & 0x88888888u, S = A >> 3;
  return (P ^ (A - S)) + S;
}

// Eight codes (element 2i in the low nibble of byte i) to four fp16 pairs
// times the block scale d2 = (d, d).
template <int GRID>
__device__ __forceinline__ void expand8(uint32_t word, f16x2 d2, uint32_t out[4]) {
  if (GRID == kGridINT4) word = signmag8(word);
  const uint32_t lo = f16_hi_lo<GRID>(), hi = f16_hi_hi<GRID>();
  // high bytes of the even (low-nibble) and odd (high-nibble) elements; the
  // sign bits are merged by one three-input bitwise op, a | (b & c)
  // (truth table 0xF8)
  const uint32_t he = (uint32_t)__builtin_amdgcn_bitop3_b32(__builtin_amdgcn_perm(hi, lo, word & 0x07070707u),
                                                             word << 4, 0x80808080u, 0xF8);
  const uint32_t ho = (uint32_t)__builtin_amdgcn_bitop3_b32(__builtin_amdgcn_perm(hi, lo, (word >> 4) & 0x07070707u),
                                                             word, 0x80808080u, 0xF8);
  // (element 2i, element 2i+1) = (0x00, he.byte i, 0x00, ho.byte i); selector
  // 0x0C gives a zero byte, 0..3 the bytes of he, 4..7 those of ho
  out[0] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x040C000Cu)) * d2);
  out[1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x050C010Cu)) * d2);
  out[2] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x060C020Cu)) * d2);
  out[3] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x070C030Cu)) * d2);
}

// One 16-element block: 8 code bytes and its E4M3 scale byte, to 16 fp16
// values (eight words, element 2i in the low half of word i).
template <int GRID>
__device__ __forceinline__ void expand16(g32x2 codes, uint32_t sbyte, uint32_t o[8]) {
  // the hardware OCP E4M3 decode of the (non-negative) scale byte; exact,
  // and every E4M3 value is an fp16 value
  const _Float16 d = (_Float16)__builtin_amdgcn_cvt_pk_f32_fp8((int)(sbyte & 0x7Fu), false)[0];
  const f16x2 d2 = {d, d};
  expand8<GRID>(codes.x, d2, o);
  expand8<GRID>(codes.y, d2, o + 4);
}

// The 16 fp16 values of a block to dst (16-byte aligned).
__device__ __forceinline__ void store16(const uint32_t o[8], _Float16* dst) {
  g32x4* p = reinterpret_cast<g32x4*>(dst);
  p[0] = g32x4{o[0], o[1], o[2], o[3]};
  p[1] = g32x4{o[4], o[5], o[6], o[7]};
}

// ------------------------------------------------------------------------
// The grouped products' expansion: the same values times 2^-kExpandShift, in
// fewer operations.  fp16 is linear under the exponents 0 and 1 (bits b are
// b 2^-24 up to 2047), so a code needs no table if it becomes the bits of one;
// the scale is applied as d 2^7 (at most 57344).
//   E1M2: the magnitude goes to bits 8..10 (m 2^-16), the sign to the sign bit;
//     two bitwise operations make four high bytes.  The result is value d 2^-8.
//   INT4: value + 8 goes to bits 4..7 ((value + 8) 2^-20), and one fused
//     operation multiplies and takes the 8 off: value d 2^-13.  (11 operations
//     for eight codes; over signs and magnitudes it were 18.)
//   E2M1 codes have a hardware conversion: value d.
// Every result is a multiple of 2^-22 of at most 11 bits, exact in fp16
// (subnormals included, which the MFMA takes as they are).
template <int GRID>
constexpr int kExpandShift = GRID == kGridE1M2 ? 8 : GRID == kGridINT4 ? 13 : 0;

// The scales of two neighbouring blocks from their E4M3 bytes (sign bits 0).
template <int GRID>
__device__ __forceinline__ f16x2 expand_scales(uint32_t two_bytes) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)two_bytes, kExpandShift<GRID> ? 128.0f : 1.0f, false);
}

template <int GRID>
__device__ __forceinline__ void expand8_shifted(uint32_t w, f16x2 d, uint32_t out[4]) {
  f16x2 v[4];
  if (GRID == kGridINT4) {
    const uint32_t he = ((w << 4) & 0xF0F0F0F0u) ^ 0x80808080u, ho = (w & 0xF0F0F0F0u) ^ 0x80808080u;
    const _Float16 eight = (_Float16)(-1.0f / 131072.0f);  // -8 2^-20
    const f16x2 off = d * f16x2{eight, eight};
    v[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x0C040C00u));
    v[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x0C050C01u));
    v[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x0C060C02u));
    v[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x0C070C03u));
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v[i], d, off));
    return;
  }
  if (GRID == kGridE2M1 || GRID == kGridE2M1C) {
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
  } else {
    const uint32_t he = (w & 0x07070707u) | ((w << 4) & 0x80808080u);
    const uint32_t ho = ((w >> 4) & 0x07070707u) | (w & 0x80808080u);
    v[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x040C000Cu));
    v[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x050C010Cu));
    v[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x060C020Cu));
    v[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(ho, he, 0x070C030Cu));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = __builtin_bit_cast(uint32_t, v[i] * d);
}

}  // namespace ufp4
