// ufp4_vec.hpp -- eight-value vector loads and stores of bf16 and fp32 rows at
// any element alignment, and the 8-bit checkpoint's block arithmetic (device
// code of the expert-layer kernels).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ufp4_device.hpp"

namespace ufp4 {

typedef uint32_t v32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t v32x4 __attribute__((ext_vector_type(4)));

// 16 and 8 bytes at any address.  gfx950 runs with
// unaligned vector access to global memory on, so these are one instruction
// at every alignment (an odd row width only costs the extra cache lines that
// a vector straddles).
// S: past the caches (nontemporal), for calls whose data does not fit them.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
template <bool S = false>
__device__ __forceinline__ v32x4 load16(const void* p) {
  const u32x4_any* q = static_cast<const u32x4_any*>(p);
  const u32x4_any v = S ? __builtin_nontemporal_load(q) : *q;
  return v32x4{v.x, v.y, v.z, v.w};
}
template <bool S = false>
__device__ __forceinline__ void store_16(void* p, v32x4 v) {
  u32x4_any* q = static_cast<u32x4_any*>(p);
  if (S) __builtin_nontemporal_store(u32x4_any{v.x, v.y, v.z, v.w}, q);
  else *q = u32x4_any{v.x, v.y, v.z, v.w};
}
template <bool S = false>
__device__ __forceinline__ v32x2 load8(const void* p) {
  const u32x2_any* q = static_cast<const u32x2_any*>(p);
  const u32x2_any v = S ? __builtin_nontemporal_load(q) : *q;
  return v32x2{v.x, v.y};
}
template <bool S = false>
__device__ __forceinline__ void store_8(void* p, v32x2 v) {
  u32x2_any* q = static_cast<u32x2_any*>(p);
  if (S) __builtin_nontemporal_store(u32x2_any{v.x, v.y}, q);
  else *q = u32x2_any{v.x, v.y};
}

// Fewer than eight values of 2 (or 1) bytes each, as the 4, 2 and 1 of them that
// n's bits name, packed to the front: a row's end costs up to three accesses.
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));
__device__ __forceinline__ v32x4 tail_load(const uint16_t* p, int n) {
  v32x2 a = {0u, 0u};
  uint32_t b = 0, c = 0;
  if (n & 4) a = load8(p);
  if (n & 2) b = *reinterpret_cast<const u32_any*>(p + (n & 4));
  if (n & 1) c = p[n & 6];
  const uint32_t bc = n & 2 ? b : c, cb = n & 2 ? c : 0u;  // what follows the four
  return n & 4 ? v32x4{a.x, a.y, bc, cb} : v32x4{bc, cb, 0u, 0u};
}
__device__ __forceinline__ void tail_store(uint16_t* p, v32x4 w, int n) {
  const uint32_t w0 = n & 4 ? w.z : w.x, w1 = n & 4 ? w.w : w.y;
  if (n & 4) store_8(p, v32x2{w.x, w.y});
  if (n & 2) *reinterpret_cast<u32_any*>(p + (n & 4)) = w0;
  if (n & 1) p[n & 6] = (uint16_t)(n & 2 ? w1 : w0);
}
__device__ __forceinline__ v32x2 tail_load(const uint8_t* p, int n) {
  uint32_t a = 0, b = 0, c = 0;
  if (n & 4) a = *reinterpret_cast<const u32_any*>(p);
  if (n & 2) b = *reinterpret_cast<const u16_any*>(p + (n & 4));
  if (n & 1) c = p[n & 6];
  const uint32_t bc = n & 2 ? b | (c << 16) : c;
  return n & 4 ? v32x2{a, bc} : v32x2{bc, 0u};
}
__device__ __forceinline__ void tail_store(uint8_t* p, v32x2 w, int n) {
  const uint32_t r = n & 4 ? w.y : w.x;
  if (n & 4) *reinterpret_cast<u32_any*>(p) = w.x;
  if (n & 2) *reinterpret_cast<u16_any*>(p + (n & 4)) = (uint16_t)r;
  if (n & 1) p[n & 6] = (uint8_t)(n & 2 ? r >> 16 : r);
}

// Two fp32 values to a bf16 pair (round to nearest even, NaN stays NaN).
typedef float f32x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2v v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2v));
}
__device__ __forceinline__ uint16_t to_bf16(float f) { return (uint16_t)(pack_bf16(f, 0.0f) & 0xFFFFu); }
__device__ __forceinline__ float from_bf16(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// Rows of bf16 (uint16_t) or fp32 values: eight at a time, n of them valid.
struct V8 {
  float v[8];
};
__device__ __forceinline__ V8 unpack(v32x4 w) {
  return V8{{bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y), bf_lo(w.z), bf_hi(w.z), bf_lo(w.w), bf_hi(w.w)}};
}
__device__ __forceinline__ v32x4 pack(const V8& a) {
  return v32x4{pack_bf16(a.v[0], a.v[1]), pack_bf16(a.v[2], a.v[3]), pack_bf16(a.v[4], a.v[5]),
               pack_bf16(a.v[6], a.v[7])};
}
template <bool S = false>
__device__ __forceinline__ V8 row_load(const uint16_t* p, int n) {
  if (n >= 8) return unpack(load16<S>(p));
  return unpack(tail_load(p, n));
}
template <bool S = false>
__device__ __forceinline__ V8 row_load(const float* p, int n) {
  V8 r;
  if (n >= 8) {
    const v32x4 a = load16<S>(p), b = load16<S>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[i] = __uint_as_float(a[i]);
      r.v[4 + i] = __uint_as_float(b[i]);
    }
    return r;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = i < n ? p[i] : 0.0f;
  return r;
}
template <bool S = false>
__device__ __forceinline__ void row_store(uint16_t* p, const V8& a, int n) {
  const v32x4 w = pack(a);
  if (n >= 8) {
    store_16<S>(p, w);
    return;
  }
  tail_store(p, w, n);
}
template <bool S = false>
__device__ __forceinline__ void row_store(float* p, const V8& a, int n) {
  if (n >= 8) {
    v32x4 x, y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __float_as_uint(a.v[i]);
      y[i] = __float_as_uint(a.v[4 + i]);
    }
    store_16<S>(p, x);
    store_16<S>(p + 4, y);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = a.v[i];
}
// Raw bf16 bits, moved without conversion.
template <bool S = false>
__device__ __forceinline__ v32x4 row_bits(const uint16_t* p, int n) {
  if (n >= 8) return load16<S>(p);
  return tail_load(p, n);
}
template <bool S = false>
__device__ __forceinline__ void row_store_bits(uint16_t* p, v32x4 w, int n) {
  if (n >= 8) {
    store_16<S>(p, w);
    return;
  }
  tail_store(p, w, n);
}
template <bool S = false>
__device__ __forceinline__ v32x2 code_bits(const uint8_t* p, int n) {
  if (n >= 8) return load8<S>(p);
  return tail_load(p, n);
}
template <bool S = false>
__device__ __forceinline__ void code_store(uint8_t* p, v32x2 w, int n) {
  if (n >= 8) {
    store_8<S>(p, w);
    return;
  }
  tail_store(p, w, n);
}

// ------------------------------------------------------- 8-bit checkpoint
// A block of 32 lies in four neighbouring lanes, eight values each.
constexpr int kCkptINT8 = 0, kCkptE4M3 = 1;
constexpr int kCkptBlock = 32;

// Largest of four neighbouring lanes' values.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
  v = v > a ? v : a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
  return v > b ? v : b;
}

// Largest magnitude of eight bf16 values, as its bit pattern (an infinity or
// a NaN is above every finite value).
__device__ __forceinline__ uint32_t bits_max(v32x4 w) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    m = m > lo ? m : lo;
    m = m > hi ? m : hi;
  }
  return m;
}

// The block's scale (bf16 bits) from the bits of its largest magnitude.
// amax / Q is divided by its reciprocal and one corrected step, which gives
// the correctly rounded quotient; rounding its bits up to 16 then gives the
// smallest bf16 >= amax / Q, since amax has 8 significant bits and a quotient
// that is not a bf16 itself is further from one than fp32's rounding.
template <int FMT>
__device__ __forceinline__ uint32_t ckpt_scale(uint32_t amax_bits) {
  constexpr float Q = FMT == kCkptINT8 ? 127.0f : 448.0f, R = 1.0f / Q;
  if (amax_bits >= 0x7F80u) return 0x7FC0u;
  const float a = __uint_as_float(amax_bits << 16);
  float q = a * R;
  q = __builtin_fmaf(__builtin_fmaf(-q, Q, a), R, q);
  const uint32_t s = (__float_as_uint(q) + 0xFFFFu) >> 16;
  return s > 0x0D80u ? s : 0x0D80u;  // 2^-100
}

// Eight values to codes under the block's scale.  r is 1/s correctly rounded
// (hardware estimate, one Newton step; s has 8 significant bits), and x r
// corrected by the exact remainder is x / s correctly rounded, so a tie of
// x / s reaches the code's rounding as a tie.
template <int FMT>
__device__ __forceinline__ v32x2 ckpt_encode(v32x4 w, uint32_t scale_bits) {
  if (scale_bits == 0x7FC0u) return v32x2{0u, 0u};
  const float s = __uint_as_float(scale_bits << 16);
  float r = __builtin_amdgcn_rcpf(s);
  r = __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
  const V8 x = unpack(w);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = x.v[i] * r;
    q[i] = __builtin_fmaf(__builtin_fmaf(-a, s, x.v[i]), r, a);
  }
  v32x2 c;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* p = q + 4 * h;
    if (FMT == kCkptINT8) {
      // adding 1.5 2^23 rounds to a whole number, whose two's complement is
      // then the low byte of the sum
      const float M = 12582912.0f;
      const uint32_t ab = __builtin_amdgcn_perm(__float_as_uint(p[1] + M), __float_as_uint(p[0] + M), 0x0C0C0400u);
      const uint32_t cd = __builtin_amdgcn_perm(__float_as_uint(p[3] + M), __float_as_uint(p[2] + M), 0x04000C0Cu);
      c[h] = ab | cd;
    } else {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(p[0], p[1], 0, false);
      c[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(p[2], p[3], v, true);
    }
  }
  return c;
}

// The kept values, code * scale, exact in fp32.
template <int FMT>
__device__ __forceinline__ V8 ckpt_decode(v32x2 c, float s) {
  V8 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (FMT == kCkptINT8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r.v[4 * h + i] = (float)(int8_t)(c[h] >> (8 * i)) * s;
    } else {
      const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], false);
      const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], true);
      r.v[4 * h] = a[0] * s;
      r.v[4 * h + 1] = a[1] * s;
      r.v[4 * h + 2] = b[0] * s;
      r.v[4 * h + 3] = b[1] * s;
    }
  }
  return r;
}

}  // namespace ufp4
