// ufp4_matvec.hip -- products of a few rows of x with a 4-bit weight matrix:
// y[t][n] = S sum over k of x'[t][k] w[n][k].
//
// The codes are expanded to 16-bit numbers in registers (exact) and multiplied on
// the matrix cores as they come from memory: lane (r, g) of a wave holds 32
// neighbouring codes of row r of 16, which are four fragments of 16 rows x 32
// values of K.  The order of the values along K inside a step is free as long as
// x' has the same, so nothing is exchanged between lanes.
//   NV16: fp16 (ufp4_expand.hpp), the block scale in the operand.  fp16 has the
//     range for a code times an E4M3 scale; x' is brought into it by a power of
//     two for each token.
//   MX32: bf16, which has the range of the power-of-two scales; x' is the sum of
//     one or three bf16 numbers.
#include "ufp4_expand.hpp"
#include "ufp4_serve.hpp"
#include "ufp4_vec.hpp"

namespace ufp4 {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kMvWaves = 8, kMvThreads = 64 * kMvWaves;
constexpr int kLdsTokens = 4;
constexpr size_t kLdsX = 96 << 10;  // bytes

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // normal e
__device__ __forceinline__ double pow2d(int e) { return __longlong_as_double((long long)(e + 1023) << 52); }

// ---------------------------------------------------------------- x'
// Fragments of x': element k of a token is element k % 8 of the 16-byte piece of
// lane group g = k % 128 / 32, step i = k % 32 / 8, chunk c = k / 128.  Pieces are
// ordered [c][i][part][g][token of TP].
__device__ __forceinline__ size_t piece_at(int64_t c, int i, int parts, int part, int g, int TP, int t) {
  return ((((size_t)c * 4 + i) * parts + part) * 4 + g) * TP + t;
}

// 16 values of x, zeros past K.
__device__ __forceinline__ void load_block(const MatvecParams& p, int64_t t, int64_t k, float v[16]) {
  if (t < p.tokens && k < p.K) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const V8 a = p.x_f32 ? row_load(static_cast<const float*>(p.x) + t * p.ldx + k + 8 * h, 8)
                           : row_load(static_cast<const uint16_t*>(p.x) + t * p.ldx + k + 8 * h, 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * h + j] = a.v[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = 0.0f;
  }
}

// Largest finite magnitude, as bits.
__device__ __forceinline__ uint32_t block_max(const float v[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t a = __float_as_uint(v[j]) & 0x7FFFFFFFu;
    m = a < 0x7F800000u && a > m ? a : m;
  }
  return m;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_xor(v, d);
    v = v > o ? v : o;
  }
  return v;
}
// The power of two of a token whose largest |x| has these bits: it goes to
// [2^14, 2^15), or with the transform, whose sums of 16 values / 4 reach four
// times as far, to [2^12, 2^13).  Kept to normal factors.
__device__ __forceinline__ int shift_of(uint32_t bits, bool rht) {
  if (bits == 0) return 0;
  const int s = (rht ? 12 : 14) + 127 - (int)(bits >> 23);
  return s > 126 ? 126 : s;
}

// 16 values to the parts' pieces.  MX: bf16 parts cut from the front (8 bits
// each, three hold all 24); else fp16, the second part what the first's rounding
// left (what is left of 24 bits, 22 kept).  The remainder of a non-finite value
// counts as zero.
template <bool MX, int PARTS>
__device__ __forceinline__ void store_parts(const float v[16], uint16_t* xp, int64_t k, int TP, int t) {
  const int64_t c = k / kMvChunk;
  const int g = (int)(k % kMvChunk) / 32, i0 = (int)(k % 32) / 8;
  float r[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) r[j] = v[j];
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t b[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = r[8 * h + 2 * j + e];
          float kept;
          if (MX) {
            const uint32_t top = x == x ? __float_as_uint(x) & 0xFFFF0000u : 0x7FC00000u;
            b[e] = top >> 16;
            kept = __uint_as_float(top);
          } else {
            const _Float16 f = (_Float16)x;
            b[e] = __builtin_bit_cast(uint16_t, f);
            kept = (float)f;
          }
          const float left = x - kept;
          x = fabsf(kept) <= 3.0e38f || MX ? (left == left ? left : 0.0f) : 0.0f;
        }
        w[j] = b[0] | (b[1] << 16);
      }
      reinterpret_cast<v32x4*>(xp)[piece_at(c, i0 + h, PARTS, q, g, TP, t)] = v32x4{w[0], w[1], w[2], w[3]};
    }
  }
}

template <bool MX, int PARTS>
__device__ __forceinline__ void prepare_block(const MatvecParams& p, int64_t t, int64_t k, int shift, uint16_t* xp, int TP,
                                              int at) {
  float v[16];
  load_block(p, t, k, v);
  if (!MX) {
    const float f = pow2f(shift);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= f;
  }
  if (p.rht) {
    fwht16_inlane(v, p.sg);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= p.sg.fin;
  }
  store_parts<MX, PARTS>(v, xp, k, TP, at);
}

// One workgroup a token of a whole number of 16; the last ones are zeros.
template <bool MX, int PARTS>
__global__ __launch_bounds__(1024) void ufp4_matvec_prepare_kernel(MatvecParams p) {
  __shared__ uint32_t top;
  const int64_t t = blockIdx.x, K = (p.K + kMvChunk - 1) / kMvChunk * kMvChunk;
  int shift = 0;
  if (!MX) {
    if (threadIdx.x == 0) top = 0;
    __syncthreads();
    uint32_t m = 0;
    for (int64_t k = threadIdx.x * 16; k < p.K; k += blockDim.x * 16) {
      float v[16];
      load_block(p, t, k, v);
      const uint32_t b = block_max(v);
      m = m > b ? m : b;
    }
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) atomicMax(&top, m);
    __syncthreads();
    shift = shift_of(top, p.rht);
  }
  if (threadIdx.x == 0 && t < p.tokens) p.shift[t] = shift;
  uint16_t* xp = p.xp + (size_t)(t / 16) * (K / kMvChunk) * PARTS * 16 * kMvChunk;
  for (int64_t k = threadIdx.x * 16; k < K; k += blockDim.x * 16)
    prepare_block<MX, PARTS>(p, t, k, shift, xp, 16, (int)(t % 16));
}

// ---------------------------------------------------------------- weights
// Eight codes under the scale 2^e (as a float) to four bf16 pairs, exact.
template <int GRID>
__device__ __forceinline__ void expand8_mx(uint32_t w, float scale, uint32_t out[4]) {
  if (GRID == kGridE2M1) {
    out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    out[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    out[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    out[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    return;
  }
  // E4M3 encodings of the magnitudes by index, then the hardware conversion
  if (GRID == kGridINT4) w = signmag8(w);
  const uint32_t lo = GRID == kGridE1M2 ? 0x3C383000u : 0x44403800u, hi = GRID == kGridE1M2 ? 0x46444240u : 0x4E4C4A48u;
  const uint32_t he = __builtin_amdgcn_perm(hi, lo, w & 0x07070707u) | ((w << 4) & 0x80808080u);
  const uint32_t ho = __builtin_amdgcn_perm(hi, lo, (w >> 4) & 0x07070707u) | (w & 0x80808080u);
  const int a = (int)__builtin_amdgcn_perm(ho, he, 0x05010400u), b = (int)__builtin_amdgcn_perm(ho, he, 0x07030602u);
  out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false));
  out[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true));
  out[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false));
  out[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true));
}

// 32 codes of a row and their scale bytes.
struct Granule {
  v32x4 c;
  uint32_t s;
};
template <bool MX>
__device__ __forceinline__ Granule load_granule(const uint8_t* codes, const uint8_t* scales, int64_t k, bool in) {
  Granule w{v32x4{0u, 0u, 0u, 0u}, 0u};
  if (in) {
    w.c = *reinterpret_cast<const v32x4*>(codes + k / 2);
    w.s = MX ? (uint32_t)scales[k / 32] : (uint32_t)*reinterpret_cast<const uint16_t*>(scales + k / 16);
  }
  return w;
}
template <int GRID, bool MX>
__device__ __forceinline__ void expand_granule(const Granule& w, v32x4 f[4]) {
  if (MX) {
    const float scale = __uint_as_float(w.s << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t e[4];
      expand8_mx<GRID>(w.c[i], scale, e);
      f[i] = v32x4{e[0], e[1], e[2], e[3]};
    }
  } else {
    const f16x2 ds = expand_scales<GRID>(w.s & 0x7F7Fu);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t e[4];
      expand8_shifted<GRID>(w.c[i], i < 2 ? f16x2{ds.x, ds.x} : f16x2{ds.y, ds.y}, e);
      f[i] = v32x4{e[0], e[1], e[2], e[3]};
    }
  }
}
template <bool MX>
__device__ __forceinline__ f32x4 mfma(v32x4 a, v32x4 b, f32x4 c) {
  if (MX)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Four neighbouring values of a row of y, n of them inside it.
__device__ __forceinline__ void store_y(const MatvecParams& p, int64_t at, const f32x4& v, int64_t n) {
  if (p.y_f32) {
    float* y = static_cast<float*>(p.y) + at;
    if (n >= 4) {
      store_16(y, v32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
    } else {
      for (int i = 0; i < n; ++i) y[i] = v[i];
    }
  } else {
    uint16_t* y = static_cast<uint16_t*>(p.y) + at;
    const v32x2 w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    if (n >= 4) store_8(y, w);
    else tail_store(y, v32x4{w.x, w.y, 0u, 0u}, (int)n);
  }
}

// Rows of w in tiles of 16, walked over by the workgroups; a tile's values of K
// are split over the waves, whose sums meet in LDS.  LDSX: up to four tokens,
// prepared by every workgroup; else 16 NT of the tokens the kernel above prepared.
template <int GRID, bool MX, int PARTS, int NT, bool LDSX>
__global__ __launch_bounds__(kMvThreads) void ufp4_matvec_kernel(MatvecParams p) {
  extern __shared__ v32x4 xs[];
  __shared__ f32x4 part[2][kMvWaves][NT][64];
  __shared__ uint32_t top[kLdsTokens];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int chunks = (int)((p.K + kMvChunk - 1) / kMvChunk);
  const int64_t t0 = (int64_t)blockIdx.y * 16 * NT;
  const int TP = LDSX ? (int)p.tokens : 16;
  if (LDSX) {
    if (!MX) {
      if (tid < kLdsTokens) top[tid] = 0;
      __syncthreads();
      for (int t = 0; t < TP; ++t) {
        uint32_t m = 0;
        for (int64_t k = tid * 16; k < p.K; k += kMvThreads * 16) {
          float v[16];
          load_block(p, t, k, v);
          const uint32_t b = block_max(v);
          m = m > b ? m : b;
        }
        m = wave_max(m);
        if (lane == 0) atomicMax(&top[t], m);
      }
      __syncthreads();
    }
    for (int t = 0; t < TP; ++t)
      for (int64_t k = tid * 16; k < (int64_t)chunks * kMvChunk; k += kMvThreads * 16)
        prepare_block<MX, PARTS>(p, t, k, MX ? 0 : shift_of(top[t], p.rht), reinterpret_cast<uint16_t*>(xs), TP, t);
    __syncthreads();
  }
  const v32x4* xf[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (LDSX) {
      xf[n] = xs + g * TP + (r < TP ? r : TP - 1);
    } else {
      // past the last token's sixteen: any sixteen, whose results are not stored
      const int64_t t16 = (t0 / 16 + n) * 16 < p.tokens ? t0 / 16 + n : t0 / 16;
      xf[n] = reinterpret_cast<const v32x4*>(p.xp) + (size_t)t16 * chunks * PARTS * 4 * 64 + g * 16 + r;
    }
  }
  constexpr float kUnshift = MX ? 1.0f : (float)(1 << kExpandShift<GRID>);
  const int64_t tiles = (p.N + 15) / 16;
  int buf = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    const int64_t row = tile * 16 + r < p.N ? tile * 16 + r : p.N - 1;
    const uint8_t* codes = p.codes + row * (p.K / 2);
    const uint8_t* scales = p.scales + row * (p.K / (MX ? 32 : 16));
    f32x4 acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = wave; c < chunks; c += kMvWaves) {
      const int64_t k = (int64_t)c * kMvChunk + 32 * g;
      v32x4 f[4];
      expand_granule<GRID, MX>(load_granule<MX>(codes, scales, k, k < p.K), f);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < PARTS; ++q) acc[n] = mfma<MX>(f[i], xf[n][((size_t)c * 4 + i) * PARTS * 4 * TP + q * 4 * TP], acc[n]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) part[buf][wave][n][lane] = acc[n];
    __syncthreads();
    if (wave < NT) {
      f32x4 v = part[buf][0][wave][lane];
#pragma unroll
      for (int w = 1; w < kMvWaves; ++w) v += part[buf][w][wave][lane];
      // a lane holds token r of the 16 and four neighbouring rows of w
      const int64_t t = t0 + 16 * wave + r, n = tile * 16 + 4 * g;
      if (t < p.tokens && n < p.N) {
        const int shift = MX || p.K == 0 ? 0 : LDSX ? shift_of(top[r], p.rht) : p.shift[t];
        // in 64 bits: neither factor alone has to be in fp32's range
        const double s = pow2d(-shift) * (double)kUnshift * (MX || p.K == 0 ? 1.0 : (double)p.ts[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)((double)v[i] * s);
        store_y(p, t * p.ldy + n, v, p.N - n);
      }
    }
  }
}

template <int GRID, bool MX, int PARTS>
hipError_t launch_grid(const MatvecParams& p, hipStream_t s) {
  const int64_t tiles = (p.N + 15) / 16;
  const unsigned gx = (unsigned)(tiles < 1024 ? tiles : 1024);
  if (matvec_in_lds(p.tokens, p.K, PARTS)) {
    const size_t lds = (size_t)((p.K + kMvChunk - 1) / kMvChunk) * kMvChunk * p.tokens * PARTS * 2;
    ufp4_matvec_kernel<GRID, MX, PARTS, 1, true><<<gx, kMvThreads, lds, s>>>(p);
    return hipGetLastError();
  }
  const unsigned t16 = (unsigned)((p.tokens + 15) / 16);
  if (p.K > 0) {
    ufp4_matvec_prepare_kernel<MX, PARTS><<<16 * t16, 1024, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (t16 == 1) ufp4_matvec_kernel<GRID, MX, PARTS, 1, false><<<gx, kMvThreads, 0, s>>>(p);
  else if (t16 == 2) ufp4_matvec_kernel<GRID, MX, PARTS, 2, false><<<gx, kMvThreads, 0, s>>>(p);
  else ufp4_matvec_kernel<GRID, MX, PARTS, 4, false><<<dim3(gx, (t16 + 3) / 4), kMvThreads, 0, s>>>(p);
  return hipGetLastError();
}

template <bool MX, int PARTS>
hipError_t launch_parts(const MatvecParams& p, hipStream_t s) {
  switch (p.grid) {
    case kGridE1M2: return launch_grid<kGridE1M2, MX, PARTS>(p, s);
    case kGridINT4: return launch_grid<kGridINT4, MX, PARTS>(p, s);
    case kGridE2M1:  // the clamped grid's codes are E2M1 codes
    case kGridE2M1C: return launch_grid<kGridE2M1, MX, PARTS>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

bool matvec_in_lds(int64_t tokens, int64_t K, int parts) {
  if (tokens > kLdsTokens) return false;
  const int64_t padded = (K + kMvChunk - 1) / kMvChunk * kMvChunk;
  return padded * tokens * parts * 2 <= (int64_t)kLdsX;
}

hipError_t launch_matvec(const MatvecParams& p, hipStream_t s) {
  const int parts = matvec_parts(p.mx, p.rht, p.x_f32, p.y_f32);
  if (p.mx) return parts == 1 ? launch_parts<true, 1>(p, s) : launch_parts<true, 3>(p, s);
  return parts == 1 ? launch_parts<false, 1>(p, s) : launch_parts<false, 2>(p, s);
}

}  // namespace ufp4
