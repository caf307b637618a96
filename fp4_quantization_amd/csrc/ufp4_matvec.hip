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
//
// Bound by reading the weights.  One token, kernel times: 65536 x 8192 (302 MB) 63 to
// 65 us, 4.7 TB/s, where reading alone takes 48; 4096 x 4096 7.5, reading alone 5.9
// with its launch.  16 tokens, 16384 x 4096: 11.9, and 4 for x'.
#include "ufp4_expand.hpp"
#include "ufp4_serve.hpp"
#include "ufp4_vec.hpp"

namespace ufp4 {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kMvThreads = 64 * kMvWaves;

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
__device__ __forceinline__ void prepare_block(const MatvecParams& p, float v[16], int64_t k, int shift, uint16_t* xp, int TP,
                                              int at) {
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

// blockIdx.x: a token of a whole number of 16 (the last ones are zeros); blockIdx.y:
// a part of its values, after the token's maximum, which every part finds itself.
constexpr int kPrepareThreads = 256;
template <bool MX, int PARTS>
__global__ __launch_bounds__(kPrepareThreads) void ufp4_matvec_prepare_kernel(MatvecParams p) {
  __shared__ uint32_t top[kPrepareThreads / 64];
  const int64_t t = blockIdx.x, K = (p.K + kMvChunk - 1) / kMvChunk * kMvChunk;
  int shift = 0;
  if (!MX) {
    uint32_t m = 0;
    for (int64_t k = threadIdx.x * 16; k < p.K; k += kPrepareThreads * 16) {
      float v[16];
      load_block(p, t, k, v);
      const uint32_t b = block_max(v);
      m = m > b ? m : b;
    }
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPrepareThreads / 64; ++w) m = m > top[w] ? m : top[w];
    shift = shift_of(m, p.rht);
  }
  if (threadIdx.x == 0 && blockIdx.y == 0 && t < p.tokens) p.shift[t] = shift;
  uint16_t* xp = p.xp + (size_t)(t / 16) * (K / kMvChunk) * PARTS * 16 * kMvChunk;
  for (int64_t k = (blockIdx.y * kPrepareThreads + threadIdx.x) * 16; k < K; k += (int64_t)gridDim.y * kPrepareThreads * 16)
  {
    float v[16];
    load_block(p, t, k, v);
    prepare_block<MX, PARTS>(p, v, k, shift, xp, 16, (int)(t % 16));
  }
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

// A lane's part of a segment of up to kSegment chunks of 128 values, of row r: 32 codes
// of each chunk (those of its group g), and the scales of all groups of chunk g,
// which one load of 8 (MX32: 4) bytes brings where loads of 2 (1) for each chunk
// took 10 of 71 us (65536 x 8192).  Where a row's scales are not whole words (APART)
// they are loaded for each chunk all the same: the last word would lie half behind
// the array.
struct Segment {
  v32x4 c[kSegment];
  uint32_t s[kSegment];
};
// Up to 16 rows of w from row `row` on; what lies past them (or past the end of a
// row, by an offset of kOutside) reads as zeros.
constexpr uint32_t kOutside = 0x80000000u;
struct Rows {
  __amdgpu_buffer_rsrc_t codes, scales;
};
template <bool MX>
__device__ __forceinline__ Rows rows_of(const MatvecParams& p, int64_t row) {
  const int64_t left = p.N - row;
  const uint32_t n = left <= 0 ? 0u : left < 16 ? (uint32_t)left : 16u;
  const int64_t at = n ? row * p.K : 0;
  const uint32_t values = n * (uint32_t)p.K;
  // word 3: 32-bit data, raw addressing
  return Rows{__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.codes + at / 2), 0, (int)(values / 2), 0x00020000),
              __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.scales + at / (MX ? 32 : 16)), 0,
                                                (int)(values / (MX ? 32 : 16)), 0x00020000)};
}
// The scales of this lane's codes in chunks 0 .. 3: the 4 x 4 transposition over the
// lane groups of what they loaded.  NV16: two bytes each (low half of s[i]).
template <bool MX, bool APART>
__device__ __forceinline__ void own_scales(const Segment& w, int g, uint32_t (&s)[kSegment]) {
  if (APART) {
#pragma unroll
    for (int j = 0; j < kSegment; ++j) s[j] = w.s[j];
  } else if (MX) {
    const auto h = __builtin_amdgcn_permlane32_swap(w.s[0], w.s[0], false, false);  // chunk g & 1, and 2 more
    const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    s[0] = (a[0] >> (8 * g)) & 0xFFu;
    s[1] = (a[1] >> (8 * g)) & 0xFFu;
    s[2] = (b[0] >> (8 * g)) & 0xFFu;
    s[3] = (b[1] >> (8 * g)) & 0xFFu;
  } else {
    // groups g & 2 and its next of the chunks g & 1 (h[0]) and (g & 1) + 2 (h[1])
    const auto h = __builtin_amdgcn_permlane32_swap(w.s[0], w.s[1], false, false);
    const uint32_t even = __builtin_amdgcn_perm(h[1], h[0], 0x05040100u), odd = __builtin_amdgcn_perm(h[1], h[0], 0x07060302u);
    const auto o = __builtin_amdgcn_permlane16_swap(even, odd, false, false);
    s[0] = o[0];
    s[1] = o[1];
    s[2] = o[0] >> 16;
    s[3] = o[1] >> 16;
  }
}
// 32 codes and their scale bytes as four fragments.
template <int GRID, bool MX>
__device__ __forceinline__ void expand_granule(const v32x4& c, uint32_t s, v32x4 f[4]) {
  if (MX) {
    const float scale = __uint_as_float(s << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t e[4];
      expand8_mx<GRID>(c[i], scale, e);
      f[i] = v32x4{e[0], e[1], e[2], e[3]};
    }
  } else {
    const f16x2 ds = expand_scales<GRID>(s & 0x7F7Fu);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t e[4];
      expand8_shifted<GRID>(c[i], i < 2 ? f16x2{ds.x, ds.x} : f16x2{ds.y, ds.y}, e);
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

// Rows of w in tiles of 16, walked over by the workgroups.  kw of the eight waves
// share a tile's chunks of K, and their sums meet in LDS; 8 / kw tiles side by side.
// A wave's weights are loaded a segment (four chunks) ahead of their use, the first
// ones before x' is prepared.
template <int GRID, bool MX, int PARTS, int NT, XSource X, bool APART>
__global__ __launch_bounds__(kMvThreads, X == kXRegisters ? 2 : 4) void ufp4_matvec_kernel(MatvecParams p, int log_kw) {
  extern __shared__ v32x4 xs[];
  __shared__ f32x4 part[2][kMvWaves][NT][64];
  __shared__ uint32_t top[kLdsTokens];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int chunks = (int)((p.K + kMvChunk - 1) / kMvChunk);
  const int kw = 1 << log_kw, wk = wave & (kw - 1), wt = wave >> log_kw, side = kMvWaves >> log_kw;
  const int segments = chunks > 0 ? (chunks + kSegment * kw - 1) / (kSegment * kw) : 1;
  // neighbouring chunks of a wave's segment: 256 bytes of each row together
  const int run = chunks < kSegment * kw ? (chunks + kw - 1) >> log_kw : kSegment;
  auto chunk_of = [&](int segment, int j) { return j < run ? segment * kSegment * kw + wk * run + j : chunks; };
  const int64_t t0 = (int64_t)blockIdx.y * 16 * NT;
  const int TP = X == kXLds ? (int)p.tokens : 16;
  const int tiles = (int)((p.N + 15) / 16), groups = (tiles + side - 1) / side;

  // this wave's weights of a segment, row r of a tile
  auto fetch = [&](int group, int segment, Segment& w) {
    const Rows rows = rows_of<MX>(p, ((int64_t)group * side + wt) * 16);
    const uint32_t line = (uint32_t)r * (uint32_t)p.K;
#pragma unroll
    for (int j = 0; j < kSegment; ++j) {
      const uint32_t k = (uint32_t)chunk_of(segment, j) * kMvChunk + 32 * g;
      w.c[j] = __builtin_bit_cast(v32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             rows.codes, (int)(k < (uint32_t)p.K ? (line + k) / 2 : kOutside), 0, 0));
    }
    if (APART) {
#pragma unroll
      for (int j = 0; j < kSegment; ++j) {
        const uint32_t k = (uint32_t)chunk_of(segment, j) * kMvChunk + 32 * g;
        w.s[j] = MX ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rows.scales, (int)(k < (uint32_t)p.K ? (line + k) / 32 : kOutside), 0, 0)
                    : (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rows.scales, (int)(k < (uint32_t)p.K ? (line + k) / 16 : kOutside), 0, 0);
      }
      return;
    }
    const uint32_t k = (uint32_t)(segment * kSegment * kw + wk * run + g) * kMvChunk;
    const bool in = g < run && k < (uint32_t)p.K;
    if (MX) {
      w.s[0] = __builtin_amdgcn_raw_buffer_load_b32(rows.scales, (int)(in ? (line + k) / 32 : kOutside), 0, 0);
    } else {
      const v32x2 x = __builtin_bit_cast(v32x2, __builtin_amdgcn_raw_buffer_load_b64(rows.scales, (int)(in ? (line + k) / 16 : kOutside), 0, 0));
      w.s[0] = x.x;
      w.s[1] = x.y;
    }
  };
  // position (tile group and segment) of the next load.  Behind the last group
  // nothing is read, without a branch: the compiler would wait for all loads where
  // some may not have been made.
  int load_group = blockIdx.x, load_segment = 0;
  auto fetch_next = [&](Segment& w) {
    fetch(load_group, load_segment, w);
    const bool last = load_segment + 1 == segments;
    load_segment = last ? 0 : load_segment + 1;
    load_group += last ? (int)gridDim.x : 0;
  };
  Segment wa, wb;
  if (X == kXLds) {
    // blocks of 16 values: one a thread where that suffices, loaded ahead of the
    // first weights (loads return in order)
    const int blocks = chunks * (kMvChunk / 16), all = TP * blocks;
    float v[16];
    const int t1 = tid < all ? tid / blocks : 0, k1 = (tid - t1 * blocks) * 16;
    if (tid < all) load_block(p, t1, k1, v);
    fetch_next(wa);
    if (!MX) {
      if (tid < kLdsTokens) top[tid] = 0;
      __syncthreads();
      for (int i = tid; i < all; i += kMvThreads) {
        float u[16];
        const int t = i / blocks;
        if (i != tid) load_block(p, t, (i - t * blocks) * 16, u);
        const uint32_t m = block_max(i != tid ? u : v);
        // all lanes of a wave have one token where its blocks are a multiple of 64
        if (blocks % 64 == 0) {
          const uint32_t wm = wave_max(m);
          if (lane == 0) atomicMax(&top[t], wm);
        } else {
          atomicMax(&top[t], m);
        }
      }
      __syncthreads();
    }
    for (int i = tid; i < all; i += kMvThreads) {
      const int t = i / blocks, k = (i - t * blocks) * 16;
      if (i != tid) load_block(p, t, k, v);
      prepare_block<MX, PARTS>(p, v, k, MX ? 0 : shift_of(top[t], p.rht), reinterpret_cast<uint16_t*>(xs), TP, t);
    }
    __syncthreads();
  } else {
    fetch_next(wa);
  }
  fetch_next(wb);
  const v32x4* xf[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (X == kXLds) {
      xf[n] = xs + g * TP + (r < TP ? r : TP - 1);
    } else {
      // past the last token's sixteen: any sixteen, whose results are not stored
      const int64_t t16 = (t0 / 16 + n) * 16 < p.tokens ? t0 / 16 + n : t0 / 16;
      xf[n] = reinterpret_cast<const v32x4*>(p.xp) + (size_t)t16 * chunks * PARTS * 4 * 64 + g * 16 + r;
    }
  }
  auto piece = [&](int n, int c, int i, int q) { return xf[n][(((size_t)c * 4 + i) * PARTS + q) * 4 * TP]; };
  v32x4 xr[X == kXRegisters ? kSegment : 1][4];
  if (X == kXRegisters && chunks > 0) {  // (without chunks there is no x' to read)
#pragma unroll
    for (int j = 0; j < kSegment; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) xr[j][i] = piece(0, chunk_of(0, j) < chunks ? chunk_of(0, j) : 0, i, 0);
  }
  // what a sum is multiplied by, for each of this lane's tokens: in 64 bits, since
  // neither the token's power of two nor S alone has to be in fp32's range
  double factor[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t t = t0 + 16 * n + r;
    factor[n] = MX ? 1.0 : 0.0;
    if (!MX && t < p.tokens && p.K > 0) {
      const int shift = X == kXLds ? shift_of(top[r], p.rht) : p.shift[t];
      factor[n] = pow2d(-shift) * (double)(1 << kExpandShift<GRID>) * (double)p.ts[0];
    }
  }
  f32x4 acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int group = blockIdx.x, segment = 0, buf = 0;
  // multiplies the segment in x and has the one after the next loaded in its place
  auto step = [&](Segment& x) {
    uint32_t scales[kSegment];
    own_scales<MX, APART>(x, g, scales);
#pragma unroll
    for (int j = 0; j < kSegment; ++j) {
      const int c = chunk_of(segment, j);
      if (c >= chunks || group >= groups) break;
      v32x4 f[4];
      // (past the end of a row its scale bytes are the next row's)
      expand_granule<GRID, MX>(x.c[j], c * kMvChunk + 32 * g < (int)p.K ? scales[j] : 0u, f);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
            acc[n] = mfma<MX>(f[i], X == kXRegisters ? xr[X == kXRegisters ? j : 0][i] : piece(n, c, i, q), acc[n]);
    }
    fetch_next(x);
    const bool last = ++segment == segments;
    if (!last || group >= groups) return;
    // the tile's sums; a wave that has a tile of its own holds them already
    if (kw > 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n) part[buf][wave][n][lane] = acc[n];
      __syncthreads();
    }
    const int tile = group * side + wt;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      f32x4 v = acc[i];
      acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if ((i & (kw - 1)) != wk) continue;
      if (kw > 1) {
        v = part[buf][wt << log_kw][i][lane];
        for (int u = 1; u < kw; ++u) v += part[buf][(wt << log_kw) + u][i][lane];
      }
      // a lane holds token r of the 16 and four neighbouring rows of w
      const int64_t t = t0 + 16 * i + r, n = (int64_t)tile * 16 + 4 * g;
      if (t < p.tokens && n < p.N) {
        if (!MX) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (float)((double)v[e] * factor[i]);
        }
        store_y(p, t * p.ldy + n, v, p.N - n);
      }
    }
    segment = 0;
    group += gridDim.x;
    buf ^= 1;
  };
  // two at a time, without an exit in between: where it met the loop's, the compiler
  // would take each buffer's loads for the youngest and wait for both.  A step
  // behind the last one does nothing.
  const int steps = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x * segments;
  for (int i = 0; i < steps; i += 2) {
    step(wa);
    step(wb);
  }
}

template <int GRID, bool MX, int PARTS, bool APART>
hipError_t launch_apart(const MatvecParams& p, hipStream_t s) {
  const MatvecPlan m = matvec_plan(p.tokens, p.N, p.K, PARTS);
  const dim3 grid((unsigned)m.gx, (unsigned)m.gy);
  if (m.x == kXLds) {
    const size_t lds = (size_t)((p.K + kMvChunk - 1) / kMvChunk) * kMvChunk * p.tokens * PARTS * 2;
    ufp4_matvec_kernel<GRID, MX, PARTS, 1, kXLds, APART><<<grid, kMvThreads, lds, s>>>(p, m.log_kw);
    return hipGetLastError();
  }
  if (p.K > 0) {
    const int64_t parts = (p.K + 16 * kPrepareThreads - 1) / (16 * kPrepareThreads), t16 = (p.tokens + 15) / 16;
    ufp4_matvec_prepare_kernel<MX, PARTS><<<dim3((unsigned)(16 * t16), (unsigned)(parts < 8 ? parts : 8)), kPrepareThreads, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (m.x == kXRegisters) {
    if constexpr (PARTS == 1) ufp4_matvec_kernel<GRID, MX, PARTS, 1, kXRegisters, APART><<<grid, kMvThreads, 0, s>>>(p, m.log_kw);
  } else if (m.nt == 1) {
    ufp4_matvec_kernel<GRID, MX, PARTS, 1, kXMemory, APART><<<grid, kMvThreads, 0, s>>>(p, m.log_kw);
  } else if (m.nt == 2) {
    ufp4_matvec_kernel<GRID, MX, PARTS, 2, kXMemory, APART><<<grid, kMvThreads, 0, s>>>(p, m.log_kw);
  } else {
    ufp4_matvec_kernel<GRID, MX, PARTS, 4, kXMemory, APART><<<grid, kMvThreads, 0, s>>>(p, m.log_kw);
  }
  return hipGetLastError();
}

template <int GRID, bool MX, int PARTS>
hipError_t launch_grid(const MatvecParams& p, hipStream_t s) {
  return p.K % (MX ? 128 : 64) ? launch_apart<GRID, MX, PARTS, true>(p, s) : launch_apart<GRID, MX, PARTS, false>(p, s);
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

bool matvec_in_lds(int64_t tokens, int64_t K, int parts) { return matvec_fits_lds(tokens, K, parts); }

hipError_t launch_matvec(const MatvecParams& p, hipStream_t s) {
  const int parts = matvec_parts(p.mx, p.rht, p.x_f32, p.y_f32);
  if (p.mx) return parts == 1 ? launch_parts<true, 1>(p, s) : launch_parts<true, 3>(p, s);
  return parts == 1 ? launch_parts<false, 1>(p, s) : launch_parts<false, 2>(p, s);
}

}  // namespace ufp4
