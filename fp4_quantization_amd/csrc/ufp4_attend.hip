// ufp4_attend.hip -- attention of each sequence's drafted tokens over the 4-bit
// key-value cache.
//
// A wave takes 32 tokens of one sequence and key head at a time, and 16 R rows
// (drafted tokens x the query heads that share the key head):
//   S^T = K Q^T   two MFMA tiles of 16 tokens; the token of a tile's row is
//                 chosen so that lane (column q, group g) ends up with the logits
//                 of row q and the tokens 8 g .. 8 g + 7;
//   softmax       one pass, running maximum and sum per row (a column of lanes);
//   O^T += V^T P^T  the lane's eight weights are its fragment of P^T as they are;
//                 a lane's fragment of V^T is one pair of values of eight
//                 neighbouring tokens, eight bytes of the cache's value layout.
// So nothing is exchanged between lanes but the maxima, and codes go from memory
// to registers to the MFMA.  fp16 holds code times E4M3 scale exactly
// (ufp4_expand.hpp); head scales, softmax scale and each row's power of two are
// applied to fp32 logits and sums.
//
// Work is counted in steps of 128 tokens (a tile of 32 for each of four waves) of
// one unit, that is a sequence, key head and tile of rows.  All units' steps in a
// row are cut into equal runs, one a workgroup, from the lengths, on the device: a
// batch of any lengths fills the device evenly, and the launch does not depend on
// them.  A workgroup answers the units that lie inside its run itself; a unit that
// crosses into other runs leaves partial results in the workspace (at most two a
// workgroup), which a second kernel joins.
//
// Measured: 64 sequences of up to 16384 tokens, 8 x 4 heads of 128 (605 MB) 180 to
// 185 us, 3.4 TB/s: vector work half of the time, mostly the expansion (about 390
// instructions a tile), loads waited for a third.  2 of 131072, 32 rows, heads of 256
// (302 MB): 137 and 15 for the join.
#include "ufp4_expand.hpp"
#include "ufp4_serve.hpp"
#include "ufp4_vec.hpp"

namespace ufp4 {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAtWaves = 4, kAtThreads = 64 * kAtWaves;
// Waves a SIMD holds of the kernel, which gives a wave 256 registers or 512.
constexpr int attend_waves(int dt, int r) { return dt > 128 ? (r > 1 ? 1 : 2) : (r > 1 ? 2 : 3); }
constexpr int kStep = 32 * kAtWaves;  // tokens
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
// Softmax weights enter the second product as fp16, in units that bring the largest, 1,
// to 2^15: fp16's 11 bits hold down to 2^-29 of it, and a weight is lost below 2^-40.
// (As they are, at most 1, the cut is at 2^-25: of 131072 tokens that one other exceeds
// by 18 in their logits, those of its wave were lost, a quarter of them.)  The factor is
// exact, and no time is measured for it.
constexpr float kWeightUnit = 32768.0f;

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ double pow2d(int e) { return __longlong_as_double((long long)(e + 1023) << 52); }
__device__ __forceinline__ float head_scale(const float* ts, int h) {
  const float s = ts ? ts[h] : 1.0f;
  return s > 0.0f && s <= 3.40282347e38f ? s : 1.0f;
}

// ---------------------------------------------------------------- the runs
struct Sequence {
  int64_t row0;  // of q
  int32_t n;     // drafted tokens
  int32_t rows;  // to compute: drafted tokens up to max_draft, times group
  int32_t len;   // tokens in the cache
};
__device__ __forceinline__ Sequence sequence_of(const AttendParams& p, int b) {
  const int64_t r0 = p.q_offsets[b], r1 = p.q_offsets[b + 1];
  const int len = p.lengths[b];
  const int64_t most = p.ld_pages * p.c.page_tokens;
  Sequence s{r0, 0, 0, 0};
  if (r0 < 0 || r1 < r0 || r1 > p.q_rows) return s;
  s.n = (int32_t)(r1 - r0);
  s.rows = (s.n < p.max_draft ? s.n : p.max_draft) * p.group;
  s.len = len < 0 ? 0 : (len > most ? (int32_t)most : len);
  return s;
}
// Steps of one unit of a sequence: one at least, so that a sequence without tokens
// is answered too.
__device__ __forceinline__ int unit_steps(const Sequence& s) { return s.len > kStep ? (s.len + kStep - 1) / kStep : 1; }
template <int ROWS>
__device__ __forceinline__ int units_of(const AttendParams& p, const Sequence& s) {
  return (s.rows + ROWS - 1) / ROWS * p.c.heads;
}

// A workgroup's run of steps, and the sequence that it begins in.
struct Run {
  int64_t lo, hi;  // steps
  int64_t each;    // steps a run
  int64_t first;   // the sequence's first step
  int32_t b;
};
template <int ROWS>
__device__ Run run_of(const AttendParams& p, int64_t* sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // sums of up to 256 sequences' steps are kept for the search; more are read again
  int64_t mine = 0, total = 0;
  for (int b = tid; b < p.sequences; b += kAtThreads) {
    const Sequence s = sequence_of(p, b);
    const int64_t n = (int64_t)unit_steps(s) * units_of<ROWS>(p, s);
    if (b < kAtThreads) mine = n;
    total += n;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
  if (lane == 0) sh[wave] = total;
  if (tid == 0) sh[kAtWaves] = -1;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kAtWaves; ++w) total += sh[w];
  Run r;
  r.each = (total + gridDim.x - 1) / gridDim.x;
  if (r.each < 1) r.each = 1;
  r.lo = blockIdx.x * r.each;
  r.hi = r.lo + r.each < total ? r.lo + r.each : total;
  r.b = -1;
  r.first = 0;
  if (r.lo >= r.hi) return r;
  int64_t before = 0;
  for (int b0 = 0; b0 < p.sequences; b0 += kAtThreads) {
    if (b0 > 0) {
      const Sequence s = sequence_of(p, b0 + tid < p.sequences ? b0 + tid : 0);
      mine = b0 + tid < p.sequences ? (int64_t)unit_steps(s) * units_of<ROWS>(p, s) : 0;
    }
    int64_t inc = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    __syncthreads();
    if (lane == 63) sh[wave] = inc;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < kAtWaves; ++w) {
      if (w < wave) inc += sh[w];
      all += sh[w];
    }
    const int64_t at = before + inc - mine;
    if (r.lo >= at && r.lo < at + mine) {
      sh[kAtWaves] = b0 + tid;
      sh[kAtWaves + 1] = at;
    }
    __syncthreads();
    if (sh[kAtWaves] >= 0) {
      r.b = (int)sh[kAtWaves];
      r.first = sh[kAtWaves + 1];
      return r;
    }
    before += all;
  }
  return r;
}

// Largest of the four lane groups' values of a column.
__device__ __forceinline__ float max_of_groups(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// ---------------------------------------------------------------- values
// Bytes of four neighbouring tokens (one pair of values each) to fp16 pairs of
// neighbouring tokens, times the tokens' scales: the pairs' first values, then
// their second ones, both shifted as expand8_shifted does.
template <int GRID>
__device__ __forceinline__ void expand_tokens(uint32_t w, f16x2 s01, f16x2 s23, uint32_t first[2], uint32_t second[2]) {
  f16x2 v[4];
  if (GRID == kGridINT4) {
    const uint32_t he = ((w << 4) & 0xF0F0F0F0u) ^ 0x80808080u, ho = (w & 0xF0F0F0F0u) ^ 0x80808080u;
    const _Float16 eight = (_Float16)(-1.0f / 131072.0f);  // -8 2^-20
    const f16x2 o01 = s01 * f16x2{eight, eight}, o23 = s23 * f16x2{eight, eight};
    v[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, he, 0x0C010C00u));
    v[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, he, 0x0C030C02u));
    v[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, ho, 0x0C010C00u));
    v[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, ho, 0x0C030C02u));
    first[0] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v[0], s01, o01));
    first[1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v[1], s23, o23));
    second[0] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v[2], s01, o01));
    second[1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v[3], s23, o23));
    return;
  }
  if (GRID == kGridE2M1 || GRID == kGridE2M1C) {
    const uint32_t t0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
    const uint32_t t1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
    const uint32_t t2 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
    const uint32_t t3 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
    v[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(t1, t0, 0x05040100u));
    v[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(t3, t2, 0x05040100u));
    v[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(t1, t0, 0x07060302u));
    v[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(t3, t2, 0x07060302u));
  } else {
    const uint32_t he = (w & 0x07070707u) | ((w << 4) & 0x80808080u);
    const uint32_t ho = ((w >> 4) & 0x07070707u) | (w & 0x80808080u);
    v[0] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, he, 0x010C000Cu));
    v[1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, he, 0x030C020Cu));
    v[2] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, ho, 0x010C000Cu));
    v[3] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0u, ho, 0x030C020Cu));
  }
  first[0] = __builtin_bit_cast(uint32_t, v[0] * s01);
  first[1] = __builtin_bit_cast(uint32_t, v[1] * s23);
  second[0] = __builtin_bit_cast(uint32_t, v[2] * s01);
  second[1] = __builtin_bit_cast(uint32_t, v[3] * s23);
}

template <int GRID>
__device__ __forceinline__ void scales_of(uint32_t four, f16x2& s01, f16x2& s23) {
  const float f = kExpandShift<GRID> ? 128.0f : 1.0f;
  s01 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)four, f, false);
  s23 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)four, f, true);
}

// ---------------------------------------------------------------- rows of q
// The folded signs of the transform (RhtSigns), in LDS: as scalars they would occupy
// 16 registers through the whole loop.
struct Signs {
  float q1[8], q2[4], q3[2], q4, fin;
};
// Sign j of the transform from its mask (bit j set: -1).
__device__ __forceinline__ float sign_of(uint32_t mask, int j) { return (mask >> j) & 1 ? -1.0f : 1.0f; }

// One wave's 16 rows of a tile as fp16 fragments in LDS (lane (r, g): dim DT / 4
// values of row r from g DT / 4 on): q times a power of two for the row that takes
// its largest magnitude to [2^12, 2^13) (its transform below 2^15), and with the
// transform a second part, what the first one's rounding left.  Returns the
// power's exponent.
template <int DT, int PARTS>
__device__ __forceinline__ int prepare_q(int dim, const Signs& S, const uint16_t* q, bool in, int lane,
                                         f16x8 (*to)[DT / 32][64]) {
  constexpr int N = DT / 4;
  const int g = lane >> 4;
  float v[N];
#pragma unroll
  for (int i = 0; i < N / 16; ++i) {
    const int d = g * N + 16 * i;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      V8 a{};
      if (in && d < dim) a = row_load(q + d + 8 * h, 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[16 * i + 8 * h + j] = a.v[j];
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t a = __float_as_uint(v[j]) & 0x7FFFFFFFu;
    m = a < 0x7F800000u && a > m ? a : m;
  }
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) {
    const uint32_t o = __shfl_xor(m, d);
    m = m > o ? m : o;
  }
  int shift = m ? 12 + 127 - (int)(m >> 23) : 0;
  if (shift > 126) shift = 126;
  const float f2 = __uint_as_float((uint32_t)(shift + 127) << 23);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] *= f2;
  if (PARTS == 2) {
    RhtSigns sg;
#pragma unroll
    for (int k = 0; k < 8; ++k) sg.q1[k] = S.q1[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) sg.q2[k] = S.q2[k];
    sg.q3[0] = S.q3[0];
    sg.q3[1] = S.q3[1];
    sg.q4 = S.q4;
    const float fin = S.fin;
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      fwht16_inlane(v + 16 * i, sg);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[16 * i + j] *= fin;
    }
  }
#pragma unroll
  for (int i = 0; i < DT / 32; ++i) {
    f16x8 hi, lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = v[8 * i + j];
      hi[j] = (_Float16)x;
      const float left = x - (float)hi[j];
      lo[j] = (_Float16)(left - left == 0.0f ? left : 0.0f);
    }
    to[0][i][lane] = hi;
    if (PARTS == 2) to[PARTS - 1][i][lane] = lo;
  }
  return shift;
}

// ---------------------------------------------------------------- results
// O of one row in the lane layout of the second product: the lane of group g has
// values 32 t + 8 g + j.  Inverse transform of the 16-block that lanes g and g ^ 1
// share: three stages in the lane, one across, 1/4, signs.
template <int NT>
__device__ __forceinline__ void untransform(uint32_t mask, float (&o)[NT][8], int g) {
  const uint32_t mine = mask >> (8 * (g & 1));
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float* v = o[t];
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(j & h)) {
          const float a = v[j], b = v[j + h];
          v[j] = a + b;
          v[j + h] = a - b;
        }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float other = __shfl_xor(v[j], 16);
      const float s = (g & 1) ? other - v[j] : v[j] + other;
      v[j] = s * (0.25f * sign_of(mine, j));
    }
  }
}

// A finished row: O / l, tensor scale, inverse transform, out and lse.
// The first value is column `col` of the head.
template <int NT>
__device__ __forceinline__ void finish_row(const AttendParams& p, float (&o)[NT][8], float m, float l, float vscale, bool in,
                                           int64_t row, int head, int col, int g) {
  const float f = l > 0.0f || l != l ? vscale / l : 0.0f;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) o[t][j] *= f;
  if (p.rht) untransform<NT>(p.signs, o, g);
  if (!in) return;
  uint16_t* out = p.out + row * p.ldo + (int64_t)head * p.c.dim + col + 8 * g;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (col + 32 * t < p.c.dim) {
      V8 a;
#pragma unroll
      for (int j = 0; j < 8; ++j) a.v[j] = o[t][j];
      store_16(out + 32 * t, pack(a));
    }
  }
  if (p.lse && col == 0 && g == 0)
    p.lse[row * p.q_heads + head] = l > 0.0f || l != l ? (m + __log2f(l)) * kLn2 : -__builtin_inff();
}

template <int GRID>
constexpr float unshift() { return (float)(1 << kExpandShift<GRID>); }

// ---------------------------------------------------------------- the kernel
// What a lane loads of a tile of 32 tokens: its parts of two keys (row r of the first
// product's two tiles of 16), and, 16 (or 4, 8) bytes a lane as they lie in memory,
// the scales of the keys and the values' codes and scales.  These three go through
// LDS, a wave its own, where lanes find the bytes they need: loading those from
// memory took twice as many, smaller loads.
template <int DT>
struct Tile {
  static constexpr int kWords = DT == 64 ? 2 : 4, kParts = (DT + 127) / 128, NT = DT / 32;
  uint32_t kc[2][kParts][kWords];
  v32x4 vc[NT / 2];
  uint32_t ks[kParts], vs[kParts];
};
template <int DT>
struct TileLds {
  v32x4 vc[DT];                                     // [pair of values][32 tokens], 16 DT bytes
  uint32_t vs[64 * ((DT + 127) / 128)], ks[64 * ((DT + 127) / 128)];  // [block][32], [token][block]
};
// A lane's byte offsets of key parts inside a tile.  FULL: dim is DT; else parts past
// dim get an offset that is outside every tile, and read as zeros.
template <int DT, bool FULL>
struct Offsets {
  static constexpr int kParts = Tile<DT>::kParts;
  uint32_t kc[FULL ? 1 : kParts];
  __device__ __forceinline__ Offsets(int dim, int g, int r) {
    const int tok = 8 * (r >> 2) + (r & 3);
#pragma unroll
    for (int c = 0; c < (FULL ? 1 : kParts); ++c) {
      const int d = g * (DT / 4) + 32 * c;
      kc[c] = FULL || d < dim ? (uint32_t)(tok * (FULL ? DT : dim) + d) / 2 : 0x80000000u;
    }
  }
};
// The tile whose first token has index `at` in its cache (page, head, token); !ok:
// nothing is read.
template <int DT, bool FULL>
__device__ __forceinline__ void load_tile(const AttendParams& p, int64_t at, bool ok, int lane, const Offsets<DT, FULL>& off,
                                          Tile<DT>& x) {
  const int half = FULL ? DT / 2 : p.c.dim / 2, blocks = FULL ? DT / 16 : p.c.dim / 16;
  const int bytes = ok ? kCacheTile * half : 0, sbytes = ok ? kCacheTile * blocks : 0;
  // word 3: 32-bit data, raw addressing
  const auto kc = __builtin_amdgcn_make_buffer_rsrc(p.c.kc + at * half, 0, bytes, 0x00020000);
  const auto ks = __builtin_amdgcn_make_buffer_rsrc(p.c.ks + at * blocks, 0, sbytes, 0x00020000);
  const auto vc = __builtin_amdgcn_make_buffer_rsrc(p.c.vc + at * half, 0, bytes, 0x00020000);
  const auto vs = __builtin_amdgcn_make_buffer_rsrc(p.c.vs + at * blocks, 0, sbytes, 0x00020000);
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int c = 0; c < Tile<DT>::kParts; ++c) {
      const int ko = (int)(FULL ? off.kc[0] + 16 * c + 4 * u * half : off.kc[FULL ? 0 : c]), k0 = FULL ? 0 : 4 * u * half;
      if constexpr (DT == 64) {
        const v32x2 w = __builtin_bit_cast(v32x2, __builtin_amdgcn_raw_buffer_load_b64(kc, ko, k0, 0));
        x.kc[u][c][0] = w.x;
        x.kc[u][c][1] = w.y;
      } else {
        const v32x4 w = __builtin_bit_cast(v32x4, __builtin_amdgcn_raw_buffer_load_b128(kc, ko, k0, 0));
#pragma unroll
        for (int j = 0; j < 4; ++j) x.kc[u][c][j] = w[j];
      }
    }
#pragma unroll
  for (int t = 0; t < DT / 64; ++t) x.vc[t] = __builtin_bit_cast(v32x4, __builtin_amdgcn_raw_buffer_load_b128(vc, 16 * lane + 1024 * t, 0, 0));
#pragma unroll
  for (int c = 0; c < Tile<DT>::kParts; ++c) {
    x.ks[c] = __builtin_amdgcn_raw_buffer_load_b32(ks, 4 * lane + 256 * c, 0, 0);
    x.vs[c] = __builtin_amdgcn_raw_buffer_load_b32(vs, 4 * lane + 256 * c, 0, 0);
  }
}
// Through a wave's LDS: what the wave writes here, it reads itself, in order; the
// barriers are the compiler's alone.
template <int DT>
__device__ __forceinline__ void stage_tile(const Tile<DT>& x, int lane, TileLds<DT>& to) {
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll
  for (int t = 0; t < DT / 64; ++t) to.vc[lane + 64 * t] = x.vc[t];
#pragma unroll
  for (int c = 0; c < Tile<DT>::kParts; ++c) {
    to.ks[lane + 64 * c] = x.ks[c];
    to.vs[lane + 64 * c] = x.vs[c];
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int GRID, int DT, int R, int PARTS, bool FULL>
__global__ __launch_bounds__(kAtThreads, attend_waves(DT, R)) void ufp4_attend_kernel(AttendParams p) {
  constexpr int ROWS = 16 * R, NT = DT / 32;
  constexpr int kPitch = DT + 4;
  // fragments of q that are few stay in registers, else they are read from LDS for
  // every two tiles of 16 tokens: a third wave a SIMD is worth more (batch of the head
  // comment: 213 us with two waves, 192 with three)
  constexpr bool kInLds = R * NT >= 4;
  __shared__ Signs S;
  __shared__ f16x8 ql[R][PARTS][NT][64];
  __shared__ int qshift[ROWS];
  __shared__ int64_t sh[kAtWaves + 2];
  __shared__ float ml[kAtWaves][2][ROWS];
  __shared__ float join[2][ROWS][kPitch];
  __shared__ TileLds<DT> staged[kAtWaves];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, g = lane >> 4, r = lane & 15;
  if (tid < 8) {
    const uint32_t m = p.signs;
    S.q1[tid] = sign_of(m, 2 * tid) * sign_of(m, 2 * tid + 1);
    if (tid < 4) S.q2[tid] = sign_of(m, 4 * tid) * sign_of(m, 4 * tid + 2);
    if (tid < 2) S.q3[tid] = sign_of(m, 8 * tid) * sign_of(m, 8 * tid + 4);
    if (tid == 0) {
      S.q4 = sign_of(m, 0) * sign_of(m, 8);
      S.fin = 0.25f * sign_of(m, 0);
    }
  }
  const Offsets<DT, FULL> off(p.c.dim, g, r);
  const Run run = run_of<ROWS>(p, sh);
  SplitUnit split{0, 0, 0, 0};
  int64_t lo = run.lo;
  int b = uniform(run.b);
  int64_t first = run.first;
  while (lo < run.hi) {
    const Sequence s = sequence_of(p, b);
    const int steps = unit_steps(s), units = units_of<ROWS>(p, s);
    if (lo >= first + (int64_t)steps * units) {  // behind this sequence
      first += (int64_t)steps * units;
      ++b;
      continue;
    }
    // units of a sequence: [head][tile of rows]
    const int unit = uniform((int)((lo - first) / steps)), tiles = units / p.c.heads;
    const int h = unit / tiles, tile = unit - h * tiles;
    const int64_t unit_lo = first + (int64_t)unit * steps;
    const int step0 = uniform((int)(lo - unit_lo));
    const int step1 = uniform((int)(run.hi < unit_lo + steps ? run.hi - unit_lo : steps));
    const int hist = s.len - s.n;  // below 0: drafted tokens that the cache does not hold
    const int32_t* table = p.table + b * p.ld_pages;

    f32x4 o[R][2 * NT];
    float mx[R], sum[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      mx[i] = -__builtin_inff();
      sum[i] = 0.0f;
#pragma unroll
      for (int t = 0; t < 2 * NT; ++t) o[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    const int blocks = FULL ? DT / 16 : p.c.dim / 16;
    // this wave's tiles: the next one is on its way while one is computed.  Their
    // pages are held 64 steps at a time, one a lane: a scalar load for each tile
    // would be waited for with every access to LDS, since the two share a counter
    // that scalar loads leave in any order.
    int pages_from = step0, pages = -1;
    auto load_pages = [&]() {
      const int t0 = (pages_from + lane) * kStep + 32 * wave;
      pages = pages_from + lane < step1 && t0 < s.len ? table[p.c.page.div((uint32_t)t0)] : -1;
    };
    load_pages();
    auto page_of = [&](int step) {
      if (step - pages_from >= 64) {
        pages_from = step;
        load_pages();
      }
      return __builtin_amdgcn_readlane(pages, step - pages_from);
    };
    auto fetch = [&](int step, int page, Tile<DT>& x) {
      const bool ok = page >= 0 && page < p.c.pages;
      const int t0 = step * kStep + 32 * wave;
      const int in_page = t0 - (int)p.c.page.div((uint32_t)t0) * p.c.page_tokens;
      load_tile<DT, FULL>(p, ok ? ((int64_t)page * p.c.heads + h) * p.c.page_tokens + in_page : 0, ok, lane, off, x);
      return ok;
    };
    Tile<DT> next;
    bool next_ok = fetch(step0, page_of(step0), next);

    // rows of q, by one wave for each 16
    if (wave < R) {
      const int m = tile * ROWS + 16 * wave + r;
      const bool in = m < s.rows;
      const uint16_t* q = p.q + (in ? (s.row0 + m / p.group) * p.ldq + (int64_t)(h * p.group + m % p.group) * p.c.dim : 0);
      const int shift = prepare_q<DT, PARTS>(p.c.dim, S, q, in, lane, ql[wave]);
      if (g == 0) qshift[16 * wave + r] = shift;
    }
    __syncthreads();
    f16x8 qf[kInLds ? 1 : R][PARTS][NT];
    float f[R];        // logits from sums, times log2 e
    int drafted[R];    // of this lane's row
    uint64_t bits[R];  // drafted tokens it sees
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int m = tile * ROWS + 16 * i + r;
      drafted[i] = m / p.group;
      f[i] = (float)(pow2d(-qshift[16 * i + r]) * (double)(unshift<GRID>() * kLog2e) * (double)p.scale *
                     (double)head_scale(p.c.kts, h));
      bits[i] = m < s.rows && p.mask ? p.mask[s.row0 + drafted[i]] : 0;
      if constexpr (!kInLds) {
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
#pragma unroll
          for (int t = 0; t < NT; ++t) qf[i][q][t] = ql[i][q][t][lane];
      }
    }

    for (int step = step0; step < step1; ++step) {
      const Tile<DT> x = next;
      const bool ok = next_ok;
      next_ok = fetch(step + 1, page_of(step + 1), next);
      if (!ok) continue;
      const int t0 = step * kStep + 32 * wave;
      stage_tile<DT>(x, lane, staged[wave]);
      const uint8_t* ks = reinterpret_cast<const uint8_t*>(staged[wave].ks) + (8 * (r >> 2) + (r & 3)) * blocks + g * (DT / 64);
      const uint8_t* vc = reinterpret_cast<const uint8_t*>(staged[wave].vc) + r * 32 + 8 * g;
      const uint8_t* vs = reinterpret_cast<const uint8_t*>(staged[wave].vs) + (r >> 3) * 32 + 8 * g;
      // ---- logits
      f32x4 a[R][2];
#pragma unroll
      for (int i = 0; i < R; ++i) a[i][0] = a[i][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < Tile<DT>::kParts; ++c) {
        f16x2 ds[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* from = ks + 4 * u * blocks + 2 * c;
          uint32_t two = DT == 64 ? (uint32_t)*from : (uint32_t)*reinterpret_cast<const uint16_t*>(from);
          if (!FULL && g * (DT / 4) + 32 * c >= p.c.dim) two = 0;
          ds[u] = expand_scales<GRID>(two & 0x7F7Fu);
        }
#pragma unroll
        for (int j = 0; j < Tile<DT>::kWords; ++j) {
          f16x8 kf[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t e[4];
            expand8_shifted<GRID>(x.kc[u][c][j], j < 2 ? f16x2{ds[u].x, ds[u].x} : f16x2{ds[u].y, ds[u].y}, e);
            kf[u] = __builtin_bit_cast(f16x8, g32x4{e[0], e[1], e[2], e[3]});
          }
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
              f16x8 y;
              if constexpr (kInLds) y = ql[i][q][4 * c + j][lane];
              else y = qf[i][q][4 * c + j];
#pragma unroll
              for (int u = 0; u < 2; ++u) a[i][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[u], y, a[i][u], 0, 0, 0);
            }
        }
      }
      // ---- softmax: this lane's tokens are t0 + 8 g + j
      const bool edge = t0 + 32 > hist;  // the wave's
      f16x8 pf[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = a[i][j >> 2][j & 3] * f[i];
        if (edge) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int t = t0 + 8 * g + j, d = t - hist;
            const bool chosen = p.mask ? (d < 64) & (int)((bits[i] >> (d & 63)) & 1) : d <= drafted[i];
            const bool seen = (t < s.len) & ((d < 0) | chosen);
            y[j] = seen ? y[j] : -__builtin_inff();
          }
        }
        float m = y[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) m = fmaxf(m, y[j]);
        m = fmaxf(max_of_groups(m), mx[i]);
        const float base = m == -__builtin_inff() ? 0.0f : m;
        const float alpha = __builtin_amdgcn_exp2f(mx[i] - base);
        float l = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float e = __builtin_amdgcn_exp2f(y[j] - base);
          l += e;
          pf[i][j] = (_Float16)(e * kWeightUnit);
        }
        sum[i] = sum[i] * alpha + l;
        if (__any(alpha != 1.0f)) {
#pragma unroll
          for (int t = 0; t < 2 * NT; ++t) o[i][t] *= alpha;
        }
        mx[i] = m;
      }
      // ---- values
      uint32_t keep0 = 0x7F7F7F7Fu, keep1 = 0x7F7F7F7Fu;
      if (edge) {
        // tokens that do not exist hold anything: their scales become 0
        const int left = s.len - t0 - 8 * g;
        if (left < 8) keep1 = left <= 4 ? 0u : keep1 >> (8 * (8 - left));
        if (left < 4) keep0 = left <= 0 ? 0u : keep0 >> (8 * (4 - left));
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (!FULL && 32 * t >= p.c.dim) break;
        const v32x2 codes = *reinterpret_cast<const v32x2*>(vc + 512 * t), scales = *reinterpret_cast<const v32x2*>(vs + 64 * t);
        f16x2 s01, s23, s45, s67;
        scales_of<GRID>(scales.x & keep0, s01, s23);
        scales_of<GRID>(scales.y & keep1, s45, s67);
        uint32_t v0[4], v1[4];
        expand_tokens<GRID>(codes.x, s01, s23, v0, v1);
        expand_tokens<GRID>(codes.y, s45, s67, v0 + 2, v1 + 2);
        const f16x8 even = __builtin_bit_cast(f16x8, g32x4{v0[0], v0[1], v0[2], v0[3]});
        const f16x8 odd = __builtin_bit_cast(f16x8, g32x4{v1[0], v1[1], v1[2], v1[3]});
#pragma unroll
        for (int i = 0; i < R; ++i) {
          o[i][2 * t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(even, pf[i], o[i][2 * t], 0, 0, 0);
          o[i][2 * t + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(odd, pf[i], o[i][2 * t + 1], 0, 0, 0);
        }
      }
    }

    // ---- the waves' results join: common maximum, then two and two
#pragma unroll
    for (int i = 0; i < R; ++i) {
      sum[i] += __shfl_xor(sum[i], 16);
      sum[i] += __shfl_xor(sum[i], 32);
      if (g == 0) {
        ml[wave][0][16 * i + r] = mx[i];
        ml[wave][1][16 * i + r] = sum[i];
      }
    }
    __syncthreads();
    float acc[R][NT][8];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float m = -__builtin_inff(), l = 0.0f;
#pragma unroll
      for (int k = 0; k < kAtWaves; ++k) m = fmaxf(m, ml[k][0][16 * i + r]);
      const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
      for (int k = 0; k < kAtWaves; ++k) l += ml[k][1][16 * i + r] * __builtin_amdgcn_exp2f(ml[k][0][16 * i + r] - base);
      const float alpha = __builtin_amdgcn_exp2f(mx[i] - base) * (1.0f / kWeightUnit);
      mx[i] = m;
      sum[i] = l;
      // values 32 t + 8 g + 2 k + parity, from row 4 g + k of the two tiles
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          acc[i][t][2 * k] = o[i][2 * t][k] * alpha;
          acc[i][t][2 * k + 1] = o[i][2 * t + 1][k] * alpha;
        }
    }
#pragma unroll
    for (int half = kAtWaves / 2; half >= 1; half >>= 1) {
      if (wave >= half && wave < 2 * half) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float* to = &join[wave - half][16 * i + r][32 * t + 8 * g];
#pragma unroll
            for (int j = 0; j < 8; j += 4) *reinterpret_cast<f32x4*>(to + j) = f32x4{acc[i][t][j], acc[i][t][j + 1], acc[i][t][j + 2], acc[i][t][j + 3]};
          }
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][t][j] += join[wave][16 * i + r][32 * t + 8 * g + j];
      }
      __syncthreads();
    }
    const bool whole = step0 == 0 && step1 == steps;
    if (wave == 0) {
      const float vscale = head_scale(p.c.vts, h) * unshift<GRID>();
      const int64_t slot = 2 * (int64_t)blockIdx.x + (step0 == 0 ? 1 : 0);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int m = tile * ROWS + 16 * i + r;
        if (whole) {
          finish_row<NT>(p, acc[i], mx[i], sum[i], vscale, m < s.rows, s.row0 + m / p.group, h * p.group + m % p.group, 0, g);
        } else {
          const int64_t at = slot * ROWS + 16 * i + r;
          if (g == 0) p.ml[at] = make_float2(mx[i], sum[i]);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (FULL || 32 * t < p.c.dim) {
              float* to = p.o + at * p.c.dim + 32 * t + 8 * g;
#pragma unroll
              for (int j = 0; j < 8; j += 4) *reinterpret_cast<f32x4*>(to + j) = f32x4{acc[i][t][j], acc[i][t][j + 1], acc[i][t][j + 2], acc[i][t][j + 3]};
            }
        }
      }
    }
    // the unit goes on in the runs behind this one
    if (!whole && step0 == 0) split = SplitUnit{b, h, tile, (int32_t)((unit_lo + steps - 1) / run.each - blockIdx.x + 1)};
    lo = unit_lo + step1;
  }
  if (tid == 0 && p.split) p.split[blockIdx.x] = split;
}

// Joins the partial results of the unit that begins in a run and ends in a later one:
// 16 rows and 32 columns a workgroup, whose waves share the runs.  The workgroups of
// one run are neighbours, so that they lie on all XCDs: units of equal length begin
// in every 2^n-th run, and with the runs as neighbours all work fell to one XCD.
template <int GRID, int R>
__global__ __launch_bounds__(kAtThreads) void ufp4_attend_join_kernel(AttendParams p) {
  constexpr int ROWS = 16 * R;
  __shared__ float ml[kAtWaves][2][64];
  __shared__ float part[kAtWaves][64][8 + 1];
  const int slices = R * (p.c.dim / 32), slice = (int)blockIdx.x % slices, run = (int)blockIdx.x / slices;
  const SplitUnit u = p.split[run];
  if (u.runs == 0) return;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int i = slice % R, col = slice / R * 32;
  // run k of the unit is slot 1 of its first workgroup and slot 0 of the others
  auto row_of = [&](int k) { return (2 * ((int64_t)run + k) + (k == 0)) * ROWS + 16 * i + r; };
  float m = -__builtin_inff(), l = 0.0f;
  for (int k = wave; k < u.runs; k += kAtWaves) m = fmaxf(m, p.ml[row_of(k)].x);
  ml[wave][0][lane] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kAtWaves; ++k) m = fmaxf(m, ml[k][0][lane]);
  const float base = m == -__builtin_inff() ? 0.0f : m;
  float o[1][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[0][j] = 0.0f;
#pragma unroll 4
  for (int k = wave; k < u.runs; k += kAtWaves) {
    const int64_t at = row_of(k);
    const float2 x = p.ml[at];
    const f32x4* from = reinterpret_cast<const f32x4*>(p.o + at * p.c.dim + col + 8 * g);
    const f32x4 y0 = from[0], y1 = from[1];
    const float alpha = __builtin_amdgcn_exp2f(x.x - base);
    l += x.y * alpha;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[0][j] += y0[j] * alpha;
      o[0][4 + j] += y1[j] * alpha;
    }
  }
  ml[wave][1][lane] = l;
#pragma unroll
  for (int j = 0; j < 8; ++j) part[wave][lane][j] = o[0][j];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int k = 1; k < kAtWaves; ++k) {
    l += ml[k][1][lane];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[0][j] += part[k][lane][j];
  }
  const Sequence s = sequence_of(p, u.b);
  const int q = u.tile * ROWS + 16 * i + r;
  finish_row<1>(p, o, m, l, head_scale(p.c.vts, u.h) * unshift<GRID>(), q < s.rows, s.row0 + q / p.group,
                u.h * p.group + q % p.group, col, g);
}

template <int GRID, int DT, int R>
hipError_t launch_rows(const AttendParams& p, hipStream_t s) {
  // no sequence is longer than its line of the page table
  const int64_t cap = (p.ld_pages * p.c.page_tokens + kStep - 1) / kStep, steps = cap > 0 ? cap : 1;
  const int64_t units = (int64_t)p.sequences * p.c.heads * p.row_tiles, most = units * steps;
  const unsigned runs = (unsigned)(most < p.max_runs ? most : p.max_runs);
  const bool full = p.c.dim == DT;
  if (p.rht && full) ufp4_attend_kernel<GRID, DT, R, 2, true><<<runs, kAtThreads, 0, s>>>(p);
  else if (p.rht) ufp4_attend_kernel<GRID, DT, R, 2, false><<<runs, kAtThreads, 0, s>>>(p);
  else if (full) ufp4_attend_kernel<GRID, DT, R, 1, true><<<runs, kAtThreads, 0, s>>>(p);
  else ufp4_attend_kernel<GRID, DT, R, 1, false><<<runs, kAtThreads, 0, s>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || steps == 1) return e;
  ufp4_attend_join_kernel<GRID, R><<<runs * (unsigned)(R * (p.c.dim / 32)), kAtThreads, 0, s>>>(p);
  return hipGetLastError();
}

template <int GRID>
hipError_t launch_grid(const AttendParams& p, hipStream_t s) {
  const bool two = attend_rows(p.c.dim, p.group, p.max_draft) == 32;
  if (p.c.dim <= 64) return two ? launch_rows<GRID, 64, 2>(p, s) : launch_rows<GRID, 64, 1>(p, s);
  if (p.c.dim <= 128) return two ? launch_rows<GRID, 128, 2>(p, s) : launch_rows<GRID, 128, 1>(p, s);
  return two ? launch_rows<GRID, 256, 2>(p, s) : launch_rows<GRID, 256, 1>(p, s);
}

}  // namespace

int attend_rows(int32_t dim, int32_t group, int32_t max_draft) { return (int64_t)group * max_draft > 16 ? 32 : 16; }

// Runs of a launch: the workgroups that 256 compute units hold at once.
int32_t attend_runs(int32_t dim, int32_t rows) { return 256 * attend_waves(dim, rows / 16); }

hipError_t launch_attend(const AttendParams& p, hipStream_t s) {
  switch (p.grid) {
    case kGridE1M2: return launch_grid<kGridE1M2>(p, s);
    case kGridINT4: return launch_grid<kGridINT4>(p, s);
    case kGridE2M1:  // the clamped grid's codes are E2M1 codes
    case kGridE2M1C: return launch_grid<kGridE2M1>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ufp4
