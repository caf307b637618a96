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
// The tokens of a sequence are cut into pieces of equal length, one a workgroup;
// four waves share a piece's tiles and join in LDS, and where a sequence has
// several pieces they meet through the workspace in a second kernel.  The length
// of a piece follows from all lengths, read on the device, so that a batch of any
// lengths fills the device evenly and the launch does not depend on them.
#include "ufp4_expand.hpp"
#include "ufp4_serve.hpp"
#include "ufp4_vec.hpp"

namespace ufp4 {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAtWaves = 4, kAtThreads = 64 * kAtWaves;
constexpr int kMinPiece = 128;  // tokens: a tile for each wave
constexpr int kMaxTokens = 1 << 30;  // of a sequence
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ double pow2d(int e) { return __longlong_as_double((long long)(e + 1023) << 52); }
__device__ __forceinline__ float head_scale(const float* ts, int h) {
  const float s = ts ? ts[h] : 1.0f;
  return s > 0.0f && s <= 3.40282347e38f ? s : 1.0f;
}

// ---------------------------------------------------------------- pieces
struct Sequence {
  int64_t row0;  // of q
  int32_t n;     // drafted tokens
  int32_t rows;  // to compute: drafted tokens up to max_draft, times group
  int32_t len;   // tokens in the cache
};
__device__ __forceinline__ Sequence sequence_of(const AttendParams& p, int b) {
  const int64_t r0 = p.q_offsets[b], r1 = p.q_offsets[b + 1];
  const int64_t most = p.ld_pages * p.c.page_tokens;
  Sequence s{r0, 0, 0, 0};
  if (r0 < 0 || r1 < r0 || r1 > p.q_rows) return s;
  s.n = (int32_t)(r1 - r0);
  s.rows = (s.n < p.max_draft ? s.n : p.max_draft) * p.group;
  const int len = p.lengths[b];
  s.len = len < 0 ? 0 : (len > most ? (int32_t)most : len);
  return s;
}
__device__ __forceinline__ int tiles_of(const Sequence& s, int rows) { return (s.rows + rows - 1) / rows; }
// Pieces of a sequence: at least one for each head and tile of rows, so that a
// sequence without tokens is answered too.
__device__ __forceinline__ int splits_of(const Sequence& s, int piece) {
  return s.len > 0 ? (s.len + piece - 1) / piece : 1;
}

// Sum over the workgroup of one value a thread.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* red) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kAtWaves; ++w) v += red[w];
  return v;
}

// Tokens a piece: the work of all sequences (tokens x tiles of rows x heads)
// over the number of pieces aimed at, in whole tiles for every wave.
template <int ROWS>
__device__ __forceinline__ int piece_tokens(const AttendParams& p, int64_t* red) {
  int64_t work = 0;
  for (int b = threadIdx.x; b < p.sequences; b += kAtThreads) {
    const Sequence s = sequence_of(p, b);
    work += (int64_t)s.len * tiles_of(s, ROWS);
  }
  work = block_sum(work, red) * p.c.heads;
  const int64_t t = (work + p.target - 1) / p.target;
  if (t >= kMaxTokens) return kMaxTokens;
  return t == 0 ? kMinPiece : (int)((t + kMinPiece - 1) / kMinPiece * kMinPiece);
}

struct Piece {
  int32_t b, first;  // sequence, and the first piece of it
  int32_t index;     // among its pieces
};
// The sequence that piece `id` belongs to, b = -1 past the last one.
template <int ROWS>
__device__ Piece find_piece(const AttendParams& p, int id, int piece, int32_t* sh) {
  int before = 0;
  for (int b0 = 0; b0 < p.sequences; b0 += kAtThreads) {
    const int b = b0 + threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int n = 0;
    if (b < p.sequences) {
      const Sequence s = sequence_of(p, b);
      n = splits_of(s, piece) * tiles_of(s, ROWS) * p.c.heads;
    }
    int inc = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    __syncthreads();
    if (lane == 63) sh[wave] = inc;
    if (threadIdx.x == 0) sh[kAtWaves] = -1;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kAtWaves; ++w) {
      if (w < wave) inc += sh[w];
      total += sh[w];
    }
    const int first = before + inc - n;
    if (id >= first && id < first + n) {
      sh[kAtWaves] = b;
      sh[kAtWaves + 1] = first;
    }
    __syncthreads();
    if (sh[kAtWaves] >= 0) return Piece{uniform(sh[kAtWaves]), uniform(sh[kAtWaves + 1]), id - uniform(sh[kAtWaves + 1])};
    before += total;
  }
  return Piece{-1, 0, 0};
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
// A lane's part of row `row` of a tile (dim DT / 4 values from g DT / 4 on), as
// fp16 fragments: q times a power of two for the row that takes its largest
// magnitude to [2^12, 2^13) (its transform below 2^15), and with the transform a
// second part, what the first one's rounding left.  Returns the power's exponent.
template <int DT, int PARTS>
__device__ __forceinline__ int load_q(const AttendParams& p, const uint16_t* q, bool in, int g, f16x8 (&f)[PARTS][DT / 32]) {
  constexpr int N = DT / 4;
  float v[N];
#pragma unroll
  for (int i = 0; i < N / 16; ++i) {
    const int d = g * N + 16 * i;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      V8 a{};
      if (in && d < p.c.dim) a = row_load(q + d + 8 * h, 8);
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
  for (int i = 0; i < N / 16; ++i) {
    float* x = v + 16 * i;
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] *= f2;
    if (PARTS == 2) {
      fwht16_inlane(x, p.sg);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] *= p.sg.fin;
    }
  }
#pragma unroll
  for (int i = 0; i < DT / 32; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = v[8 * i + j];
      const _Float16 a = (_Float16)x;
      f[0][i][j] = a;
      if (PARTS == 2) {
        const float left = x - (float)a;
        f[PARTS - 1][i][j] = (_Float16)(left - left == 0.0f ? left : 0.0f);
      }
    }
  return shift;
}

// ---------------------------------------------------------------- results
// O of one row in the lane layout of the second product: the lane of group g has
// values 32 t + 8 g + j.  Inverse transform of the 16-block that lanes g and g ^ 1
// share: three stages in the lane, one across, 1/4, signs.
template <int NT>
__device__ __forceinline__ void untransform(const AttendParams& p, float (&o)[NT][8], int g) {
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
      v[j] = s * (0.25f * ((g & 1) ? p.d[8 + j] : p.d[j]));
    }
  }
}

// A finished row: O / l, tensor scale, inverse transform, out and lse.
template <int NT>
__device__ __forceinline__ void finish_row(const AttendParams& p, float (&o)[NT][8], float m, float l, float vscale, bool in,
                                           int64_t row, int head, int g) {
  const float f = l > 0.0f || l != l ? vscale / l : 0.0f;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) o[t][j] *= f;
  if (p.rht) untransform<NT>(p, o, g);
  if (!in) return;
  uint16_t* out = p.out + row * p.ldo + (int64_t)head * p.c.dim + 8 * g;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (32 * t < p.c.dim) {
      V8 a;
#pragma unroll
      for (int j = 0; j < 8; ++j) a.v[j] = o[t][j];
      store_16(out + 32 * t, pack(a));
    }
  }
  if (p.lse && g == 0)
    p.lse[row * p.q_heads + head] = l > 0.0f || l != l ? (m + __log2f(l)) * kLn2 : -__builtin_inff();
}

template <int GRID>
constexpr float unshift() { return (float)(1 << kExpandShift<GRID>); }

// ---------------------------------------------------------------- the kernel
template <int GRID, int DT, int R, int PARTS>
__global__ __launch_bounds__(kAtThreads) void ufp4_attend_kernel(AttendParams p) {
  constexpr int ROWS = 16 * R, NT = DT / 32;
  constexpr int kPitch = DT + 4;
  __shared__ int64_t red[kAtWaves];
  __shared__ int32_t sh[kAtWaves + 2];
  __shared__ float ml[kAtWaves][2][ROWS];
  __shared__ float join[2][ROWS][kPitch];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int piece = uniform(piece_tokens<ROWS>(p, red));
  if (blockIdx.x == 0 && tid == 0) p.plan[0] = piece;
  const Piece w = find_piece<ROWS>(p, (int)blockIdx.x, piece, sh);
  if (w.b < 0) return;
  const Sequence s = sequence_of(p, w.b);
  const int splits = splits_of(s, piece);
  // pieces of a sequence: [tile of rows][head][split]
  const int split = w.index % splits, h = w.index / splits % p.c.heads, tile = w.index / splits / p.c.heads;
  const int hist = s.len - s.n;  // below 0: drafted tokens that the cache does not hold
  const int t_begin = split * piece, t_end = t_begin + piece < s.len ? t_begin + piece : s.len;

  f16x8 qf[R][PARTS][NT];
  float f[R];         // logits from sums, times log2 e
  int drafted[R];     // of this lane's row
  uint64_t bits[R];   // drafted tokens it sees
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int m = tile * ROWS + 16 * i + r;
    const bool in = m < s.rows;
    drafted[i] = m / p.group;
    const int64_t row = s.row0 + drafted[i];
    const int head = h * p.group + m % p.group;
    const int shift = load_q<DT, PARTS>(p, p.q + (in ? row * p.ldq + (int64_t)head * p.c.dim : 0), in, g, qf[i]);
    f[i] = (float)(pow2d(-shift) * (double)(unshift<GRID>() * kLog2e) * (double)p.scale * (double)head_scale(p.c.kts, h));
    bits[i] = in && p.mask ? p.mask[row] : 0;
  }
  f32x4 o[R][2 * NT];
  float mx[R], sum[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    mx[i] = -__builtin_inff();
    sum[i] = 0.0f;
#pragma unroll
    for (int t = 0; t < 2 * NT; ++t) o[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  const int half = p.c.dim / 2, blocks = p.c.dim / 16;
  const int key = 8 * (r >> 2) + (r & 3);  // token of row r of the first tile of 16

  for (int t0 = t_begin + 32 * wave; t0 < t_end; t0 += 32 * kAtWaves) {
    const uint32_t slot = p.c.page.div((uint32_t)t0);
    const int page = uniform(p.table[w.b * p.ld_pages + slot]);
    if (page < 0 || page >= p.c.pages) continue;
    const int64_t at = ((int64_t)page * p.c.heads + h) * p.c.page_tokens + (t0 - (int)slot * p.c.page_tokens);
    const uint8_t* kc = p.c.kc + at * half;
    const uint8_t* ks = p.c.ks + at * blocks;
    const uint8_t* vc = p.c.vc + at * half;
    const uint8_t* vs = p.c.vs + at * blocks;
    // ---- logits
    f32x4 a[R][2];
#pragma unroll
    for (int i = 0; i < R; ++i) a[i][0] = a[i][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int tok = key + 4 * u;
#pragma unroll
      for (int c = 0; c < (DT + 127) / 128; ++c) {
        // up to 32 codes of the key and their one or two scales
        const int d = g * (DT / 4) + 32 * c;
        constexpr int W = DT == 64 ? 2 : 4;
        uint32_t codes[4] = {0u, 0u, 0u, 0u}, two = 0;
        if (d < p.c.dim) {
          if (W == 2) {
            const v32x2 x = *reinterpret_cast<const v32x2*>(kc + tok * half + d / 2);
            codes[0] = x.x;
            codes[1] = x.y;
            two = ks[tok * blocks + d / 16];
          } else {
            const v32x4 x = *reinterpret_cast<const v32x4*>(kc + tok * half + d / 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) codes[j] = x[j];
            two = *reinterpret_cast<const uint16_t*>(ks + tok * blocks + d / 16);
          }
        }
        const f16x2 ds = expand_scales<GRID>(two & 0x7F7Fu);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          uint32_t e[4];
          expand8_shifted<GRID>(codes[j], j < 2 ? f16x2{ds.x, ds.x} : f16x2{ds.y, ds.y}, e);
          const f16x8 kf = __builtin_bit_cast(f16x8, g32x4{e[0], e[1], e[2], e[3]});
#pragma unroll
          for (int i = 0; i < R; ++i)
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
              a[i][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[i][q][4 * c + j], a[i][u], 0, 0, 0);
        }
      }
    }
    // ---- softmax: this lane's tokens are t0 + 8 g + j
    const bool edge = t0 + 32 > hist;  // the wave's
    uint32_t alive = 0xFF;             // tokens that exist
    f16x8 pf[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = a[i][j >> 2][j & 3] * f[i];
      if (edge) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = t0 + 8 * g + j, d = t - hist;
          const bool seen = t < s.len && (d < 0 || (p.mask ? d < 64 && ((bits[i] >> d) & 1) : d <= drafted[i]));
          x[j] = seen ? x[j] : -__builtin_inff();
        }
      }
      float m = x[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) m = fmaxf(m, x[j]);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      m = fmaxf(m, mx[i]);
      const float base = m == -__builtin_inff() ? 0.0f : m;
      const float alpha = __builtin_amdgcn_exp2f(mx[i] - base);
      float l = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = __builtin_amdgcn_exp2f(x[j] - base);
        l += e;
        pf[i][j] = (_Float16)e;
      }
      sum[i] = sum[i] * alpha + l;
      if (__any(alpha != 1.0f)) {
#pragma unroll
        for (int t = 0; t < 2 * NT; ++t) o[i][t] *= alpha;
      }
      mx[i] = m;
    }
    if (edge) {
      const int left = s.len - t0 - 8 * g;
      alive = left >= 8 ? 0xFFu : left <= 0 ? 0u : (1u << left) - 1u;
    }
    // ---- values
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (32 * t >= p.c.dim) break;
      const v32x2 c = *reinterpret_cast<const v32x2*>(vc + (16 * t + r) * 32 + 8 * g);
      v32x2 b = *reinterpret_cast<const v32x2*>(vs + (2 * t + (r >> 3)) * 32 + 8 * g) & 0x7F7F7F7Fu;
      if (edge) {
        // tokens that do not exist hold anything
        uint32_t k0 = 0, k1 = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          k0 |= (alive >> j) & 1 ? 0xFFu << (8 * j) : 0u;
          k1 |= (alive >> (4 + j)) & 1 ? 0xFFu << (8 * j) : 0u;
        }
        b.x &= k0;
        b.y &= k1;
      }
      f16x2 s01, s23, s45, s67;
      scales_of<GRID>(b.x, s01, s23);
      scales_of<GRID>(b.y, s45, s67);
      uint32_t first[4], second[4];
      expand_tokens<GRID>(c.x, s01, s23, first, second);
      expand_tokens<GRID>(c.y, s45, s67, first + 2, second + 2);
      const f16x8 v0 = __builtin_bit_cast(f16x8, g32x4{first[0], first[1], first[2], first[3]});
      const f16x8 v1 = __builtin_bit_cast(f16x8, g32x4{second[0], second[1], second[2], second[3]});
#pragma unroll
      for (int i = 0; i < R; ++i) {
        o[i][2 * t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[i], o[i][2 * t], 0, 0, 0);
        o[i][2 * t + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[i], o[i][2 * t + 1], 0, 0, 0);
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
    const float alpha = __builtin_amdgcn_exp2f(mx[i] - base);
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
  for (int step = kAtWaves / 2; step >= 1; step >>= 1) {
    if (wave >= step && wave < 2 * step) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float* to = &join[wave - step][16 * i + r][32 * t + 8 * g];
#pragma unroll
          for (int j = 0; j < 8; j += 4) *reinterpret_cast<f32x4*>(to + j) = f32x4{acc[i][t][j], acc[i][t][j + 1], acc[i][t][j + 2], acc[i][t][j + 3]};
        }
    }
    __syncthreads();
    if (wave < step) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[i][t][j] += join[wave][16 * i + r][32 * t + 8 * g + j];
    }
    __syncthreads();
  }
  if (wave != 0) return;
  const float vscale = head_scale(p.c.vts, h) * unshift<GRID>();
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int m = tile * ROWS + 16 * i + r;
    if (splits == 1) {
      finish_row<NT>(p, acc[i], mx[i], sum[i], vscale, m < s.rows, s.row0 + m / p.group, h * p.group + m % p.group, g);
    } else {
      const int64_t at = (int64_t)blockIdx.x * ROWS + 16 * i + r;
      if (g == 0) p.ml[at] = make_float2(mx[i], sum[i]);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (32 * t < p.c.dim) {
          float* to = p.o + at * p.c.dim + 32 * t + 8 * g;
#pragma unroll
          for (int j = 0; j < 8; j += 4) *reinterpret_cast<f32x4*>(to + j) = f32x4{acc[i][t][j], acc[i][t][j + 1], acc[i][t][j + 2], acc[i][t][j + 3]};
        }
    }
  }
}

// Joins the pieces of a sequence: one wave takes 16 rows of a tile and head,
// blockIdx.y the sequence.
template <int GRID, int DT, int R>
__global__ __launch_bounds__(kAtThreads) void ufp4_attend_join_kernel(AttendParams p) {
  constexpr int ROWS = 16 * R, NT = DT / 32;
  __shared__ int64_t red[kAtWaves];
  const int b = blockIdx.y, piece = uniform(p.plan[0]);
  const Sequence s = sequence_of(p, b);
  const int splits = splits_of(s, piece), tiles = tiles_of(s, ROWS);
  if (splits == 1 || tiles == 0) return;
  int64_t before = 0;
  for (int i = threadIdx.x; i < b; i += kAtThreads) {
    const Sequence o = sequence_of(p, i);
    before += (int64_t)splits_of(o, piece) * tiles_of(o, ROWS) * p.c.heads;
  }
  before = block_sum(before, red);
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int unit = (int)blockIdx.x * kAtWaves + wave;  // [tile][head][16 rows]
  const int part = unit % R, h = unit / R % p.c.heads, tile = unit / R / p.c.heads;
  if (tile >= tiles) return;
  const int64_t first = ((before + ((int64_t)tile * p.c.heads + h) * splits) * ROWS) + 16 * part + r;
  float m = -__builtin_inff(), l = 0.0f;
  for (int k = 0; k < splits; ++k) m = fmaxf(m, p.ml[first + (int64_t)k * ROWS].x);
  const float base = m == -__builtin_inff() ? 0.0f : m;
  float o[NT][8];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) o[t][j] = 0.0f;
  for (int k = 0; k < splits; ++k) {
    const int64_t at = first + (int64_t)k * ROWS;
    const float2 x = p.ml[at];
    const float alpha = __builtin_amdgcn_exp2f(x.x - base);
    l += x.y * alpha;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (32 * t < p.c.dim) {
        const float* from = p.o + at * p.c.dim + 32 * t + 8 * g;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[t][j] += from[j] * alpha;
      }
  }
  const int q = tile * ROWS + 16 * part + r;
  finish_row<NT>(p, o, m, l, head_scale(p.c.vts, h) * unshift<GRID>(), q < s.rows, s.row0 + q / p.group,
                 h * p.group + q % p.group, g);
}

template <int GRID, int DT, int R>
hipError_t launch_rows(const AttendParams& p, hipStream_t s) {
  // no sequence is longer than its line of the page table
  const int64_t most = (p.ld_pages * p.c.page_tokens + kMinPiece - 1) / kMinPiece;
  const int64_t units = (int64_t)p.sequences * p.c.heads * p.row_tiles;
  const int64_t pieces = units * (most > 0 ? most : 1) < p.max_pieces ? units * (most > 0 ? most : 1) : p.max_pieces;
  if (p.rht) ufp4_attend_kernel<GRID, DT, R, 2><<<(unsigned)pieces, kAtThreads, 0, s>>>(p);
  else ufp4_attend_kernel<GRID, DT, R, 1><<<(unsigned)pieces, kAtThreads, 0, s>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || most <= 1) return e;
  const unsigned gx = (unsigned)(((int64_t)p.row_tiles * p.c.heads * R + kAtWaves - 1) / kAtWaves);
  ufp4_attend_join_kernel<GRID, DT, R><<<dim3(gx, (unsigned)p.sequences), kAtThreads, 0, s>>>(p);
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

int64_t attend_max_pieces(int32_t heads, int32_t row_tiles, int32_t sequences) {
  return kAttendTarget + (int64_t)sequences * heads * row_tiles;
}

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
