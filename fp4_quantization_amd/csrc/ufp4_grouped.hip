// ufp4_grouped.hip -- products of grouped NV16 operands on the fp16 MFMA: the
// rows of every expert's segment with that expert's matrix (nt), and every
// expert's weight gradient, reduced over its rows (dw).  One launch for all
// experts; the segments are read from the device.
//
// Operands are expanded to fp16 exactly (ufp4_expand.hpp), multiplied with
// fp32 accumulation, and the two tensor scales are applied to the sums.
#include "ufp4_expand.hpp"
#include "ufp4_moe.hpp"
#include "ufp4_vec.hpp"

namespace ufp4 {

namespace {

// The tile kernel: one workgroup of 12 waves per CU walks over 256 x 256 tiles
// of C in steps of 64 along the reduction axis.  Four producer waves (one per
// SIMD) load codes and expand them to fp16 in LDS; eight consumer waves (two
// per SIMD, each 64 x 128 of the tile) multiply what the producers wrote one
// step earlier, so the expansion's vector work runs beside the matrix work of
// other waves instead of between it (65536 rows, 64 segments, N = K = 4096: 2455 us
// against 2548 where all waves expand and then multiply, both otherwise as they
// were then).  All waves meet in one barrier per step.
//
// Measured there, medians of 20 calls in four runs: 1803 to 1823 us (single calls
// 1726 to 2185), 1.21 PFLOP/s, where the library's fp16 product of 16384^3 reaches
// 1.45; weight gradients of 4096 x 2048 1155 to 1159 us (1088 to 1278), 0.95, of
// which the 2.1 GB of stores would take 310 alone.  A step takes 2640 clocks (3.07 M
// clocks for a unit's 1160 steps), at 1.4 to 2.0 GHz from call to call: 2048 are the
// matrix instructions', about 2500 a producer wave's beside them (2050 by itself: 260
// vector instructions, 16 stores to LDS, 8 loads), the rest the stores' drain and
// the barrier.  The producers bound it, and the power that the matrix units take:
// 9% fewer clocks a step gave 4% of time.
constexpr int kTileM = 256, kTileN = 256, kTileK = 64;
constexpr int kConsumers = 8, kProducers = 4;
constexpr uint32_t kXcds = 8;
constexpr int64_t kXcdRows = 32;
constexpr int kTileThreads = 64 * (kConsumers + kProducers);
constexpr int kPieces = (kTileM + kTileN) / (16 * kProducers);  // per producer lane

// LDS: [A, B][buffer][line][64 fp16] (both buffers of an operand inside the
// 16-bit offset of an LDS instruction).  The eight 16-byte chunks of a line are
// stored in the order chunk ^ swizzle(line): the same chunk of neighbouring lines
// (a fragment load) and neighbouring chunks of a line (an expansion store of two
// lines) then fall on different banks.
constexpr int kLineHalves = kTileK;
__device__ __forceinline__ int swizzle(int line) { return ((line >> 1) & 7) ^ (line & 1); }
__device__ __forceinline__ int lds_at(int line, int chunk) { return line * kLineHalves + 8 * (chunk ^ swizzle(line)); }

// A value that all lanes of the wave hold, as a scalar: branches, loop counts
// and barriers that depend on it are the wave's.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ int64_t clamp_row(int64_t r, int64_t total) { return r < 0 ? 0 : (r > total ? total : r); }

// Segment e of the rows: [max(0, offsets[e]), offsets[e+1]) inside
// [0, total); segment `groups` is what is left behind the last one.
__device__ __forceinline__ void segment_rows(const GroupedParams& p, int e, int64_t* lo, int64_t* hi) {
  *lo = e == 0 ? 0 : clamp_row(p.offsets[e], p.total_rows);
  *hi = e < p.groups ? clamp_row(p.offsets[e + 1], p.total_rows) : p.total_rows;
  if (e > p.groups || *hi < *lo) *hi = *lo;
}

// The segments as every workgroup keeps them in LDS.
//   nt: lo / hi, the rows of segment e (e = groups: the rest), and first, the
//       number of row tiles before it;
//   dw: lo / hi, its positions along the column-wise layouts (whole blocks of
//       16, after those of the segments before it).
constexpr int kMaxSegments = 1025;
struct Segments {
  int32_t lo[kMaxSegments], hi[kMaxSegments], first[kMaxSegments];
};

// Filled by one wave: 64 segments at a time, their sizes summed over lanes.
template <bool DW>
__device__ void fill_segments(const GroupedParams& p, int rows, Segments& S) {
  const int lane = threadIdx.x & 63;
  const int n = DW ? p.groups : p.groups + 1;
  int64_t before = 0;
  for (int e0 = 0; e0 < n; e0 += 64) {
    const int e = e0 + lane;
    int64_t lo, hi;
    segment_rows(p, e < n ? e : p.groups, &lo, &hi);
    if (e >= n) hi = lo;
    const int size = DW ? (int)((hi - lo + 15) / 16 * 16) : (int)((hi - lo + rows - 1) / rows);
    int inc = size;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    if (e < n) {
      const int64_t first = before + inc - size;
      S.lo[e] = (int32_t)(DW ? clamp_row(first, p.total_rows) : lo);
      S.hi[e] = (int32_t)(DW ? clamp_row(first + size, p.total_rows) : hi);
      if (!DW) S.first[e] = (int32_t)first;
    }
    before += uniform(__shfl(inc, 63));
  }
}

// Rows [lo, hi) of the row tile `tile` (of `rows` rows) and its segment, -1 if
// there are fewer tiles.  One wave.
struct RowTile {
  int32_t e, lo, hi;
};
__device__ __forceinline__ RowTile find_tile(const GroupedParams& p, const Segments& S, int tile, int rows) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 <= p.groups; e0 += 64) {
    const int e = e0 + lane < p.groups ? e0 + lane : p.groups;
    const int lo = S.lo[e], hi = S.hi[e], at = lo + (tile - S.first[e]) * rows;
    const uint64_t hit = __ballot(tile >= S.first[e] && at < hi);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      const int from = uniform(__shfl(at, src)), end = uniform(__shfl(hi, src));
      return RowTile{uniform(__shfl(e, src)), from, from + rows < end ? from + rows : end};
    }
  }
  return RowTile{-1, 0, 0};
}

// Two neighbouring values of a row of C, n of them inside it.
__device__ __forceinline__ void store_c(float* c, float v0, float v1, int n) {
  if (n >= 2)
    store_8(c, v32x2{__float_as_uint(v0), __float_as_uint(v1)});
  else if (n == 1)
    *c = v0;
}
// The same inside C, past the caches: the weight gradients of a step are larger
// than them (64 experts, 4096 x 2048, fp32: 1270 us through them, 1134 past).
typedef float f32x2s __attribute__((ext_vector_type(2), aligned(4)));
__device__ __forceinline__ void stream_c(float* c, float v0, float v1) {
  __builtin_nontemporal_store(f32x2s{v0, v1}, reinterpret_cast<f32x2s*>(c));
}
struct __attribute__((packed, aligned(2))) Pair16 {
  uint32_t w;
};
__device__ __forceinline__ void store_c(uint16_t* c, float v0, float v1, int n) {
  if (n >= 2)
    reinterpret_cast<Pair16*>(c)->w = pack_bf16(v0, v1);
  else if (n == 1)
    *c = to_bf16(v0);
}
__device__ __forceinline__ void stream_c(uint16_t* c, float v0, float v1) { store_c(c, v0, v1, 2); }

// The line of B (of each 64) that LDS row r holds: columns 2 i and 2 i + 1 of
// C come from the same lane of two neighbouring column tiles of 32, so a lane
// stores them together and a row of a store is 64 neighbouring columns.
__device__ __forceinline__ int b_line_of(int r) { return 2 * (r & 31) + (r >> 5); }

// One tile's place: rows [m0, m_end) of A and C, lines n0.. of B, the
// reduction range of K values at ka / kb, matrix e.  e < 0: no such tile.
struct Tile {
  int32_t e;
  bool live;  // false: rows behind the last segment, zeros
  int32_t m0, m_end, n0, K, ka;
  int64_t kb, b_line;
};
// Tile ids.  The tiles of one row of tiles (`nt` of them) share a panel of A.
// Workgroups are dealt to the XCDs in turn, so id % 8 is the XCD: rows of tiles
// go to XCDs in turn and a row's tiles stay on its XCD, whose L2 then reads the
// panel once.  With few rows the ids are the tiles in order.
struct TileGrid {
  uint32_t ids;
  FastDiv nt, mt;  // column tiles; row tiles a group (dw)
  int32_t xcd;
};
template <bool DW>
__device__ __forceinline__ Tile tile_at(const GroupedParams& p, const Segments& S, uint32_t id, const TileGrid& g) {
  const uint32_t l = g.xcd ? id / kXcds : id, q = g.nt.div(l);
  const uint32_t row = g.xcd ? q * kXcds + id % kXcds : q;
  const int32_t n0 = (int32_t)(l - q * g.nt.d) * kTileN;
  if (DW) {
    const uint32_t e = g.mt.div(row);
    if (e >= (uint32_t)p.groups) return Tile{-1, false, 0, 0, 0, 0, 0, 0, 0};
    const int lo = uniform(S.lo[e]), hi = uniform(S.hi[e]);
    return Tile{(int32_t)e, true, (int32_t)(row - e * g.mt.d) * kTileM, (int32_t)p.M, n0, hi - lo, lo, lo, 0};
  }
  const RowTile s = find_tile(p, S, (int)row, kTileM);
  const int e = uniform(s.e);
  const bool live = e < p.groups;
  return Tile{e, live, uniform(s.lo), uniform(s.hi), n0, live ? (int32_t)p.K : 0, 0, live ? e * p.b.seg_k : 0,
              live ? e * p.b.seg_lines : 0};
}

// One operand's lines of a tile as bounds-checked buffers: loads of lines past
// the last one give zeros.  A line has fewer than 2^24 bytes of codes, so the
// 256 lines of a tile stay inside 32-bit offsets.
struct Lines {
  __amdgpu_buffer_rsrc_t codes, scales;
};
__device__ __forceinline__ Lines lines_of(const GroupedOperand& o, int64_t line, int64_t count, int64_t k) {
  const int64_t n = count < kTileM ? count : kTileM, at = line * o.pitch + k, len = n * o.pitch - k;
  const uint32_t bytes = (uint32_t)(len / 2);
  // word 3: 32-bit data, raw addressing
  return Lines{__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(o.codes + at / 2), 0, (int)bytes, 0x00020000),
               __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(o.scales + at / 16), 0, (int)(bytes / 8), 0x00020000)};
}

// 32 values of one line (two blocks): 16 bytes of codes and two scale bytes.
struct Piece {
  g32x4 c;
  uint32_t s;
};
constexpr uint32_t kOutside = 0xFFFFFFF0u;  // an offset past every buffer

// off, scale: byte offsets of the lane's codes and scales; `chunk` chunks of 128
// values behind them go into the scalar offset.
__device__ __forceinline__ void load_piece(const Lines& b, uint32_t off, uint32_t scale, int chunk, Piece& v) {
  v.c = __builtin_bit_cast(g32x4, __builtin_amdgcn_raw_buffer_load_b128(b.codes, (int)off, 64 * chunk, 0));
  v.s = __builtin_amdgcn_raw_buffer_load_b16(b.scales, (int)scale, 8 * chunk, 0);
}
// The first block of a line, and zeros; zeros where it is not `mine`.
__device__ __forceinline__ void load_block(const Lines& b, uint32_t off, bool mine, Piece& v) {
  const int at = (int)(mine ? off : kOutside), scale = (int)(mine ? off / 8 : kOutside);
  const g32x2 lo = __builtin_bit_cast(g32x2, __builtin_amdgcn_raw_buffer_load_b64(b.codes, at, 0, 0));
  const g32x2 hi = __builtin_bit_cast(g32x2, __builtin_amdgcn_raw_buffer_load_b64(b.codes, (int)kOutside, 0, 0));
  v.c = g32x4{lo.x, lo.y, hi.x, hi.y};
  v.s = __builtin_amdgcn_raw_buffer_load_b8(b.scales, scale, 0, 0);
}
constexpr uint32_t kScaleBits = 0x7F7Fu;  // of a piece's two scales

template <int GRID, bool DW, typename TC>
__global__ __launch_bounds__(kTileThreads) void ufp4_grouped_tile_kernel(GroupedParams p, TileGrid g) {
  __shared__ __attribute__((aligned(16))) _Float16 As[2][kTileM * kLineHalves], Bs[2][kTileN * kLineHalves];
  __shared__ Segments S;
  const int t = threadIdx.x, wave = uniform(t >> 6), lane = t & 63;
  if (wave == 0) fill_segments<DW>(p, kTileM, S);
  __syncthreads();
  // Both kinds of waves walk over the same tiles and chunks of 128 values, two
  // steps and barriers each; step h of a chunk is in buffer h.
  if (wave >= kConsumers) {
    // ---- producers.  A lane holds 32 values of eight lines (every 64th), a
    // quad of lanes 128 neighbouring values of a line (64 bytes of codes).
    // Step h expands block h of every piece: a step's 64 values are 16 of
    // every 32, the same ones of A and B, and a sum does not depend on its
    // order.
    const int q = t & 3, l0 = (t - 64 * kConsumers) >> 2;
    const int at0 = lds_at(l0, 2 * q), at1 = lds_at(l0, 2 * q + 1);  // (the swizzle repeats every 16 lines)
    for (uint32_t id = blockIdx.x; id < g.ids; id += gridDim.x) {
      const Tile T = tile_at<DW>(p, S, id, g);
      if (T.e < 0 || T.K <= 0) continue;
      const Lines A = lines_of(p.a, T.m0, T.m_end - T.m0, T.ka);
      const Lines B = lines_of(p.b, T.b_line + T.n0, p.N - T.n0, T.kb);
      uint32_t off[kPieces], soff[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces / 2; ++i) {
        off[i] = (uint32_t)(l0 + 64 * i) * (uint32_t)(p.a.pitch / 2) + 16 * q;
        off[i + kPieces / 2] = (uint32_t)(b_line_of(l0) + 64 * i) * (uint32_t)(p.b.pitch / 2) + 16 * q;
      }
      // Block h of every piece of v; after the second one load(i) follows.
      auto expand = [&](Piece (&v)[kPieces], uint32_t mask, auto load) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            if (i >= kPieces / 2 || 64 * i < T.m_end - T.m0) {  // (not the lines of waves without rows)
              const f16x2 ds = expand_scales<GRID>(v[i].s & mask);
              const f16x2 d = h ? f16x2{ds.y, ds.y} : f16x2{ds.x, ds.x};
              uint32_t e[8];
              expand8_shifted<GRID>(h ? v[i].c.z : v[i].c.x, d, e);
              expand8_shifted<GRID>(h ? v[i].c.w : v[i].c.y, d, e + 4);
              _Float16* to = (i < kPieces / 2 ? As : Bs)[h] + 64 * (i % (kPieces / 2)) * kLineHalves;
              *reinterpret_cast<g32x4*>(to + at0) = g32x4{e[0], e[1], e[2], e[3]};
              *reinterpret_cast<g32x4*>(to + at1) = g32x4{e[4], e[5], e[6], e[7]};
            }
            if (h == 1) load(i);
          }
          __syncthreads();
        }
      };
      if (T.K <= 16) {  // a single block
        Piece v[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) load_block(i < kPieces / 2 ? A : B, off[i], q == 0, v[i]);
        expand(v, kScaleBits & 0x00FFu, [](int) {});
        continue;
      }
      // Chunks are requested two ahead of the one that is expanded: piece by
      // piece into the registers that the expansion has just read, so that loads
      // are issued between vector instructions and not in one burst (65536 rows,
      // 64 segments, N = K = 4096, one after the other on one device: 1850 us in
      // bursts, 1785 so; weight gradients 1150, 1122).  A wait for a piece counts
      // the loads behind it, so every request takes the same loads without a
      // branch; behind the last chunk that one is requested again.
      // In a chunk that the range ends in, a piece of which one block is left is
      // read one block earlier, so that no access crosses the buffer's end, one
      // that is outside is read from the line's start, and the scales of blocks
      // that do not count are masked.
#pragma unroll
      for (int i = 0; i < kPieces; ++i) soff[i] = off[i] / 8;
      const int chunks = (T.K + 127) / 128, whole = T.K / 128, left = T.K - 128 * whole - 32 * q;
      const uint32_t end_mask = left >= 32 ? kScaleBits : left >= 16 ? kScaleBits & 0xFF00u : 0;
      int at = 0;
      auto request = [&](int chunk) {
        if (chunk < whole) {
          at = uniform(chunk);
        } else if (chunk < chunks) {
          at = 0;
          const int by = left >= 32 ? 64 * whole : left >= 16 ? 64 * whole - 8 : -16 * q;
#pragma unroll
          for (int i = 0; i < kPieces; ++i) off[i] += by, soff[i] += by / 8;
        }
      };
      auto load = [&](Piece (&v)[kPieces], int i) { load_piece(i < kPieces / 2 ? A : B, off[i], soff[i], at, v[i]); };
      auto step = [&](Piece (&v)[kPieces], int chunk) {
        request(chunk + 2);
        expand(v, chunk < whole ? kScaleBits : end_mask, [&](int i) {
          __builtin_amdgcn_sched_barrier(0);
          load(v, i);
          __builtin_amdgcn_sched_barrier(0);
        });
      };
      Piece u[kPieces], v[kPieces];
      request(0);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) load(u, i);
      request(1);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) load(v, i);
      for (int c = 0; c < chunks; c += 2) {
        step(u, c);
        if (c + 1 >= chunks) break;
        step(v, c + 1);
      }
    }
    __syncthreads();  // the consumers' last step
    return;
  }
  // ---- consumers.  At the barrier that ends a producers' step the step's
  // buffer is complete and the other one is free again.
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 128;
  // chunk 2 kk + h of a line is chunk h with bits 1 and 2 of its place flipped
  const int a_at = lds_at(lane & 31, lane >> 5) + wm * kLineHalves, b_at = lds_at(lane & 31, lane >> 5) + wn * kLineHalves;
  for (uint32_t id = blockIdx.x; id < g.ids; id += gridDim.x) {
    const Tile T = tile_at<DW>(p, S, id, g);
    if (T.e < 0) continue;
    const bool busy = T.m0 + wm < T.m_end;  // the wave has rows
    f32x16 acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};
    const int chunks = (T.K + 127) / 128;
    for (int c = 0; c < chunks; ++c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __syncthreads();
        if (!busy) continue;
        // Fragments are requested ahead of their use: A's of the next 16 values
        // during this ones', B's two before their turn (two matrix
        // instructions each, and as many of the SIMD's other consumer between).
        f16x8 fa[2][2], fb[3];
        auto read_a = [&](int kk, int i) {
          fa[kk & 1][i] = *reinterpret_cast<const f16x8*>(As[h] + (a_at ^ (16 * kk)) + 32 * i * kLineHalves);
        };
        auto read_b = [&](int n) {  // n: column tile n % 4 of values 16 (n / 4) ..
          fb[n % 3] = *reinterpret_cast<const f16x8*>(Bs[h] + (b_at ^ (16 * (n >> 2))) + 32 * (n & 3) * kLineHalves);
        };
        read_a(0, 0);
        read_b(0);
        read_a(0, 1);
        read_b(1);
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const int kk = n >> 2, j = n & 3;
          if (n + 2 < 16) read_b(n + 2);
          if (kk < 3 && (j == 1 || j == 2)) read_a(kk + 1, j - 1);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[kk & 1][i], fb[n % 3], acc[i][j], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    constexpr float kUnshift = (float)(1 << (2 * kExpandShift<GRID>));
    const float s = T.live ? p.a.ts[T.e] * p.b.ts[T.e] : 0.0f;
    const int col = T.n0 + wn + 2 * (lane & 31), row = T.m0 + wm + 4 * (lane >> 5), left = (int)p.N - col;
    TC* c = static_cast<TC*>(p.c) + (DW ? (int64_t)T.e * p.M * p.N : 0) + (int64_t)row * p.ldc + col;
    const int rows = T.m_end - row;
    const float s2 = kUnshift * s;
    if (T.n0 + kTileN <= p.N && T.m0 + wm + 64 <= T.m_end) {  // (the wave's part is inside C)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          TC* to = c + (32 * i + 8 * (r >> 2) + (r & 3)) * p.ldc;
          stream_c(to, acc[i][0][r] * s2, acc[i][1][r] * s2);
          stream_c(to + 64, acc[i][2][r] * s2, acc[i][3][r] * s2);
        }
      continue;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int at = 32 * i + 8 * (r >> 2) + (r & 3);
        if (at >= rows) continue;
        TC* to = c + at * p.ldc;
        store_c(to, acc[i][0][r] * s2, acc[i][1][r] * s2, left);
        store_c(to + 64, acc[i][2][r] * s2, acc[i][3][r] * s2, left - 64);
      }
  }
  __syncthreads();
}

// ------------------------------------------------------------- few rows
// Products with few rows a segment read the segment's matrix once and are
// bound by that.  A workgroup takes 16 NT lines of B and up to 16 MT rows of a
// segment; its four waves take the reduction's stretches of 512 values in turn
// and their sums are added in LDS in a fixed order.  Operands go from memory to
// registers: a lane holds 128 neighbouring values of a line (its codes four
// 16-byte loads, its scales one of 8 bytes), the four lane groups of the MFMA
// 512 of the line.  The MFMA's 32 values are then 8 of each group's, the same
// ones of both operands, so nothing is exchanged between lanes.  128 rows, 64
// segments, N = K = 4096: 110 us for 511 MB of codes and scales, 4.6 TB/s.
typedef float f32x4 __attribute__((ext_vector_type(4)));
constexpr int kRowWaves = 4, kRowThreads = 64 * kRowWaves, kStretch = 512;

// 128 values of a line: codes and scales of its eight blocks.
struct Stretch {
  g32x4 c[4];
  g32x2 s;
};
// off: byte offset of the lane's first code in `stretch` 0.  whole: the stretch
// is inside the range; else `left` values of the lane's are (whole pieces of
// 32; the others read as code and scale zero).
__device__ __forceinline__ Stretch load_stretch(const Lines& b, uint32_t off, int stretch, bool whole, int left) {
  Stretch v;
  if (whole) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v.c[i] = __builtin_bit_cast(g32x4, __builtin_amdgcn_raw_buffer_load_b128(b.codes, (int)(off + 16 * i), 256 * stretch, 0));
    v.s = __builtin_bit_cast(g32x2, __builtin_amdgcn_raw_buffer_load_b64(b.scales, (int)(off / 8), 32 * stretch, 0));
  } else {
    const uint32_t at = off + 256 * (uint32_t)stretch;
    uint32_t s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = 32 * i < left;
      v.c[i] = __builtin_bit_cast(g32x4, __builtin_amdgcn_raw_buffer_load_b128(b.codes, (int)(in ? at + 16 * i : kOutside), 0, 0));
      s[i] = __builtin_amdgcn_raw_buffer_load_b16(b.scales, (int)(in ? at / 8 + 2 * i : kOutside), 0, 0);
    }
    v.s = g32x2{s[0] | (s[1] << 16), s[2] | (s[3] << 16)};
  }
  return v;
}
// Piece i (32 values) as four MFMA fragments.
template <int GRID>
__device__ __forceinline__ void expand_piece(const Stretch& v, int i, f16x8 (&f)[4]) {
  const f16x2 ds = expand_scales<GRID>(((i < 2 ? v.s.x : v.s.y) >> (16 * (i & 1))) & kScaleBits);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t e[4];
    expand8_shifted<GRID>(v.c[i][j], j < 2 ? f16x2{ds.x, ds.x} : f16x2{ds.y, ds.y}, e);
    f[j] = __builtin_bit_cast(f16x8, g32x4{e[0], e[1], e[2], e[3]});
  }
}

// The row tile `tile` straight from the offsets, by each wave for itself.
__device__ __forceinline__ RowTile find_tile(const GroupedParams& p, int tile, int rows) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 <= p.groups; e0 += 64) {
    const int e = e0 + lane < p.groups ? e0 + lane : p.groups;
    int64_t lo, hi;
    segment_rows(p, e, &lo, &hi);
    if (e0 + lane > p.groups) hi = lo;
    const int n = (int)((hi - lo + rows - 1) / rows);
    int inc = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    const int first = before + inc - n;
    const uint64_t hit = __ballot(tile >= first && tile < first + n);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      const int from = uniform(__shfl((int)lo + (tile - first) * rows, src)), end = uniform(__shfl((int)hi, src));
      return RowTile{uniform(__shfl(e, src)), from, from + rows < end ? from + rows : end};
    }
    before += uniform(__shfl(inc, 63));
  }
  return RowTile{-1, 0, 0};
}

// Four neighbouring values of a row of C, n of them inside it.
__device__ __forceinline__ void store_c4(float* c, const f32x4& v, int n) {
  store_c(c, v[0], v[1], n);
  store_c(c + 2, v[2], v[3], n - 2);
}
__device__ __forceinline__ void store_c4(uint16_t* c, const f32x4& v, int n) {
  if (n >= 4) {
    store_8(c, v32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])});
  } else {
    store_c(c, v[0], v[1], n);
    store_c(c + 2, v[2], v[3], n - 2);
  }
}

template <int GRID, int MT, int NT, typename TC>
__global__ __launch_bounds__(kRowThreads) void ufp4_grouped_rows_kernel(GroupedParams p, FastDiv nt) {
  __shared__ f32x4 part[kRowWaves][MT * NT][64];
  const int t = threadIdx.x, wave = uniform(t >> 6), lane = t & 63, g = lane >> 4, r = lane & 15;
  const uint32_t tile = nt.div(blockIdx.x);
  const int n0 = (int)(blockIdx.x - tile * nt.d) * 16 * NT;
  const RowTile T = find_tile(p, (int)tile, 16 * MT);
  if (T.e < 0) return;
  const bool live = T.e < p.groups;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (live) {
    const int K = (int)p.K;
    const Lines A = lines_of(p.a, T.lo, T.hi - T.lo, 0);
    const Lines B = lines_of(p.b, T.e * p.b.seg_lines + n0, p.N - n0, T.e * p.b.seg_k);
    const uint32_t pa = (uint32_t)(p.a.pitch / 2), pb = (uint32_t)(p.b.pitch / 2);
    for (int c = wave; c * kStretch < K; c += kRowWaves) {
      const bool whole = (c + 1) * kStretch <= K;
      const int left = K - c * kStretch - 128 * g;
      Stretch a[MT], b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) b[n] = load_stretch(B, (uint32_t)(16 * n + r) * pb + 64 * g, c, whole, left);
#pragma unroll
      for (int m = 0; m < MT; ++m) a[m] = load_stretch(A, (uint32_t)(16 * m + r) * pa + 64 * g, c, whole, left);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f16x8 fa[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) expand_piece<GRID>(a[m], i, fa[m]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          f16x8 fb[4];
          expand_piece<GRID>(b[n], i, fb);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j], fa[m][j], acc[m][n], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) part[wave][m * NT + n][lane] = acc[m][n];
  __syncthreads();
  constexpr float kUnshift = (float)(1 << (2 * kExpandShift<GRID>));
  const float s = live ? p.a.ts[T.e] * p.b.ts[T.e] : 0.0f;
  for (int i = wave; i < MT * NT; i += kRowWaves) {
    f32x4 v = part[0][i][lane];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) v += part[w][i][lane];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = v[k] * kUnshift * s;
    // a lane holds row r of the 16 and four neighbouring columns
    const int row = T.lo + 16 * (i / NT) + r, col = n0 + 16 * (i % NT) + 4 * g;
    if (row < T.hi && col < p.N)
      store_c4(static_cast<TC*>(p.c) + (int64_t)row * p.ldc + col, v, (int)(p.N - col < 4 ? p.N - col : 4));
  }
}

// Compute units of the current device.
hipError_t compute_units(int64_t* out) {
  int dev = 0, cus = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  *out = cus;
  return e;
}

// Row tiles of a launch: every segment that has rows adds at most one partial
// tile, and so do the rows behind the last one.
int64_t segment_tiles(const GroupedParams& p, int rows) {
  return p.total_rows / rows + (p.groups < p.total_rows ? p.groups : p.total_rows) + 1;
}
int64_t row_tiles(const GroupedParams& p, bool dw) {
  return dw ? (p.M + kTileM - 1) / kTileM : segment_tiles(p, kTileM);
}

template <bool DW, typename TC>
hipError_t launch_tiles(const GroupedParams& p, int64_t cus, hipStream_t s) {
  const int64_t nt = (p.N + kTileN - 1) / kTileN, mt = row_tiles(p, DW), rows = mt * (DW ? p.groups : 1);
  const bool xcd = rows >= kXcdRows && cus % kXcds == 0;
  const int64_t ids = nt * (xcd ? (rows + kXcds - 1) / kXcds * kXcds : rows);
  const TileGrid g{(uint32_t)ids, fast_div((uint32_t)nt), fast_div((uint32_t)mt), xcd};
  const unsigned grid = (unsigned)(ids < cus ? ids : cus);
  switch (p.grid) {
    case kGridE1M2: ufp4_grouped_tile_kernel<kGridE1M2, DW, TC><<<grid, kTileThreads, 0, s>>>(p, g); break;
    case kGridINT4: ufp4_grouped_tile_kernel<kGridINT4, DW, TC><<<grid, kTileThreads, 0, s>>>(p, g); break;
    case kGridE2M1:  // the clamped grid's codes are E2M1 codes
    case kGridE2M1C: ufp4_grouped_tile_kernel<kGridE2M1, DW, TC><<<grid, kTileThreads, 0, s>>>(p, g); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

template <int MT, int NT, typename TC>
hipError_t launch_rows(const GroupedParams& p, hipStream_t s) {
  const int64_t nt = (p.N + 16 * NT - 1) / (16 * NT);
  const unsigned grid = (unsigned)(nt * segment_tiles(p, 16 * MT));
  const FastDiv d = fast_div((uint32_t)nt);
  switch (p.grid) {
    case kGridE1M2: ufp4_grouped_rows_kernel<kGridE1M2, MT, NT, TC><<<grid, kRowThreads, 0, s>>>(p, d); break;
    case kGridINT4: ufp4_grouped_rows_kernel<kGridINT4, MT, NT, TC><<<grid, kRowThreads, 0, s>>>(p, d); break;
    case kGridE2M1:
    case kGridE2M1C: ufp4_grouped_rows_kernel<kGridE2M1, MT, NT, TC><<<grid, kRowThreads, 0, s>>>(p, d); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// The kernel of an nt call.  Measured with 64 segments, N = K = 4096 (us): 2
// rows a segment 111 (16 rows a workgroup), 133 (32 rows), 248 (tiles); 8 rows
// 134, 162, 253; 16 rows 184, 174, 258; 32 rows 280, 231, 263; 64 rows 457,
// 374, 300; 128 rows 834, 659, 407.  One segment, N = K = 2048: 500 rows 20, 14,
// 42 (16 tiles leave most of the device idle).  So a round of tiles, one a
// compute unit, costs what about 11 workgroups of 32 rows a compute unit do.  A
// segment is taken to end in the middle of a tile.  Half as many lines a
// workgroup pay where there are few workgroups: 24 segments of 4 rows, N 1000, K
// 2080: 13.2 (32 lines) against 16.3 us (64); 64 segments of 8 rows, N = K =
// 4096: 144 against 136.
enum RowsKernel { kTiles, kRows16Lines32, kRows16Lines64, kRows32Lines64 };
RowsKernel rows_kernel(const GroupedParams& p, int64_t cus) {
  const int64_t nt = (p.N + 63) / 64, ends = p.groups < p.total_rows ? p.groups : p.total_rows;
  if (2 * nt * segment_tiles(p, 16) >= ((int64_t)1 << 24)) return kTiles;  // (threads of a launch)
  const int64_t wgs = (p.total_rows / 32 + (ends + 1) / 2) * nt;
  const int64_t tiles = (p.total_rows / kTileM + (ends + 1) / 2) * ((p.N + kTileN - 1) / kTileN);
  if (wgs >= 11 * cus * ((tiles + cus - 1) / cus)) return kTiles;
  if (p.total_rows > 12 * p.groups) return kRows32Lines64;
  return wgs < 2 * cus ? kRows16Lines32 : kRows16Lines64;
}

template <typename TC>
hipError_t launch_nt(const GroupedParams& p, hipStream_t s) {
  int64_t cus = 0;
  const hipError_t e = compute_units(&cus);
  if (e != hipSuccess) return e;
  switch (rows_kernel(p, cus)) {
    case kRows16Lines32: return launch_rows<1, 2, TC>(p, s);
    case kRows16Lines64: return launch_rows<1, 4, TC>(p, s);
    case kRows32Lines64: return launch_rows<2, 4, TC>(p, s);
    default: return launch_tiles<false, TC>(p, cus, s);
  }
}

}  // namespace

int64_t grouped_tiles(const GroupedParams& p, bool dw) {
  return (p.N + kTileN - 1) / kTileN * (row_tiles(p, dw) * (dw ? p.groups : 1) + kXcds);
}

hipError_t launch_grouped_nt(const GroupedParams& p, hipStream_t s) {
  return p.c_f32 ? launch_nt<float>(p, s) : launch_nt<uint16_t>(p, s);
}

hipError_t launch_grouped_dw(const GroupedParams& p, hipStream_t s) {
  int64_t cus = 0;
  const hipError_t e = compute_units(&cus);
  if (e != hipSuccess) return e;
  return p.c_f32 ? launch_tiles<true, float>(p, cus, s) : launch_tiles<true, uint16_t>(p, cus, s);
}

}  // namespace ufp4
