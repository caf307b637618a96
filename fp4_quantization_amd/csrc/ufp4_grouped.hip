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

constexpr int kTileM = 256, kTileN = 256, kTileK = 64;
constexpr int kTileLd = kTileK + 8;
constexpr int kTileThreads = 512;

struct Segment {
  int32_t e;        // group, `groups` for the rows behind the last one, -1: none
  int64_t lo, hi;   // rows (nt) or positions along the reduction axis (dw)
};

__device__ __forceinline__ int64_t clamp_row(int64_t r, int64_t total) { return r < 0 ? 0 : (r > total ? total : r); }

// Segment e of the rows: [max(0, offsets[e]), offsets[e+1]) inside
// [0, total); segment `groups` is what is left behind the last one.
__device__ __forceinline__ void segment_rows(const GroupedParams& p, int e, int64_t* lo, int64_t* hi) {
  *lo = e == 0 ? 0 : clamp_row(p.offsets[e], p.total_rows);
  *hi = e < p.groups ? clamp_row(p.offsets[e + 1], p.total_rows) : p.total_rows;
  if (e > p.groups || *hi < *lo) *hi = *lo;
}

// The row tile `tile` of the segments' tiles of `rows` rows, in segment order:
// its segment and rows.  One wave.
__device__ __forceinline__ Segment find_tile(const GroupedParams& p, int64_t tile, int rows) {
  const int lane = threadIdx.x & 63;
  Segment r{-1, 0, 0};
  int64_t before = 0;
  for (int e0 = 0; e0 <= p.groups; e0 += 64) {
    int64_t lo, hi;
    segment_rows(p, e0 + lane <= p.groups ? e0 + lane : p.groups, &lo, &hi);
    if (e0 + lane > p.groups) hi = lo;
    const int n = (int)((hi - lo + rows - 1) / rows);
    int inc = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(inc, d);
      if (lane >= d) inc += o;
    }
    const int64_t first = before + inc - n;
    const uint64_t hit = __ballot(tile >= first && tile < first + n);
    if (hit) {
      const int src = __ffsll((unsigned long long)hit) - 1;
      r.e = e0 + src;
      r.lo = __shfl(lo, src) + (tile - __shfl(first, src)) * rows;
      const int64_t end = __shfl(hi, src);
      r.hi = r.lo + rows < end ? r.lo + rows : end;
      return r;
    }
    before += __shfl(inc, 63);
  }
  return r;
}

// Positions of segment e along the column-wise layouts: whole blocks of 16,
// after those of the segments before it.  One wave.
__device__ __forceinline__ Segment find_columns(const GroupedParams& p, int e) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0, mine = 0;
  for (int e0 = 0; e0 <= e; e0 += 64) {
    const int i = e0 + lane;
    int64_t n = 0;
    if (i <= e) {
      const int64_t lo = i == 0 ? 0 : clamp_row(p.offsets[i], p.total_rows);
      const int64_t hi = clamp_row(p.offsets[i + 1], p.total_rows);
      n = hi > lo ? (hi - lo + 15) / 16 * 16 : 0;
    }
    if (i < e) before += n;
    if (i == e) mine = n;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    before += __shfl_xor(before, d);
    mine += __shfl_xor(mine, d);
  }
  return Segment{e, clamp_row(before, p.total_rows), clamp_row(before + mine, p.total_rows)};
}

__device__ __forceinline__ void store_c(float* c, float v) { __builtin_nontemporal_store(v, c); }
__device__ __forceinline__ void store_c(uint16_t* c, float v) { *c = to_bf16(v); }

// nt: grid (row tiles, column tiles); dw: grid (column tiles, row tiles,
// groups).  Eight waves, each 64 x 128 of the 256 x 256 tile.
template <int GRID, bool DW, typename TC>
__global__ __launch_bounds__(kTileThreads) void ufp4_grouped_tile_kernel(GroupedParams p) {
  __shared__ __attribute__((aligned(16))) _Float16 As[2][kTileM][kTileLd];
  __shared__ __attribute__((aligned(16))) _Float16 Bs[2][kTileN][kTileLd];
  __shared__ Segment seg_lds;
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  if (wave == 0) {
    const Segment s = DW ? find_columns(p, blockIdx.z) : find_tile(p, blockIdx.x, kTileM);
    if (lane == 0) seg_lds = s;
  }
  __syncthreads();
  const Segment sg = seg_lds;
  if (sg.e < 0) return;
  // rows of A (and C) this tile covers, and the reduction range [k0, k0 + K)
  const int64_t m0 = DW ? (int64_t)blockIdx.y * kTileM : sg.lo;
  const int64_t m_end = DW ? p.M : sg.hi;
  const int64_t n0 = (int64_t)(DW ? blockIdx.x : blockIdx.y) * kTileN;
  const bool live = DW || sg.e < p.groups;  // else rows of no segment: zeros
  const int64_t K = live ? (DW ? sg.hi - sg.lo : p.K) : 0;
  const int64_t ka = DW ? sg.lo : 0, kb = DW ? sg.lo : (live ? sg.e * p.b.seg_k : 0);
  const int64_t b_line = DW || !live ? 0 : sg.e * p.b.seg_lines;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 128;
  const int lr = t >> 1, lb = 2 * (t & 1);
  const bool a_ok = m0 + lr < m_end, b_ok = n0 + lr < p.N;
  const int64_t ao = (a_ok ? m0 + lr : 0) * p.a.pitch + ka + 16 * lb;
  const int64_t bo = (b_line + (b_ok ? n0 + lr : 0)) * p.b.pitch + kb + 16 * lb;
  const uint8_t* ac = p.a.codes + ao / 2;
  const uint8_t* as = p.a.scales + ao / 16;
  const uint8_t* bc = p.b.codes + bo / 2;
  const uint8_t* bs = p.b.scales + bo / 16;
  const int nsteps = (int)((K + kTileK - 1) / kTileK);
  struct Stage {
    g32x4 a, b;
    uint32_t sa, sb;
  };
  // two neighbouring blocks of one line: 16 bytes of codes, two scale bytes
  // (blocks past the range are zero; a range ends on a block)
  auto two = [&](const uint8_t* c, const uint8_t* s, bool ok, int64_t st, int64_t left, g32x4* w, uint32_t* sc) {
    g32x4 v = {0u, 0u, 0u, 0u};
    uint32_t q = 0;
    const uint8_t* cp = c + st * (kTileK / 2);
    const uint8_t* sp = s + st * (kTileK / 16);
    if (ok && left >= 32) {
      if (DW) {
        const g32x2 x = *reinterpret_cast<const g32x2*>(cp), y = *reinterpret_cast<const g32x2*>(cp + 8);
        v = g32x4{x.x, x.y, y.x, y.y};
      } else {
        v = *reinterpret_cast<const g32x4*>(cp);
      }
      q = (uint32_t)sp[0] | ((uint32_t)sp[1] << 8);
    } else if (ok && left >= 16) {
      const g32x2 x = *reinterpret_cast<const g32x2*>(cp);
      v = g32x4{x.x, x.y, 0u, 0u};
      q = sp[0];
    }
    *w = v;
    *sc = q;
  };
  auto fetch = [&](int64_t st) {
    Stage f;
    const int64_t left = K - st * kTileK - 16 * lb;
    two(ac, as, a_ok, st, left, &f.a, &f.sa);
    two(bc, bs, b_ok, st, left, &f.b, &f.sb);
    return f;
  };
  auto put = [&](const Stage& f, int buf) {
    uint32_t e[8];
    expand16<GRID>(g32x2{f.a.x, f.a.y}, f.sa & 0xFFu, e);
    store16(e, &As[buf][lr][16 * lb]);
    expand16<GRID>(g32x2{f.a.z, f.a.w}, f.sa >> 8, e);
    store16(e, &As[buf][lr][16 * lb + 16]);
    expand16<GRID>(g32x2{f.b.x, f.b.y}, f.sb & 0xFFu, e);
    store16(e, &Bs[buf][lr][16 * lb]);
    expand16<GRID>(g32x2{f.b.z, f.b.w}, f.sb >> 8, e);
    store16(e, &Bs[buf][lr][16 * lb + 16]);
  };
  f32x16 acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};
  Stage nxt{};
  if (nsteps > 0) {
    put(fetch(0), 0);
    nxt = fetch(1);
  }
  __syncthreads();
  for (int st = 0; st < nsteps; ++st) {
    const int cur = st & 1;
    if (st + 1 < nsteps) {
      put(nxt, cur ^ 1);
      nxt = fetch(st + 2);
    }
#pragma unroll
    for (int kk = 0; kk < kTileK / 16; ++kk) {
      f16x8 fa[2], fb[4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        fa[i] = *reinterpret_cast<const f16x8*>(&As[cur][wm + 32 * i + (lane & 31)][16 * kk + 8 * (lane >> 5)]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        fb[j] = *reinterpret_cast<const f16x8*>(&Bs[cur][wn + 32 * j + (lane & 31)][16 * kk + 8 * (lane >> 5)]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  }
  const int64_t e = DW ? (int64_t)blockIdx.z : sg.e;
  const float s = live ? p.a.ts[e] * p.b.ts[e] : 0.0f;
  TC* c = static_cast<TC*>(p.c) + (DW ? e * p.M * p.N : 0);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t row = m0 + wm + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        const int64_t col = n0 + wn + 32 * j + (lane & 31);
        if (row < m_end && col < p.N) store_c(&c[row * p.ldc + col], acc[i][j][r] * s);
      }
}

template <bool DW, typename TC>
hipError_t launch_tiles(const GroupedParams& p, dim3 grid, hipStream_t s) {
  switch (p.grid) {
    case kGridE1M2: ufp4_grouped_tile_kernel<kGridE1M2, DW, TC><<<grid, kTileThreads, 0, s>>>(p); break;
    case kGridINT4: ufp4_grouped_tile_kernel<kGridINT4, DW, TC><<<grid, kTileThreads, 0, s>>>(p); break;
    case kGridE2M1:  // the clamped grid's codes are E2M1 codes
    case kGridE2M1C: ufp4_grouped_tile_kernel<kGridE2M1, DW, TC><<<grid, kTileThreads, 0, s>>>(p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_nt(const GroupedParams& p, hipStream_t s) {
  // a segment adds at most one partial tile
  const dim3 grid((unsigned)(p.total_rows / kTileM + p.groups + 1), (unsigned)((p.N + kTileN - 1) / kTileN));
  return p.c_f32 ? launch_tiles<false, float>(p, grid, s) : launch_tiles<false, uint16_t>(p, grid, s);
}

hipError_t launch_grouped_dw(const GroupedParams& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + kTileN - 1) / kTileN), (unsigned)((p.M + kTileM - 1) / kTileM), (unsigned)p.groups);
  return p.c_f32 ? launch_tiles<true, float>(p, grid, s) : launch_tiles<true, uint16_t>(p, grid, s);
}

}  // namespace ufp4
