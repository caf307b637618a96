// ufp4_matvec_plan.hpp -- how a product of a few rows is launched: where the
// kernel finds x', tokens and waves a workgroup (plain host code, without HIP).
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace ufp4 {

constexpr int kMvChunk = 128;  // values of K a step
constexpr int kMvWaves = 8;
constexpr int kSegment = 4;  // chunks of a wave whose weights are on the way at once
constexpr int kLdsTokens = 4;
constexpr size_t kLdsX = 96 << 10;  // bytes
constexpr int kCus = 256;

// Where the fragments of x' come from: LDS, where every workgroup has prepared them
// (up to four tokens); registers, read once from what a kernel in front has prepared
// (one fragment a step, K of one segment); or that memory, tile by tile.
enum XSource { kXLds, kXRegisters, kXMemory };

struct MatvecPlan {
  XSource x;
  int nt;       // 16-token tiles a workgroup
  int log_kw;   // waves that share a tile of 16 rows of w
  int64_t gx, gy;
};

// Whether x' (parts 16-bit numbers a value) fits the LDS of every workgroup.
inline bool matvec_fits_lds(int64_t tokens, int64_t K, int parts) {
  if (tokens > kLdsTokens) return false;
  const int64_t padded = (K + kMvChunk - 1) / kMvChunk * kMvChunk;
  return padded * tokens * parts * 2 <= (int64_t)kLdsX;
}

// Waves that share a tile: those that have a whole segment of K each, and more where
// that leaves waves of the device (16 a compute unit) without work.  One token, N x K
// = 65536 x 8192: 70 us with 1, 2, 4 or 8; 4096 x 4096: 19, 12.5, 9.5, 7.5; 16 tokens,
// 16384 x 4096: 26.6, 15.7, 16.2, 14.3.
inline int matvec_log_waves(int64_t tiles, int64_t chunks) {
  int log_kw = 0;
  while (log_kw < 3 && (kSegment << log_kw) < chunks) ++log_kw;
  while (log_kw < 3 && (2 << log_kw) <= chunks && (tiles << log_kw) < 16 * kCus) ++log_kw;
  return log_kw;
}

inline MatvecPlan matvec_plan(int64_t tokens, int64_t N, int64_t K, int parts) {
  const int64_t tiles = (N + 15) / 16, chunks = (K + kMvChunk - 1) / kMvChunk, t16 = (tokens + 15) / 16;
  MatvecPlan m;
  m.log_kw = matvec_log_waves(tiles, chunks);
  const int side = kMvWaves >> m.log_kw;
  const int64_t groups = (tiles + side - 1) / side;
  m.gx = groups < 2 * kCus ? groups : 2 * kCus;
  if (matvec_fits_lds(tokens, K, parts)) {
    m.x = kXLds;
    m.nt = 1;
    m.gy = 1;
    return m;
  }
  // as many tokens a workgroup as leave every compute unit one
  m.nt = t16 > 2 ? 4 : (int)t16;
  while (m.nt > 1 && groups * ((t16 + m.nt - 1) / m.nt) < kCus) m.nt /= 2;
  m.gy = (t16 + m.nt - 1) / m.nt;
  // (K of 0 has no workspace: only kXMemory reads nothing where there are no chunks)
  m.x = m.nt == 1 && parts == 1 && chunks > 0 && chunks <= (kSegment << m.log_kw) ? kXRegisters : kXMemory;
  if (m.x == kXRegisters && m.gx > kCus) m.gx = kCus;
  return m;
}

}  // namespace ufp4
