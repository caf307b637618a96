// ufp4_serve.hpp -- host/device shared parameter blocks and launchers of the
// decoding operators: products of a few rows with 4-bit weights, the 4-bit
// key-value cache, attention over it (internal to the library; the public ABI
// is ufp4.h).
#pragma once
#include "ufp4_internal.hpp"
#include "ufp4_matvec_plan.hpp"
#include "ufp4_moe.hpp"

namespace ufp4 {

// ------------------------------------------------------------------ products
struct MatvecParams {
  const void* x;
  int32_t x_f32, y_f32;
  int64_t tokens, N, K, ldx, ldy;
  const uint8_t* codes;
  const uint8_t* scales;
  const float* ts;
  int32_t grid, mx, rht;
  RhtSigns sg;
  void* y;
  // the prepared x: 16-bit fragments, then one exponent a token
  uint16_t* xp;
  int32_t* shift;
};
// 16-bit numbers that x' is split into, one where that is exact.  For a bf16 result one
// fp16 number does as well: off by 2^-11 where the result's own rounding is off by 2^-8
// (errors of whole results, that rounding included, are 0.7 to 0.9% larger than from
// fp32 x'), for half the MFMAs and LDS of two.  fp32 results take two (22 bits); MX32,
// whose numbers are bf16, three (24).
inline int matvec_parts(bool mx, bool rht, bool x_f32, bool y_f32) {
  if (mx) return rht || x_f32 ? 3 : 1;
  return y_f32 && (rht || x_f32) ? 2 : 1;
}
// Whether a call prepares x in every workgroup's LDS (no workspace) or by a
// kernel of its own.
bool matvec_in_lds(int64_t tokens, int64_t K, int parts);
hipError_t launch_matvec(const MatvecParams& p, hipStream_t s);

// ------------------------------------------------------------------ the cache
constexpr int kCacheTile = 32;  // tokens of a tile

struct CacheView {
  uint8_t* kc;
  uint8_t* ks;
  uint8_t* vc;
  uint8_t* vs;
  const float* kts;
  const float* vts;
  int64_t pages;
  int32_t page_tokens, heads, dim;
  FastDiv page;  // division by page_tokens
};

struct CacheParams {
  CacheView c;
  int32_t grid, rht;  // rht: transform (append), inverse transform (read)
  RhtSigns sg;
  uint32_t signs;  // of the inverse transform, bit j set: -1
  FastDiv pieces;  // division by the pieces (of one lane) of a token's head
  int64_t tokens;
  const int64_t* slots;
  const uint16_t* k;
  const uint16_t* v;
  void* k_out;
  void* v_out;
  int64_t ldk, ldv;
  int32_t out_f32;
};
hipError_t launch_cache_append(const CacheParams& p, hipStream_t s);
hipError_t launch_cache_read(const CacheParams& p, hipStream_t s);

// ------------------------------------------------------------------ attention
// A unit of attention (a sequence, key head and tile of rows) that begins in a run
// and ends in a later one; runs: how many it lies in, 0: there is none.
struct SplitUnit {
  int32_t b, h, tile, runs;
};
struct AttendParams {
  CacheView c;
  int32_t grid, rht;
  uint32_t signs;  // of the transform, bit j set: -1
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t ldq, ldo, q_rows;
  int32_t q_heads, group;  // group: query heads a key head
  const int64_t* q_offsets;
  const int32_t* lengths;
  const int32_t* table;
  int64_t ld_pages;
  int32_t sequences, max_draft;
  const uint64_t* mask;
  float scale;
  int32_t row_tiles;  // of a sequence with max_draft drafted tokens
  int32_t max_runs;   // of a launch
  SplitUnit* split;   // [run]
  float2* ml;         // [run][2][row]: maximum and sum
  float* o;           // [run][2][row][dim]
};
// Rows (drafted tokens x query heads) of a tile, and the most runs of a launch.
int attend_rows(int32_t dim, int32_t group, int32_t max_draft);
int32_t attend_runs(int32_t dim, int32_t rows);
hipError_t launch_attend(const AttendParams& p, hipStream_t s);

}  // namespace ufp4
