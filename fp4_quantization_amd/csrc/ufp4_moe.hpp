// ufp4_moe.hpp -- host/device shared parameter blocks and launchers of the
// expert-layer kernels: sort / dispatch / combine, 8-bit checkpoints and
// grouped products (internal to the library; the public ABI is ufp4.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ufp4 {

// Quotient of a 31-bit number by a fixed divisor: with 2^sh >= d > 2^(sh-1)
// and m = ceil(2^(31+sh) / d), m d - 2^(31+sh) < d <= 2^sh, so n m / 2^(31+sh)
// exceeds n / d by less than 1 / d for n < 2^31 and the floors agree.
struct FastDiv {
  uint32_t d, m, sh;
  __host__ __device__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> (31 + sh)); }
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f;
  f.d = d;
  f.sh = 0;
  while (((uint64_t)1 << f.sh) < d) ++f.sh;
  f.m = (uint32_t)((((uint64_t)1 << (31 + f.sh)) + d - 1) / d);
  return f;
}

constexpr int64_t kLastLevelCache = (int64_t)256 << 20;  // bytes, MI355X

constexpr int kMaxExperts = 1023;  // + the padding segment = the grouped quantizer's 1024
constexpr int kMaxSlots = 1024;
constexpr int kMaxAlign = 4096;

struct SortParams {
  const int32_t* ids;
  int64_t ld_ids;
  int32_t n;  // tokens * slots
  FastDiv slots;
  int32_t experts, align, total_rows;
  int64_t* offsets;
  int32_t* row_of_slot;
  int32_t* slot_of_row;
};
hipError_t launch_expert_sort(const SortParams& p, hipStream_t s);

struct DispatchParams {
  const uint16_t* x;      // bf16 rows, or null:
  const uint8_t* codes;   // a checkpoint's codes and scales
  const uint16_t* scales;
  int32_t format;
  int64_t tokens, cols, ld;
  int32_t slots;
  const int32_t* row_of_slot;
  const int32_t* slot_of_row;
  int64_t total_rows;
  uint16_t* out;
  int64_t ldo;
};
hipError_t launch_expert_dispatch(const DispatchParams& p, hipStream_t s);

struct CombineParams {
  const void* z;
  int32_t z_f32, out_f32;
  int64_t total_rows, cols, ldz;
  const int32_t* row_of_slot;
  const float* weights;
  int64_t tokens;
  int32_t slots;
  void* out;
  int64_t ldo;
};
hipError_t launch_expert_combine(const CombineParams& p, hipStream_t s);

struct CombineBwdParams {
  const void* d;
  int32_t d_f32, z_f32;
  int64_t tokens, cols, ldd;
  int32_t slots;
  const void* z;
  int64_t total_rows, ldz;
  const int32_t* row_of_slot;
  const int32_t* slot_of_row;
  const float* weights;
  void* dz;
  int64_t lddz;
  float* dw;
};
hipError_t launch_expert_combine_backward(const CombineBwdParams& p, hipStream_t s);

struct CkptParams {
  const uint16_t* x;
  int64_t rows, cols, ld;
  int32_t format, out_f32;
  uint8_t* codes;
  uint16_t* scales;
  void* out;
  int64_t ldo;
};
hipError_t launch_ckpt_save(const CkptParams& p, hipStream_t s);
hipError_t launch_ckpt_load(const CkptParams& p, hipStream_t s);

struct GatedParams {
  const uint16_t* in;  // gu, or dh
  int64_t ld_in;
  int64_t rows, width;
  int32_t act, format;
  uint8_t* codes;
  uint16_t* scales;
  uint16_t* h;  // forward output, or the backward's h (may be null there)
  int64_t ldh;
  uint16_t* dgu;
  int64_t lddg;
};
hipError_t launch_gated(const GatedParams& p, hipStream_t s);
hipError_t launch_gated_backward(const GatedParams& p, hipStream_t s);

// One operand of a grouped product: lines of codes and block scales along the
// reduction axis.  Matrix e starts at line e * seg_lines and, along the axis,
// at value e * seg_k.
struct GroupedOperand {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* ts;
  int64_t pitch;  // values a line
  int64_t seg_lines, seg_k;
};
struct GroupedParams {
  GroupedOperand a, b;
  const int64_t* offsets;
  int32_t groups, grid, c_f32;
  int64_t total_rows;  // nt: rows of a and c;  dw: padded_rows
  int64_t M, N, K;     // M: dw only; K: nt only
  void* c;
  int64_t ldc;
};
// 256 x 256 tiles of a call's grid (a launch takes fewer than 2^31).
int64_t grouped_tiles(const GroupedParams& p, bool dw);
hipError_t launch_grouped_nt(const GroupedParams& p, hipStream_t s);
hipError_t launch_grouped_dw(const GroupedParams& p, hipStream_t s);

}  // namespace ufp4
