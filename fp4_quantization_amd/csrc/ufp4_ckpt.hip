// ufp4_ckpt.hip -- 8-bit activation checkpoints and the gated activation that
// keeps and uses them.
//
// A block of 32 values along a row is held by four neighbouring lanes, eight
// values (16 bytes of bf16) each; its largest magnitude takes two exchanges
// inside the quad.  Everything is one pass over the data, bound by memory:
// a lane's work item is (row, eighth of a block pair), items are laid out
// along the rows, so a wave's loads and stores are contiguous.
#include "ufp4_moe.hpp"
#include "ufp4_vec.hpp"

namespace ufp4 {

namespace {

constexpr int kCkptThreads = 256;
constexpr int64_t kMaxItems = (int64_t)1 << 30;

// f(g) = g sigma and f'(g) = sigma + g sigma (1 - sigma) y'(g) for the two
// gates, sigma = sigmoid(y): SiLU has y = g; tanh-GELU has
// y = 2 sqrt(2/pi) (g + 0.044715 g^3), infinite for large g, where sigma is 0 or 1.
// The exponential and reciprocal are the hardware's (1 ulp).  Below y = -80,
// where exp(-y) nears its overflow and the reciprocal its subnormal results,
// sigma is exp(y) itself, taken 2^64 too large (1 + exp(y) is 1 to the last bit);
// few waves hold such a value, the others skip it (for every value: 4096 x 2048,
// forward and backward, 28.9 us instead of 27.8 with GELU).
// So sigma is right to |y| 2^-23 relative, inside the bf16 rounding of every
// output, down to fp32's subnormal numbers, and to their step of 2^-149 there.
constexpr float kLog2e = 1.4426950408889634f;
template <int ACT>
__device__ __forceinline__ V8 gate_sigma(const V8& g) {
  V8 y, s;
  float lowest = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float t = g.v[k];
    y.v[k] = ACT == 0 ? t : 1.5957691216057308f * t * __builtin_fmaf(0.044715f * t, t, 1.0f);
    s.v[k] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * y.v[k]));
    lowest = fminf(lowest, y.v[k]);  // (passes over a NaN, whose sigma is NaN)
  }
  if (__any(lowest < -80.0f)) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (y.v[k] < -80.0f) s.v[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(kLog2e, y.v[k], 64.0f)) * 0x1p-64f;
  }
  return s;
}
// (GELU's y' is taken at a g clamped to +-16, beyond which sigma (1 - sigma) is 0
// and y' must not be infinite; a NaN, which the clamp drops, is in sg)
template <int ACT>
__device__ __forceinline__ float gate_slope(float g, float sg) {
  if (ACT == 0) return __builtin_fmaf(g * sg, 1.0f - sg, sg);
  const float t = fminf(fmaxf(g, -16.0f), 16.0f);
  const float dy = 1.5957691216057308f * __builtin_fmaf(0.134145f * t, t, 1.0f);
  return __builtin_fmaf(t * dy * sg, 1.0f - sg, sg);
}

// One row position of an item: row and first column of its eight values, and
// how many of them the row has (0 for the lanes behind a short last block).
struct Item {
  int64_t row;
  int32_t col, n, block;
};
__device__ __forceinline__ Item item_of(uint32_t i, int64_t row0, const FastDiv& lanes, int32_t width) {
  Item it;
  const uint32_t r = lanes.div(i);
  const int32_t v = (int32_t)(i - r * lanes.d);
  it.row = row0 + r;
  it.col = 8 * v;
  it.block = v >> 2;
  const int32_t left = width - it.col;
  it.n = left < 0 ? 0 : (left < 8 ? left : 8);
  return it;
}

// 65536 x 4096: save 136 us, 6.1 TB/s, load 144, 5.7; 8192 x 4096 18 us; 4099 x
// 1365, odd alignment, 6.0 us, 2.9 TB/s.
template <int FMT>
__global__ __launch_bounds__(kCkptThreads) void ufp4_ckpt_save_kernel(CkptParams p, int64_t row0, uint32_t items,
                                                                      FastDiv lanes) {
  const uint32_t i = blockIdx.x * kCkptThreads + threadIdx.x;
  if (i >= items) return;
  const Item it = item_of(i, row0, lanes, (int32_t)p.cols);
  const v32x4 w = row_bits(p.x + it.row * p.ld + it.col, it.n);
  const uint32_t s = ckpt_scale<FMT>(quad_max(bits_max(w)));
  code_store(p.codes + it.row * p.cols + it.col, ckpt_encode<FMT>(w, s), it.n);
  if ((i & 3) == 0) p.scales[it.row * (lanes.d >> 2) + it.block] = (uint16_t)s;
}

template <int FMT, typename T>
__global__ __launch_bounds__(kCkptThreads) void ufp4_ckpt_load_kernel(CkptParams p, int64_t row0, uint32_t items,
                                                                      FastDiv lanes) {
  const uint32_t i = blockIdx.x * kCkptThreads + threadIdx.x;
  if (i >= items) return;
  const Item it = item_of(i, row0, lanes, (int32_t)p.cols);
  const float s = from_bf16(p.scales[it.row * (lanes.d >> 2) + it.block]);
  const v32x2 c = code_bits(p.codes + it.row * p.cols + it.col, it.n);
  row_store(static_cast<T*>(p.out) + it.row * p.ldo + it.col, ckpt_decode<FMT>(c, s), it.n);
}

// FMT < 0: nothing is kept.  S: past the caches.  The exponentials and the codes
// hide behind memory: 65536 x 2048 with an INT8 checkpoint 172 us for 1.09 GB,
// 6.3 TB/s, its backward pass 225 us for 1.36 GB, 6.0 TB/s; 8 rows 2.8 us.
template <int ACT, int FMT, bool S>
__global__ __launch_bounds__(kCkptThreads) void ufp4_gated_kernel(GatedParams p, int64_t row0, uint32_t items,
                                                                  FastDiv lanes) {
  const uint32_t i = blockIdx.x * kCkptThreads + threadIdx.x;
  if (i >= items) return;
  const Item it = item_of(i, row0, lanes, (int32_t)p.width);
  const uint16_t* src = p.in + it.row * p.ld_in + it.col;
  const v32x4 gw = row_bits<S>(src, it.n), uw = row_bits<S>(src + p.width, it.n);
  const V8 g = unpack(gw), u = unpack(uw), sig = gate_sigma<ACT>(g);
  V8 h;
#pragma unroll
  for (int k = 0; k < 8; ++k) h.v[k] = g.v[k] * sig.v[k] * u.v[k];
  row_store<S>(p.h + it.row * p.ldh + it.col, h, it.n);
  if constexpr (FMT >= 0) {
    const uint32_t sg = ckpt_scale<FMT>(quad_max(bits_max(gw))), su = ckpt_scale<FMT>(quad_max(bits_max(uw)));
    uint8_t* dst = p.codes + it.row * 2 * p.width + it.col;
    code_store<S>(dst, ckpt_encode<FMT>(gw, sg), it.n);
    code_store<S>(dst + p.width, ckpt_encode<FMT>(uw, su), it.n);
    const int32_t nb = (int32_t)(lanes.d >> 2);
    if ((i & 3) < 2) p.scales[it.row * 2 * nb + ((i & 3) ? nb : 0) + it.block] = (uint16_t)((i & 3) ? su : sg);
  }
}

template <int ACT, int FMT, bool S>
__global__ __launch_bounds__(kCkptThreads) void ufp4_gated_bwd_kernel(GatedParams p, int64_t row0, uint32_t items,
                                                                      FastDiv lanes) {
  const uint32_t i = blockIdx.x * kCkptThreads + threadIdx.x;
  if (i >= items) return;
  const Item it = item_of(i, row0, lanes, (int32_t)p.width);
  const int32_t nb = (int32_t)(lanes.d >> 2);
  const uint16_t* sc = p.scales + it.row * 2 * nb + it.block;
  const float sg = from_bf16(sc[0]), su = from_bf16(sc[nb]);
  const uint8_t* src = p.codes + it.row * 2 * p.width + it.col;
  const v32x2 gc = code_bits<S>(src, it.n), uc = code_bits<S>(src + p.width, it.n);
  const V8 dh = unpack(row_bits<S>(p.in + it.row * p.ld_in + it.col, it.n));
  const V8 g = ckpt_decode<FMT>(gc, sg), u = ckpt_decode<FMT>(uc, su), sig = gate_sigma<ACT>(g);
  V8 dg, du, h;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float f = g.v[k] * sig.v[k];
    dg.v[k] = dh.v[k] * u.v[k] * gate_slope<ACT>(g.v[k], sig.v[k]);
    du.v[k] = dh.v[k] * f;
    h.v[k] = f * u.v[k];
  }
  uint16_t* dst = p.dgu + it.row * p.lddg + it.col;
  row_store<S>(dst, dg, it.n);
  row_store<S>(dst + p.width, du, it.n);
  if (p.h) row_store<S>(p.h + it.row * p.ldh + it.col, h, it.n);
}

// Launches over slices of rows of at most 2^30 items (31-bit item indices).
template <typename F>
hipError_t over_rows(int64_t rows, int64_t width, F launch) {
  const int64_t lanes = 4 * ((width + kCkptBlock - 1) / kCkptBlock);
  const int64_t step = kMaxItems / lanes;
  for (int64_t r0 = 0; r0 < rows; r0 += step) {
    const int64_t n = rows - r0 < step ? rows - r0 : step;
    const uint32_t items = (uint32_t)(n * lanes);
    launch(dim3((items + kCkptThreads - 1) / kCkptThreads), r0, items, fast_div((uint32_t)lanes));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_ckpt_save(const CkptParams& p, hipStream_t s) {
  return over_rows(p.rows, p.cols, [&](dim3 g, int64_t r0, uint32_t n, FastDiv d) {
    if (p.format == kCkptINT8)
      ufp4_ckpt_save_kernel<kCkptINT8><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
    else
      ufp4_ckpt_save_kernel<kCkptE4M3><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
  });
}

hipError_t launch_ckpt_load(const CkptParams& p, hipStream_t s) {
  return over_rows(p.rows, p.cols, [&](dim3 g, int64_t r0, uint32_t n, FastDiv d) {
    if (p.format == kCkptINT8) {
      if (p.out_f32)
        ufp4_ckpt_load_kernel<kCkptINT8, float><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
      else
        ufp4_ckpt_load_kernel<kCkptINT8, uint16_t><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
    } else {
      if (p.out_f32)
        ufp4_ckpt_load_kernel<kCkptE4M3, float><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
      else
        ufp4_ckpt_load_kernel<kCkptE4M3, uint16_t><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
    }
  });
}

namespace {

// Calls that move more than the last-level cache holds go past the caches
// (forward and backward of 65536 x 2048: 430 -> 395 us; of 4096 x 2048, whose
// checkpoint the backward pass still finds in the cache: 27 -> 30 us).
template <bool S>
hipError_t gated(const GatedParams& p, hipStream_t s) {
  return over_rows(p.rows, p.width, [&](dim3 g, int64_t r0, uint32_t n, FastDiv d) {
    const int f = p.codes ? p.format : -1;
    if (p.act == 0) {
      if (f < 0) ufp4_gated_kernel<0, -1, S><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
      else if (f == kCkptINT8) ufp4_gated_kernel<0, kCkptINT8, S><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
      else ufp4_gated_kernel<0, kCkptE4M3, S><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
    } else {
      if (f < 0) ufp4_gated_kernel<1, -1, S><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
      else if (f == kCkptINT8) ufp4_gated_kernel<1, kCkptINT8, S><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
      else ufp4_gated_kernel<1, kCkptE4M3, S><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
    }
  });
}

template <bool S>
hipError_t gated_backward(const GatedParams& p, hipStream_t s) {
  return over_rows(p.rows, p.width, [&](dim3 g, int64_t r0, uint32_t n, FastDiv d) {
    if (p.act == 0) {
      if (p.format == kCkptINT8) ufp4_gated_bwd_kernel<0, kCkptINT8, S><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
      else ufp4_gated_bwd_kernel<0, kCkptE4M3, S><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
    } else {
      if (p.format == kCkptINT8) ufp4_gated_bwd_kernel<1, kCkptINT8, S><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
      else ufp4_gated_bwd_kernel<1, kCkptE4M3, S><<<g, kCkptThreads, 0, s>>>(p, r0, n, d);
    }
  });
}

}  // namespace

hipError_t launch_gated(const GatedParams& p, hipStream_t s) {
  return p.rows * p.width * (p.codes ? 8 : 6) > kLastLevelCache ? gated<true>(p, s) : gated<false>(p, s);
}

hipError_t launch_gated_backward(const GatedParams& p, hipStream_t s) {
  return p.rows * p.width * (p.h ? 10 : 8) > kLastLevelCache ? gated_backward<true>(p, s) : gated_backward<false>(p, s);
}

}  // namespace ufp4
