// ufp4_cache.hip -- the 4-bit key-value cache: tokens' keys and values quantized
// as they are written, and read back.
//
// A block of 16 values along a head is one lane's: transform, largest magnitude,
// E4M3 scale under the head's tensor scale, codes (the NV16 steps of the
// quantizer, ufp4_device.hpp).  Keys lie token by token.  Values lie so that
// the tokens of one pair of neighbouring values are side by side in tiles of 32
// (what the second product of attention reads), so they pass through LDS and
// leave, or come, as bytes of neighbouring tokens.
#include "ufp4_serve.hpp"
#include "ufp4_vec.hpp"

namespace ufp4 {

namespace {

constexpr int kTok = 32;  // tokens of a workgroup (of one head)
constexpr int kCacheThreads = 256;
constexpr int kMaxHalf = 128;            // dim / 2
constexpr int kMaxBlocks = 16;           // dim / 16
constexpr int kPitch = kMaxHalf + 4;     // bytes of a token's values in LDS

// A head's tensor scale: 1 unless the entry is a positive finite number.
__device__ __forceinline__ float head_scale(const float* ts, int h) {
  const float s = ts ? ts[h] : 1.0f;
  return s > 0.0f && s <= 3.40282347e38f ? s : 1.0f;
}

struct Place {
  int64_t page;  // -1: none
  int32_t at;
};
__device__ __forceinline__ Place place_of(const CacheView& c, int64_t slot) {
  if (slot < 0 || slot >= c.pages * c.page_tokens) return Place{-1, 0};
  const int64_t page = slot / c.page_tokens;
  return Place{page, (int32_t)(slot - page * c.page_tokens)};
}
// Bytes before a token's key codes (dim/2 each; scales dim/16 each), and before
// its tile's value codes.
__device__ __forceinline__ int64_t token_at(const CacheView& c, Place s, int h) {
  return (s.page * c.heads + h) * c.page_tokens + s.at;
}

template <int GRID>
__device__ __forceinline__ void quantize16(float v[16], const RhtSigns* sg, float ts, v32x2& codes, uint32_t& scale) {
  if (sg) {
    fwht16_inlane(v, *sg);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= sg->fin;
  }
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) m = fabsf(v[j]) > m ? fabsf(v[j]) : m;
  scale = e4m3_encode_sat(m / (grid_qmax<GRID>() * ts));
  const float d = e4m3_decode_pos(scale) * ts;
  const float inv = d > 0.0f ? 1.0f / d : 0.0f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) c |= round_rtne<GRID>(v[8 * w + j] * inv) << (4 * j);
    codes[w] = c;
  }
}

__device__ __forceinline__ void load16v(const uint16_t* x, float v[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const V8 a = row_load(x + 8 * h, 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[8 * h + j] = a.v[j];
  }
}

template <int GRID>
__global__ __launch_bounds__(kCacheThreads) void ufp4_cache_append_kernel(CacheParams p) {
  __shared__ Place place[kTok];
  __shared__ __attribute__((aligned(16))) uint8_t codes[kTok * kPitch];
  __shared__ uint8_t scales[kTok][kMaxBlocks + 4];
  const int h = blockIdx.y, tid = threadIdx.x, half = p.c.dim / 2, blocks = p.c.dim / 16;
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  if (tid < kTok) place[tid] = t0 + tid < p.tokens ? place_of(p.c, p.slots[t0 + tid]) : Place{-1, 0};
  __syncthreads();
  const float kts = head_scale(p.c.kts, h), vts = head_scale(p.c.vts, h);
  for (int i = tid; i < kTok * blocks; i += kCacheThreads) {
    const int t = i / blocks, b = i - t * blocks;
    const Place s = place[t];
    if (s.page < 0) continue;
    float v[16];
    v32x2 c;
    uint32_t e;
    load16v(p.k + (t0 + t) * p.ldk + h * p.c.dim + 16 * b, v);
    quantize16<GRID>(v, p.rht ? &p.sg : nullptr, kts, c, e);
    const int64_t at = token_at(p.c, s, h);
    *reinterpret_cast<v32x2*>(p.c.kc + at * half + 8 * b) = c;
    p.c.ks[at * blocks + b] = (uint8_t)e;
    load16v(p.v + (t0 + t) * p.ldv + h * p.c.dim + 16 * b, v);
    quantize16<GRID>(v, p.rht ? &p.sg : nullptr, vts, c, e);
    uint32_t* to = reinterpret_cast<uint32_t*>(codes + t * kPitch + 8 * b);
    to[0] = c.x;
    to[1] = c.y;
    scales[t][b] = (uint8_t)e;
  }
  __syncthreads();
  // neighbouring lanes: neighbouring tokens, whose bytes are neighbours if their
  // slots are
  const int t = tid & (kTok - 1);
  const Place s = place[t];
  if (s.page < 0) return;
  const int64_t tile = (token_at(p.c, s, h) - s.at % kCacheTile) / kCacheTile;
  uint8_t* vc = p.c.vc + tile * half * kCacheTile + s.at % kCacheTile;
  uint8_t* vs = p.c.vs + tile * blocks * kCacheTile + s.at % kCacheTile;
  for (int j = tid / kTok; j < half; j += kCacheThreads / kTok) vc[j * kCacheTile] = codes[t * kPitch + j];
  for (int b = tid / kTok; b < blocks; b += kCacheThreads / kTok) vs[b * kCacheTile] = scales[t][b];
}

// Codes times d = scale * tensor scale, and the inverse transform: butterflies
// without signs, 1/4, signs.
template <int GRID>
__device__ __forceinline__ void dequantize16(v32x2 c, uint32_t scale, float ts, const float* d16, float v[16]) {
  const float d = e4m3_decode_pos(scale) * ts;
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = code_value<GRID>((j < 8 ? c.x : c.y) >> (4 * (j & 7))) * d;
  if (!d16) return;
  RhtSigns plain;
#pragma unroll
  for (int k = 0; k < 8; ++k) plain.q1[k] = 1.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) plain.q2[k] = 1.0f;
  plain.q3[0] = plain.q3[1] = 1.0f;
  plain.q4 = 1.0f;
  plain.fin = 0.25f;
  fwht16_inlane(v, plain);
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = v[j] * (0.25f * d16[j]);
}

template <typename TO>
__device__ __forceinline__ void store16v(TO* out, const float v[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    V8 a;
#pragma unroll
    for (int j = 0; j < 8; ++j) a.v[j] = v[8 * h + j];
    row_store(out + 8 * h, a, 8);
  }
}

template <int GRID, typename TO>
__global__ __launch_bounds__(kCacheThreads) void ufp4_cache_read_kernel(CacheParams p) {
  __shared__ Place place[kTok];
  __shared__ __attribute__((aligned(16))) uint8_t codes[kTok * kPitch];
  __shared__ uint8_t scales[kTok][kMaxBlocks + 4];
  const int h = blockIdx.y, tid = threadIdx.x, half = p.c.dim / 2, blocks = p.c.dim / 16;
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  if (tid < kTok) place[tid] = t0 + tid < p.tokens ? place_of(p.c, p.slots[t0 + tid]) : Place{-1, 0};
  __syncthreads();
  if (p.v_out) {
    const int t = tid & (kTok - 1);
    const Place s = place[t];
    if (s.page >= 0) {
      const int64_t tile = (token_at(p.c, s, h) - s.at % kCacheTile) / kCacheTile;
      const uint8_t* vc = p.c.vc + tile * half * kCacheTile + s.at % kCacheTile;
      const uint8_t* vs = p.c.vs + tile * blocks * kCacheTile + s.at % kCacheTile;
      for (int j = tid / kTok; j < half; j += kCacheThreads / kTok) codes[t * kPitch + j] = vc[j * kCacheTile];
      for (int b = tid / kTok; b < blocks; b += kCacheThreads / kTok) scales[t][b] = vs[b * kCacheTile];
    }
    __syncthreads();
  }
  const float kts = head_scale(p.c.kts, h), vts = head_scale(p.c.vts, h);
  for (int i = tid; i < kTok * blocks; i += kCacheThreads) {
    const int t = i / blocks, b = i - t * blocks;
    if (t0 + t >= p.tokens) break;
    const Place s = place[t];
    const int64_t at = s.page < 0 ? 0 : token_at(p.c, s, h);
    float v[16];
    if (p.k_out) {
      if (s.page < 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.0f;
      } else {
        dequantize16<GRID>(*reinterpret_cast<const v32x2*>(p.c.kc + at * half + 8 * b), p.c.ks[at * blocks + b], kts,
                           p.rht ? p.d : nullptr, v);
      }
      store16v(static_cast<TO*>(p.k_out) + (t0 + t) * p.ldk + h * p.c.dim + 16 * b, v);
    }
    if (p.v_out) {
      if (s.page < 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.0f;
      } else {
        const uint32_t* c = reinterpret_cast<const uint32_t*>(codes + t * kPitch + 8 * b);
        dequantize16<GRID>(v32x2{c[0], c[1]}, scales[t][b], vts, p.rht ? p.d : nullptr, v);
      }
      store16v(static_cast<TO*>(p.v_out) + (t0 + t) * p.ldv + h * p.c.dim + 16 * b, v);
    }
  }
}

dim3 grid_of(const CacheParams& p) { return dim3((unsigned)((p.tokens + kTok - 1) / kTok), (unsigned)p.c.heads); }

template <int GRID>
hipError_t launch_read(const CacheParams& p, hipStream_t s) {
  if (p.out_f32) ufp4_cache_read_kernel<GRID, float><<<grid_of(p), kCacheThreads, 0, s>>>(p);
  else ufp4_cache_read_kernel<GRID, uint16_t><<<grid_of(p), kCacheThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(const CacheParams& p, hipStream_t s) {
  switch (p.grid) {
    case kGridE1M2: ufp4_cache_append_kernel<kGridE1M2><<<grid_of(p), kCacheThreads, 0, s>>>(p); break;
    case kGridINT4: ufp4_cache_append_kernel<kGridINT4><<<grid_of(p), kCacheThreads, 0, s>>>(p); break;
    case kGridE2M1: ufp4_cache_append_kernel<kGridE2M1><<<grid_of(p), kCacheThreads, 0, s>>>(p); break;
    case kGridE2M1C: ufp4_cache_append_kernel<kGridE2M1C><<<grid_of(p), kCacheThreads, 0, s>>>(p); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheParams& p, hipStream_t s) {
  switch (p.grid) {
    case kGridE1M2: return launch_read<kGridE1M2>(p, s);
    case kGridINT4: return launch_read<kGridINT4>(p, s);
    case kGridE2M1:  // the clamped grid's codes are E2M1 codes
    case kGridE2M1C: return launch_read<kGridE2M1>(p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace ufp4
