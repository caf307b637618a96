// ufp4_cache.hip -- the 4-bit key-value cache: tokens' keys and values quantized
// as they are written, and read back.
//
// A workgroup takes 32 tokens of one head.  A lane takes a block of 16 values (fp32
// results: a quarter of one, so that stores of neighbouring lanes meet, and the last
// stages of the transform cross lanes).  Keys lie token by token in the cache.
// Values lie so that the tokens of one pair of neighbouring values are side by side
// in tiles of 32 (what the second product of attention reads): they pass through
// LDS, and leave or come byte by byte, neighbouring lanes neighbouring tokens.
//
// What bounds these kernels is the chain of a workgroup (slots, codes, LDS,
// results) and the vector work of a value, not the memory.  8191 tokens, 8 heads of
// 128, bf16 (43 MB): half a block a lane instead of one took 22 us, words of four
// tokens for the values instead of bytes, which have to be taken apart in LDS, 15.9.
#include "ufp4_serve.hpp"
#include "ufp4_vec.hpp"

namespace ufp4 {

namespace {

constexpr int kTok = 32;  // tokens of a workgroup (of one head)
constexpr int kCacheThreads = 256;
constexpr int kMaxHalf = 128;   // dim / 2
constexpr int kMaxBlocks = 16;  // dim / 16
constexpr int kPitch = kMaxHalf + 4;  // bytes of a token's values in LDS
constexpr int kScalePitch = kMaxBlocks + 4;

// A head's tensor scale: 1 unless the entry is a positive finite number.
__device__ __forceinline__ float head_scale(const float* ts, int h) {
  const float s = ts ? ts[h] : 1.0f;
  return s > 0.0f && s <= 3.40282347e38f ? s : 1.0f;
}

// Where the workgroup's tokens are: the token's index in its cache (page, head,
// token), -1 for none.
__device__ __forceinline__ void find_places(const CacheParams& p, int64_t t0, int h, int64_t* place) {
  const int t = threadIdx.x;
  if (t < kTok) {
    int64_t at = -1;
    if (t0 + t < p.tokens) {
      const int64_t slot = p.slots[t0 + t];
      if (slot >= 0 && slot < p.c.pages * p.c.page_tokens) {
        const int64_t page = slot / p.c.page_tokens;
        at = (page * p.c.heads + h) * p.c.page_tokens + (slot - page * p.c.page_tokens);
      }
    }
    place[t] = at;
  }
  __syncthreads();
}

// Bytes of the workgroup's tokens, `lines` lines (pairs of values or blocks) of one
// byte a token, between LDS ([token][line]) and the cache's tiles.
template <bool TO_CACHE>
__device__ __forceinline__ void move_lines(const int64_t* place, int lines, int pitch, uint8_t* cache, uint8_t* lds) {
  const int t = threadIdx.x & (kTok - 1);
  const int64_t at = place[t];
  if (at < 0) return;
  uint8_t* c = cache + (at & -kCacheTile) * lines + (at & (kCacheTile - 1));
  uint8_t* l = lds + t * pitch;
#pragma unroll 4
  for (int j = threadIdx.x / kTok; j < lines; j += kCacheThreads / kTok) {
    if (TO_CACHE) c[j * kCacheTile] = l[j];
    else l[j] = c[j * kCacheTile];
  }
}

// A block of 16 values to codes and their scale: transform, largest magnitude, E4M3
// scale under the tensor scale, rounding; the steps and their order are the
// quantizer's.
template <int GRID>
__device__ __forceinline__ void quantize16(const CacheParams& p, float v[16], float ts, v32x2& codes, uint32_t& scale) {
  if (p.rht) {
    fwht16_inlane(v, p.sg);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= p.sg.fin;
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

__device__ __forceinline__ void unpack16(const v32x4 w[2], float v[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const V8 a = unpack(w[h]);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[8 * h + j] = a.v[j];
  }
}

template <int GRID>
__global__ __launch_bounds__(kCacheThreads) void ufp4_cache_append_kernel(CacheParams p) {
  __shared__ int64_t place[kTok];
  __shared__ __attribute__((aligned(16))) uint8_t codes[kTok * kPitch];
  __shared__ __attribute__((aligned(16))) uint8_t scales[kTok * kScalePitch];
  const int h = blockIdx.y, tid = threadIdx.x, half = p.c.dim / 2, blocks = p.c.dim / 16;
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const uint16_t* k0 = p.k + t0 * p.ldk + h * p.c.dim;
  const uint16_t* v0 = p.v + t0 * p.ldv + h * p.c.dim;
  const int64_t left = p.tokens - t0;
  // the first block's values come while the places are found
  v32x4 k[2], v[2];
  auto fetch = [&](int i) {
    const int t = (int)p.pieces.div((uint32_t)i), b = i - t * blocks;
    if (t >= kTok || t >= left) return;
    const uint16_t* a = k0 + (uint64_t)t * (uint32_t)p.ldk + 16 * b;
    const uint16_t* c = v0 + (uint64_t)t * (uint32_t)p.ldv + 16 * b;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      k[j] = load16(a + 8 * j);
      v[j] = load16(c + 8 * j);
    }
  };
  fetch(tid);
  find_places(p, t0, h, place);
  const float kts = head_scale(p.c.kts, h), vts = head_scale(p.c.vts, h);
  for (int i = tid; i < kTok * blocks; i += kCacheThreads) {
    const int t = (int)p.pieces.div((uint32_t)i), b = i - t * blocks;
    if (i != tid) fetch(i);
    const int64_t at = place[t];
    if (at < 0) continue;
    float x[16];
    v32x2 w;
    uint32_t e;
    unpack16(k, x);
    quantize16<GRID>(p, x, kts, w, e);
    *reinterpret_cast<v32x2*>(p.c.kc + at * half + 8 * b) = w;
    p.c.ks[at * blocks + b] = (uint8_t)e;
    unpack16(v, x);
    quantize16<GRID>(p, x, vts, w, e);
    uint32_t* to = reinterpret_cast<uint32_t*>(codes + t * kPitch + 8 * b);
    to[0] = w.x;
    to[1] = w.y;
    scales[t * kScalePitch + b] = (uint8_t)e;
  }
  __syncthreads();
  move_lines<true>(place, half, kPitch, p.c.vc, codes);
  move_lines<true>(place, blocks, kScalePitch, p.c.vs, scales);
}

// Cross-lane value of the lane whose index differs in bit 0 or bit 1.
template <int N>
__device__ __forceinline__ float lane_xor(float v) {
  return N == 1 ? dpp_xor1(v) : dpp_xor2(v);
}

// N = 16 values of a block, or 4 that it shares with three neighbouring lanes (this
// one the part-th), from their codes: value * d with d = scale * tensor scale, then
// the inverse transform: butterflies without signs (h = 1, 2, 4, 8, the last two
// across lanes), 1/4, signs.
template <int GRID, int N>
__device__ __forceinline__ void dequantize(const CacheParams& p, v32x2 codes, uint32_t scale, float ts, int part, float v[N]) {
  const float d = e4m3_decode_pos(scale) * ts;
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = code_value<GRID>(codes[j >> 3] >> (4 * (j & 7))) * d;
  if (!p.rht) return;
#pragma unroll
  for (int h = 1; h < N; h <<= 1)
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (!(j & h)) {
        const float a = v[j], b = v[j + h];
        v[j] = a + b;
        v[j + h] = a - b;
      }
  if (N == 4) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float o = lane_xor<1>(v[j]);
      v[j] = part & 1 ? o - v[j] : v[j] + o;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float o = lane_xor<2>(v[j]);
      v[j] = part & 2 ? o - v[j] : v[j] + o;
    }
  }
  const uint32_t mine = N == 4 ? p.signs >> (N * part) : p.signs;
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = v[j] * ((mine >> j) & 1 ? -0.25f : 0.25f);
}

template <bool S>
__device__ __forceinline__ void store_piece(uint16_t* out, const float v[16]) {
#pragma unroll
  for (int h = 0; h < 16; h += 8)
    store_16<S>(out + h, v32x4{pack_bf16(v[h], v[h + 1]), pack_bf16(v[h + 2], v[h + 3]), pack_bf16(v[h + 4], v[h + 5]),
                            pack_bf16(v[h + 6], v[h + 7])});
}
template <bool S>
__device__ __forceinline__ void store_piece(float* out, const float v[4]) {
  store_16<S>(out, v32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
}

template <int GRID, typename TO, bool S>
__global__ __launch_bounds__(kCacheThreads) void ufp4_cache_read_kernel(CacheParams p) {
  constexpr int N = sizeof(TO) == 2 ? 16 : 4, kLanes = 16 / N;  // values a lane, lanes a block
  __shared__ int64_t place[kTok];
  __shared__ __attribute__((aligned(16))) uint8_t codes[kTok * kPitch];
  __shared__ __attribute__((aligned(16))) uint8_t scales[kTok * kScalePitch];
  const int h = blockIdx.y, tid = threadIdx.x, half = p.c.dim / 2, blocks = p.c.dim / 16, pieces = p.c.dim / N;
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  find_places(p, t0, h, place);
  // (the lanes of a block belong to one token: pieces is a multiple of kLanes)
  struct Item {
    int t, c;
    int64_t at;
    v32x2 w;
    uint32_t scale;
  };
  // a piece of keys, on its way while values come
  auto key = [&](int i) {
    Item x;
    x.t = (int)p.pieces.div((uint32_t)i);
    x.c = i - x.t * pieces;
    x.at = place[x.t];
    x.w = v32x2{0u, 0u};
    x.scale = 0;
    if (p.k_out && x.at >= 0) {
      if (N == 16) x.w = *reinterpret_cast<const v32x2*>(p.c.kc + x.at * half + 8 * x.c);
      else x.w.x = *reinterpret_cast<const uint16_t*>(p.c.kc + x.at * half + 2 * x.c);
      x.scale = p.c.ks[x.at * blocks + x.c / kLanes];
    }
    return x;
  };
  Item x = key(tid < kTok * pieces ? tid : 0);
  if (p.v_out) {
    move_lines<false>(place, half, kPitch, p.c.vc, codes);
    move_lines<false>(place, blocks, kScalePitch, p.c.vs, scales);
    __syncthreads();
  }
  const float kts = head_scale(p.c.kts, h), vts = head_scale(p.c.vts, h);
  TO* k0 = static_cast<TO*>(p.k_out) + t0 * p.ldk + h * p.c.dim;
  TO* v0 = static_cast<TO*>(p.v_out) + t0 * p.ldv + h * p.c.dim;
  for (int i = tid; i < kTok * pieces; i += kCacheThreads) {
    if (t0 + x.t >= p.tokens) break;
    const Item y = x;
    x = key(i + kCacheThreads < kTok * pieces ? i + kCacheThreads : 0);
    float v[N];
    if (p.k_out) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = 0.0f;
      if (y.at >= 0) dequantize<GRID, N>(p, y.w, y.scale, kts, y.c % kLanes, v);
      store_piece<S>(k0 + (uint64_t)y.t * (uint32_t)p.ldk + N * y.c, v);
    }
    if (p.v_out) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = 0.0f;
      if (y.at >= 0) {
        const uint8_t* from = codes + y.t * kPitch + N / 2 * y.c;
        v32x2 w = {0u, 0u};
        if (N == 16) w = v32x2{reinterpret_cast<const uint32_t*>(from)[0], reinterpret_cast<const uint32_t*>(from)[1]};
        else w.x = *reinterpret_cast<const uint16_t*>(from);
        dequantize<GRID, N>(p, w, scales[y.t * kScalePitch + y.c / kLanes], vts, y.c % kLanes, v);
      }
      store_piece<S>(v0 + (uint64_t)y.t * (uint32_t)p.ldv + N * y.c, v);
    }
  }
}

dim3 grid_of(const CacheParams& p) { return dim3((unsigned)((p.tokens + kTok - 1) / kTok), (unsigned)p.c.heads); }

template <int GRID>
hipError_t launch_read(const CacheParams& p0, hipStream_t s) {
  CacheParams p = p0;
  p.pieces = fast_div((uint32_t)p.c.dim / (p.out_f32 ? 4 : 16));
  const int64_t bytes = p.tokens * p.c.heads * p.c.dim * (p.out_f32 ? 4 : 2) * ((p.k_out != nullptr) + (p.v_out != nullptr));
  // past the caches where results and what else lies there do not fit.  Keys and values of
  // 8 x 128, bf16, outputs of three calls in turn, past the caches / through them: 128 MiB
  // 38 / 38 us, 160 45 / 47, 192 54 / 67, 256 69 / 108; with a kernel behind that reads
  // both 69 / 67, 98 / 101, 119 / 122, 174 / 172.  fp32, 4 x 160: 96 MiB 23 / 28, 160 37 /
  // 44, 256 59 / 99, read again 51 / 50, 92 / 101, 176 / 176.
  const bool past = bytes > kLastLevelCache / 2;
  if (p.out_f32 && past) ufp4_cache_read_kernel<GRID, float, true><<<grid_of(p), kCacheThreads, 0, s>>>(p);
  else if (p.out_f32) ufp4_cache_read_kernel<GRID, float, false><<<grid_of(p), kCacheThreads, 0, s>>>(p);
  else if (past) ufp4_cache_read_kernel<GRID, uint16_t, true><<<grid_of(p), kCacheThreads, 0, s>>>(p);
  else ufp4_cache_read_kernel<GRID, uint16_t, false><<<grid_of(p), kCacheThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_append(const CacheParams& p0, hipStream_t s) {
  CacheParams p = p0;
  p.pieces = fast_div((uint32_t)p.c.dim / 16);
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
