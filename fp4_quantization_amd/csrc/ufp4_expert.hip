// ufp4_expert.hip -- the token side of the expert layer: a stable sort of
// slots by expert, the rows to their experts (dispatch), the weighted sum back
// (combine) and its gradients.
#include "ufp4_moe.hpp"
#include "ufp4_vec.hpp"

namespace ufp4 {

namespace {

// ------------------------------------------------------------------ sort
// A counting sort whose order is fixed by construction (no atomic decides a
// position): slots are cut into at most kSortBlocks blocks of whole chunks of
// kSortThreads.
//   count: each block counts its slots by expert.  The counts of block b are
//     kept in the block's own stretch of row_of_slot (at least 1024 entries),
//     which holds nothing yet, so the sort needs no workspace.
//   scan:  one workgroup turns them into the first row of every (block,
//     expert) and writes the offsets and the padding of the segments.
//   place: each block ranks its slots, chunk by chunk.  A slot's rank among the
//     slots of its expert inside a wave comes from ballots of the id's bits;
//     the waves' counts are summed in LDS.
// Up to kSortSingle slots one workgroup does all three in one launch.  Bound by
// the launches and, in the scan, by the one workgroup's latencies: 65536 slots,
// 64 experts 4.8 + 7.7 + 4.9 us as profiled, 13 in a call (counting with atomics on
// one array would save the scan's loads but not fix the order); 64 slots 4.0 us in one
// launch.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortBlocks = 64;
constexpr int kSortSingle = 5120;  // (one launch 9.7 us at 4000 slots, 15.6 at 8192; three launches 12 to 13)
constexpr int kSortMaxE = kMaxExperts + 1;  // + the key of dropped slots

__device__ __forceinline__ int sort_key(const SortParams& p, int s) {
  const uint32_t t = p.slots.div((uint32_t)s);
  const int32_t id = p.ids[(int64_t)t * p.ld_ids + (s - (int)(t * p.slots.d))];
  return (uint32_t)id < (uint32_t)p.experts ? id : p.experts;
}

// Exclusive sum over the workgroup's threads; *total gets the whole.
__device__ __forceinline__ int block_scan(int v, int* wsum, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    const int x = wsum[w];
    before += w < wave ? x : 0;
    all += x;
  }
  __syncthreads();
  *total = all;
  return before + inc - v;
}

// Thread e's segment: offsets of the segments and the padding rows of segment
// e, given the number of its slots; returns its first row.
__device__ int sort_offsets(const SortParams& p, int count, int* wsum) {
  const int e = threadIdx.x;
  const int padded = e < p.experts ? (count + p.align - 1) / p.align * p.align : 0;
  int total;
  const int first = block_scan(padded, wsum, &total);
  if (e < p.experts) {
    p.offsets[e] = first;
    for (int r = first + count; r < first + padded; ++r) p.slot_of_row[r] = -1;
  }
  if (e == 0) {
    p.offsets[p.experts] = total;
    p.offsets[p.experts + 1] = p.total_rows;
  }
  return first;
}

struct SortLds {
  int base[kSortMaxE];
  int pre[kSortWaves][kSortMaxE];
  int wsum[kSortWaves];
};

// Places the slots [s0, s1) given the first free row of every expert in
// L.base.  Every thread of the workgroup takes part.
__device__ void sort_place(const SortParams& p, int s0, int s1, SortLds& L) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int bits = 32 - __builtin_clz((uint32_t)p.experts);  // keys 0 .. experts
  for (int c = s0; c < s1; c += kSortThreads) {
    const int s = c + t;
    const bool in = s < s1;
    const int key = in ? sort_key(p, s) : p.experts;
    if (t <= p.experts)
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) L.pre[w][t] = 0;
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const bool one = (key >> b) & 1;
      const uint64_t m = __ballot(one);
      same &= one ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    __syncthreads();
    if (rank == 0) L.pre[wave][key] = __popcll(same);
    __syncthreads();
    if (t < p.experts) {
      int at = L.base[t];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const int n = L.pre[w][t];
        L.pre[w][t] = at;
        at += n;
      }
      L.base[t] = at;
    }
    __syncthreads();
    if (in) {
      const int row = key < p.experts ? L.pre[wave][key] + rank : -1;
      p.row_of_slot[s] = row;
      if (row >= 0) p.slot_of_row[row] = s;
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(kSortThreads) void ufp4_sort_single_kernel(SortParams p) {
  __shared__ SortLds L;
  const int t = threadIdx.x;
  L.base[t] = 0;
  __syncthreads();
  for (int s = t; s < p.n; s += kSortThreads) atomicAdd(&L.base[sort_key(p, s)], 1);
  __syncthreads();
  const int count = t < p.experts ? L.base[t] : 0;
  __syncthreads();
  const int first = sort_offsets(p, count, L.wsum);
  if (t < p.experts) L.base[t] = first;
  // rows behind the last segment
  int total = 0;
  block_scan(t < p.experts ? (count + p.align - 1) / p.align * p.align : 0, L.wsum, &total);
  for (int r = total + t; r < p.total_rows; r += kSortThreads) p.slot_of_row[r] = -1;
  __syncthreads();
  sort_place(p, 0, p.n, L);
}

__global__ __launch_bounds__(kSortThreads) void ufp4_sort_count_kernel(SortParams p, int per) {
  __shared__ int cnt[kSortMaxE];
  const int t = threadIdx.x, b = blockIdx.x;
  cnt[t] = 0;
  __syncthreads();
  const int s0 = b * per, s1 = b + 1 == (int)gridDim.x ? p.n : s0 + per;
  for (int s = s0 + t; s < s1; s += kSortThreads) atomicAdd(&cnt[sort_key(p, s)], 1);
  __syncthreads();
  if (t < p.experts) p.row_of_slot[s0 + t] = cnt[t];
}

// (a thread holds its expert's counts of all blocks, read together)
__global__ __launch_bounds__(kSortThreads) void ufp4_sort_scan_kernel(SortParams p, int per, int blocks) {
  __shared__ int wsum[kSortWaves];
  const int t = threadIdx.x;
  int n[kSortBlocks], count = 0;
  const int32_t* mine = p.row_of_slot + (t < p.experts ? t : p.experts - 1);
#pragma unroll
  for (int b = 0; b < kSortBlocks; ++b) n[b] = mine[(b < blocks ? b : blocks - 1) * per];  // (in bounds, no branches)
#pragma unroll
  for (int b = 0; b < kSortBlocks; ++b) n[b] = t < p.experts && b < blocks ? n[b] : 0;
#pragma unroll
  for (int b = 0; b < kSortBlocks; ++b) count += n[b];
  int at = sort_offsets(p, count, wsum);
#pragma unroll
  for (int b = 0; b < kSortBlocks; ++b)
    if (t < p.experts && b < blocks) {
      p.row_of_slot[b * per + t] = at;
      at += n[b];
    }
}

__global__ __launch_bounds__(kSortThreads) void ufp4_sort_place_kernel(SortParams p, int per) {
  __shared__ SortLds L;
  const int t = threadIdx.x, b = blockIdx.x;
  const int s0 = b * per, s1 = b + 1 == (int)gridDim.x ? p.n : s0 + per;
  if (t < p.experts) L.base[t] = p.row_of_slot[s0 + t];
  const int tail = (int)p.offsets[p.experts];
  for (int r = tail + b * kSortThreads + t; r < p.total_rows; r += gridDim.x * kSortThreads) p.slot_of_row[r] = -1;
  __syncthreads();
  sort_place(p, s0, s1, L);
}

// -------------------------------------------------------------- dispatch
// Each source row is read once and stored to the rows of its slots: an item is
// eight columns of a token.  The workgroups past the tokens' look for padding
// rows, kPadRows a wave, and zero them.  Bound by the stores: 8192 tokens of 4096
// to 8 of 64 experts 111 us for 613 MB, 5.5 TB/s, where a copy reaches 4.7 and a
// fill 6.8 (a workgroup per output row would read every token eight times).
// Calls of one generation of waves are bound by a wave's own course instead, one
// round of loads and then its stores: 3001 tokens of 1365 from an 8-bit checkpoint,
// 4 slots, 8.6 waves a SIMD, 13.7 us for 40 MB (widths of whole 16 bytes 11.7),
// where a fill of the output takes 7.0.
constexpr int kRowThreads = 256, kPadRows = 16;

// The rows of up to kSlotGroup slots from j0 on, read together (a slot past the
// last one reads the last one's place); -1 where there is none.
constexpr int kSlotGroup = 8;
__device__ __forceinline__ void load_rows(const int32_t* rs, int j0, int slots, int64_t total_rows, int32_t (&r)[kSlotGroup]) {
#pragma unroll
  for (int j = 0; j < kSlotGroup; ++j) r[j] = rs[j0 + j < slots ? j0 + j : slots - 1];
#pragma unroll
  for (int j = 0; j < kSlotGroup; ++j) r[j] = j0 + j < slots && r[j] >= 0 && r[j] < total_rows ? r[j] : -1;
}

// Eight values of a row as loaded, so that the loads of several rows can be
// under way together; those of no row count as zeros whatever row was read.
struct Raw16 {
  v32x4 w;
};
struct Raw32 {
  v32x4 a, b;
};
template <bool S>
__device__ __forceinline__ Raw16 raw_load(const uint16_t* p, int n) {
  return Raw16{row_bits<S>(p, n)};
}
template <bool S>
__device__ __forceinline__ Raw32 raw_load(const float* p, int n) {
  const V8 v = row_load<S>(p, n);
  Raw32 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.a[i] = __float_as_uint(v.v[i]);
    r.b[i] = __float_as_uint(v.v[4 + i]);
  }
  return r;
}
__device__ __forceinline__ V8 raw_values(const Raw16& r, bool ok) {
  const v32x4 none = {0u, 0u, 0u, 0u};
  return unpack(ok ? r.w : none);
}
__device__ __forceinline__ V8 raw_values(const Raw32& r, bool ok) {
  V8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.v[i] = ok ? __uint_as_float(r.a[i]) : 0.0f;
    v.v[4 + i] = ok ? __uint_as_float(r.b[i]) : 0.0f;
  }
  return v;
}
template <typename T>
struct RawOf;
template <>
struct RawOf<uint16_t> {
  using type = Raw16;
};
template <>
struct RawOf<float> {
  using type = Raw32;
};

// Source of eight values: bf16 rows, or a checkpoint (FMT).
template <int FMT>
__device__ __forceinline__ v32x4 dispatch_load(const DispatchParams& p, int64_t t, int32_t col, int n) {
  if constexpr (FMT < 0) {
    return row_bits(p.x + t * p.ld + col, n);
  } else {
    const int64_t nb = (p.cols + kCkptBlock - 1) / kCkptBlock;
    const float s = from_bf16(p.scales[t * nb + (col >> 5)]);
    return pack(ckpt_decode<FMT>(code_bits(p.codes + t * p.cols + col, n), s));
  }
}

// Zeroes the rows of [r0, r0 + kPadRows) that are padding; one wave.
template <typename T>
__device__ void zero_padding(const int32_t* slot_of_row, int64_t slots_total, int64_t r0, int64_t total_rows, T* out,
                             int64_t ld, int64_t cols) {
  const int lane = threadIdx.x & 63;
  const int64_t r = r0 + lane;
  bool pad = false;
  if (lane < kPadRows && r < total_rows) {
    const int32_t s = slot_of_row[r];
    pad = s < 0 || s >= slots_total;
  }
  uint64_t m = __ballot(pad);
  while (m) {
    const int i = __ffsll((unsigned long long)m) - 1;
    m &= m - 1;
    T* row = out + (r0 + i) * ld;
    for (int64_t c = 8 * lane; c < cols; c += 512) row_store(row + c, V8{}, cols - c < 8 ? (int)(cols - c) : 8);
  }
}

// S: stores past the caches.
template <int FMT, bool S>
__global__ __launch_bounds__(kRowThreads) void ufp4_dispatch_kernel(DispatchParams p, int64_t t0, uint32_t items,
                                                                    uint32_t item_wgs, FastDiv lanes) {
  if (blockIdx.x >= item_wgs) {
    const int64_t w = (int64_t)(blockIdx.x - item_wgs) * (kRowThreads / 64) + (threadIdx.x >> 6);
    zero_padding(p.slot_of_row, p.tokens * p.slots, w * kPadRows, p.total_rows, p.out, p.ldo, p.cols);
    return;
  }
  const uint32_t i = blockIdx.x * kRowThreads + threadIdx.x;
  if (i >= items) return;
  const uint32_t tt = lanes.div(i);
  const int32_t col = (int32_t)(8 * (i - tt * lanes.d));
  const int64_t t = t0 + tt;
  const int n = p.cols - col < 8 ? (int)(p.cols - col) : 8;
  const int32_t* rs = p.row_of_slot + t * p.slots;
  int32_t r[kSlotGroup];
  load_rows(rs, 0, p.slots, p.total_rows, r);
  const v32x4 w = dispatch_load<FMT>(p, t, col, n);
  for (int j0 = 0;;) {
#pragma unroll
    for (int j = 0; j < kSlotGroup; ++j)
      if (r[j] >= 0) row_store_bits<S>(p.out + (int64_t)r[j] * p.ldo + col, w, n);
    j0 += kSlotGroup;
    if (j0 >= p.slots) break;
    load_rows(rs, j0, p.slots, p.total_rows, r);
  }
}

// --------------------------------------------------------------- combine
// An item is eight columns of a token: the rows of its slots are read and
// summed in slot order in fp32.  Bound by the loads of z: 8192 tokens of 4096, 8
// slots, 95 us for 604 MB, 6.3 TB/s; 5119 of 2050, 6 slots, some dropped, 24 us.
template <typename TZ, typename TO, bool S>
__global__ __launch_bounds__(kRowThreads) void ufp4_combine_kernel(CombineParams p, int64_t t0, uint32_t items,
                                                                   FastDiv lanes) {
  const uint32_t i = blockIdx.x * kRowThreads + threadIdx.x;
  if (i >= items) return;
  const uint32_t tt = lanes.div(i);
  const int32_t col = (int32_t)(8 * (i - tt * lanes.d));
  const int64_t t = t0 + tt;
  const int n = p.cols - col < 8 ? (int)(p.cols - col) : 8;
  const int32_t* rs = p.row_of_slot + t * p.slots;
  V8 acc{};
  for (int j0 = 0; j0 < p.slots && p.total_rows > 0; j0 += kSlotGroup) {
    int32_t r[kSlotGroup];
    float w[kSlotGroup];
    typename RawOf<TZ>::type z[kSlotGroup];
    load_rows(rs, j0, p.slots, p.total_rows, r);
#pragma unroll
    for (int j = 0; j < kSlotGroup; ++j)
      w[j] = p.weights ? p.weights[t * p.slots + (j0 + j < p.slots ? j0 + j : p.slots - 1)] : 1.0f;
#pragma unroll
    for (int j = 0; j < kSlotGroup; ++j)
      if (j0 + j < p.slots)
        z[j] = raw_load<S>(static_cast<const TZ*>(p.z) + (int64_t)(r[j] < 0 ? 0 : r[j]) * p.ldz + col, n);
#pragma unroll
    for (int j = 0; j < kSlotGroup; ++j)
      if (j0 + j < p.slots) {
        const V8 v = raw_values(z[j], r[j] >= 0);
        const float f = r[j] >= 0 ? w[j] : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc.v[k] = __builtin_fmaf(f, v.v[k], acc.v[k]);
      }
  }
  row_store<S>(static_cast<TO*>(p.out) + t * p.ldo + col, acc, n);
}

// ------------------------------------------------------ combine's gradient
// THREADS threads (a wave or a workgroup) per token: eight columns of dout are
// held while up to kSlotGroup slots take their products with z (fp32 partial
// sums a lane, summed over lanes in a fixed order) and their rows of dz.  dout is
// read once, z and dz once a slot: 8192 tokens of 4096, 8 slots, 210 us for 1.15
// GB, 5.5 TB/s, bound by loads and stores.
template <typename TD, typename TZ, int THREADS, bool S>
__global__ __launch_bounds__(kRowThreads) void ufp4_combine_bwd_kernel(CombineBwdParams p, int64_t t0,
                                                                       uint32_t item_wgs) {
  __shared__ float part[kRowThreads / 64][kSlotGroup];
  if (blockIdx.x >= item_wgs) {
    const int64_t w = (int64_t)(blockIdx.x - item_wgs) * (kRowThreads / 64) + (threadIdx.x >> 6);
    zero_padding(p.slot_of_row, p.tokens * p.slots, w * kPadRows, p.total_rows, static_cast<TZ*>(p.dz), p.lddz,
                 p.cols);
    return;
  }
  const int lane = threadIdx.x & (THREADS - 1);
  const int64_t t = t0 + (int64_t)blockIdx.x * (kRowThreads / THREADS) + threadIdx.x / THREADS;
  const bool live = t < p.tokens;  // (every thread reaches the barriers)
  for (int j0 = 0; j0 < p.slots; j0 += kSlotGroup) {
    int32_t row[kSlotGroup];
    float w[kSlotGroup], dot[kSlotGroup];
    const int64_t tt = live ? t : 0;
    load_rows(p.row_of_slot + tt * p.slots, j0, p.slots, p.total_rows, row);
#pragma unroll
    for (int j = 0; j < kSlotGroup; ++j) {
      w[j] = p.weights ? p.weights[tt * p.slots + (j0 + j < p.slots ? j0 + j : p.slots - 1)] : 1.0f;
      dot[j] = 0.0f;
    }
    if (live)
      for (int64_t col = 8 * lane; col < p.cols; col += 8 * THREADS) {
        const int n = p.cols - col < 8 ? (int)(p.cols - col) : 8;
        typename RawOf<TZ>::type z[kSlotGroup];
        const V8 d = row_load(static_cast<const TD*>(p.d) + t * p.ldd + col, n);
        if (p.dw && p.total_rows > 0) {
#pragma unroll
          for (int j = 0; j < kSlotGroup; ++j)
            if (j0 + j < p.slots)
              z[j] = raw_load<S>(static_cast<const TZ*>(p.z) + (int64_t)(row[j] < 0 ? 0 : row[j]) * p.ldz + col, n);
#pragma unroll
          for (int j = 0; j < kSlotGroup; ++j)
            if (j0 + j < p.slots) {
              const V8 v = raw_values(z[j], row[j] >= 0);
              // (a dropped slot's sum stays 0 whatever dout holds)
#pragma unroll
              for (int k = 0; k < 8; ++k) dot[j] = row[j] >= 0 ? __builtin_fmaf(d.v[k], v.v[k], dot[j]) : 0.0f;
            }
        }
        if (p.dz) {
#pragma unroll
          for (int j = 0; j < kSlotGroup; ++j) {
            if (row[j] < 0) continue;
            V8 o;
#pragma unroll
            for (int k = 0; k < 8; ++k) o.v[k] = w[j] * d.v[k];
            row_store<S>(static_cast<TZ*>(p.dz) + (int64_t)row[j] * p.lddz + col, o, n);
          }
        }
      }
    if (!p.dw) continue;
#pragma unroll
    for (int j = 0; j < kSlotGroup; ++j)
#pragma unroll
      for (int m = 32; m >= 1; m >>= 1) dot[j] += __shfl_xor(dot[j], m);
    if (THREADS == 64) {
#pragma unroll
      for (int j = 0; j < kSlotGroup; ++j)
        if (live && lane == j && j0 + j < p.slots) p.dw[t * p.slots + j0 + j] = dot[j];
    } else {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kSlotGroup; ++j)
        if ((threadIdx.x & 63) == j) part[threadIdx.x >> 6][j] = dot[j];
      __syncthreads();
      if (live && lane < kSlotGroup && j0 + lane < p.slots) {
        float s = 0.0f;
        for (int q = 0; q < kRowThreads / 64; ++q) s += part[q][lane];
        p.dw[t * p.slots + j0 + lane] = s;
      }
    }
  }
}

uint32_t pad_wgs(int64_t rows) {
  const int64_t per = kPadRows * (kRowThreads / 64);
  return (uint32_t)((rows + per - 1) / per);
}

constexpr int64_t kMaxRowItems = (int64_t)1 << 30;
constexpr int64_t kMaxBwdTokens = (int64_t)1 << 22;  // at most one workgroup each in a launch

// Calls that move more than the last-level cache holds go past the caches:
// 8192 tokens of 4096 to 8 of 64 experts (612 MB) 128 -> 112 us (the loads stay
// cached: with them past it 125), the combination back 124 -> 111, its gradient
// (1.1 GB) 239 -> 233; half as many tokens or fewer are as fast or faster with
// the caches.
template <int FMT, bool S>
hipError_t dispatch(const DispatchParams& p, hipStream_t s) {
  const int64_t lanes = (p.cols + 7) / 8, step = kMaxRowItems / lanes;
  // slices of at most 2^30 items (31-bit item indices); the padding rows go
  // with the first
  for (int64_t t0 = 0; t0 == 0 || t0 < p.tokens; t0 += step) {
    const int64_t n = p.tokens - t0 < step ? p.tokens - t0 : step;
    const uint32_t items = (uint32_t)(n * lanes), wgs = (items + kRowThreads - 1) / kRowThreads;
    const uint32_t all = wgs + (t0 == 0 ? pad_wgs(p.total_rows) : 0);
    if (!all) return hipSuccess;
    ufp4_dispatch_kernel<FMT, S><<<all, kRowThreads, 0, s>>>(p, t0, items, wgs, fast_div((uint32_t)lanes));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename TD, typename TZ, bool S>
hipError_t combine_bwd(const CombineBwdParams& p, hipStream_t s) {
  // a wave per token up to 1024 columns (two rounds of 512), a workgroup above
  const bool wave = p.cols <= 1024;
  const int64_t per = wave ? kRowThreads / 64 : 1, step = kMaxBwdTokens;
  for (int64_t t0 = 0; t0 == 0 || t0 < p.tokens; t0 += step) {
    const int64_t n = p.tokens - t0 < step ? p.tokens - t0 : step;
    const uint32_t wgs = (uint32_t)((n + per - 1) / per);
    const uint32_t all = wgs + (p.dz && t0 == 0 ? pad_wgs(p.total_rows) : 0);
    if (!all) return hipSuccess;
    if (wave)
      ufp4_combine_bwd_kernel<TD, TZ, 64, S><<<all, kRowThreads, 0, s>>>(p, t0, wgs);
    else
      ufp4_combine_bwd_kernel<TD, TZ, kRowThreads, S><<<all, kRowThreads, 0, s>>>(p, t0, wgs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_expert_sort(const SortParams& p, hipStream_t s) {
  if (p.n <= kSortSingle) {
    ufp4_sort_single_kernel<<<1, kSortThreads, 0, s>>>(p);
    return hipGetLastError();
  }
  const int per = (((p.n + kSortBlocks - 1) / kSortBlocks) + kSortThreads - 1) / kSortThreads * kSortThreads;
  const int blocks = p.n / per;  // the last block takes the rest, so none is short
  ufp4_sort_count_kernel<<<blocks, kSortThreads, 0, s>>>(p, per);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  ufp4_sort_scan_kernel<<<1, kSortThreads, 0, s>>>(p, per, blocks);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  ufp4_sort_place_kernel<<<blocks, kSortThreads, 0, s>>>(p, per);
  return hipGetLastError();
}

namespace {

template <bool S>
hipError_t dispatch_from(const DispatchParams& p, hipStream_t s) {
  if (p.x) return dispatch<-1, S>(p, s);
  return p.format == kCkptINT8 ? dispatch<kCkptINT8, S>(p, s) : dispatch<kCkptE4M3, S>(p, s);
}

template <bool S>
hipError_t combine(const CombineParams& p, hipStream_t s) {
  const int64_t lanes = (p.cols + 7) / 8, step = kMaxRowItems / lanes;
  for (int64_t t0 = 0; t0 < p.tokens; t0 += step) {
    const int64_t n = p.tokens - t0 < step ? p.tokens - t0 : step;
    const uint32_t items = (uint32_t)(n * lanes), wgs = (items + kRowThreads - 1) / kRowThreads;
    const FastDiv d = fast_div((uint32_t)lanes);
    if (p.z_f32) {
      if (p.out_f32) ufp4_combine_kernel<float, float, S><<<wgs, kRowThreads, 0, s>>>(p, t0, items, d);
      else ufp4_combine_kernel<float, uint16_t, S><<<wgs, kRowThreads, 0, s>>>(p, t0, items, d);
    } else {
      if (p.out_f32) ufp4_combine_kernel<uint16_t, float, S><<<wgs, kRowThreads, 0, s>>>(p, t0, items, d);
      else ufp4_combine_kernel<uint16_t, uint16_t, S><<<wgs, kRowThreads, 0, s>>>(p, t0, items, d);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool S>
hipError_t combine_backward(const CombineBwdParams& p, hipStream_t s) {
  if (p.d_f32) return p.z_f32 ? combine_bwd<float, float, S>(p, s) : combine_bwd<float, uint16_t, S>(p, s);
  return p.z_f32 ? combine_bwd<uint16_t, float, S>(p, s) : combine_bwd<uint16_t, uint16_t, S>(p, s);
}

}  // namespace

hipError_t launch_expert_dispatch(const DispatchParams& p, hipStream_t s) {
  return (p.tokens + p.total_rows) * p.cols * 2 > kLastLevelCache ? dispatch_from<true>(p, s) : dispatch_from<false>(p, s);
}

hipError_t launch_expert_combine(const CombineParams& p, hipStream_t s) {
  const int64_t bytes = p.tokens * p.cols * (p.slots * (p.z_f32 ? 4 : 2) + (p.out_f32 ? 4 : 2));
  return bytes > kLastLevelCache ? combine<true>(p, s) : combine<false>(p, s);
}

hipError_t launch_expert_combine_backward(const CombineBwdParams& p, hipStream_t s) {
  const int64_t rows = p.total_rows * ((p.dz ? 1 : 0) + (p.dw ? 1 : 0));
  const int64_t bytes = p.cols * (rows * (p.z_f32 ? 4 : 2) + p.tokens * (p.d_f32 ? 4 : 2));
  return bytes > kLastLevelCache ? combine_backward<true>(p, s) : combine_backward<false>(p, s);
}

}  // namespace ufp4
