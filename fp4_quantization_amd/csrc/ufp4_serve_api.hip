// ufp4_serve_api.hip -- the C ABI of the decoding operators (include/ufp4.h):
// argument checks and launches.  Every check runs on the host before anything
// is enqueued; nothing here allocates memory or keeps state between calls.
#include "../../include/ufp4.h"
#include "ufp4_serve.hpp"

using namespace ufp4;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 25;
constexpr int64_t kMaxTokens = (int64_t)1 << 21;  // of a product: at most 2^15 blocks of 64 in y (smaller ones only below 256 workgroups)
constexpr int64_t kMaxLd = 0x7FFFFFFF;  // of a cache call's rows
constexpr int64_t kMaxRows = (int64_t)1 << 28;
constexpr int32_t kMaxSequences = 65535;  // of a launch in y
constexpr int64_t kMaxSlots64 = (int64_t)1 << 40;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool type_ok(int32_t t) { return t == UFP4_BF16 || t == UFP4_F32; }
size_t type_size(int32_t t) { return t == UFP4_F32 ? 4 : 2; }
int done(hipError_t e) { return e == hipSuccess ? UFP4_OK : UFP4_ERR_HIP; }

RhtSigns signs_of(const ufp4_config* cfg) {
  QuantParams q;
  fill_rht_signs(cfg->rht_seed, q);
  return q.sg;
}
int check_matvec(const ufp4_config* cfg, int64_t tokens, int64_t N, int64_t K) {
  if (!cfg || cfg->grid < 0 || cfg->grid > 3 || (cfg->scaling != UFP4_SCALE_NV16 && cfg->scaling != UFP4_SCALE_MX32))
    return UFP4_ERR_INVALID_ARGUMENT;
  if (tokens < 0 || N < 0 || K < 0) return UFP4_ERR_INVALID_ARGUMENT;
  if (K % 32 || tokens >= kMaxTokens || N >= kMaxDim || K >= kMaxDim) return UFP4_ERR_SHAPE;
  return UFP4_OK;
}

// Bytes of the prepared x and of the exponents behind it.  The number of parts
// depends on types the size query does not know: 3 or 2 cover all of them.
size_t matvec_x_bytes(int64_t tokens, int64_t K, int parts) {
  const size_t t16 = (size_t)(tokens + 15) / 16, chunks = (size_t)(K + kMvChunk - 1) / kMvChunk;
  return t16 * chunks * (size_t)parts * 16 * kMvChunk * 2;
}

int cache_cfg(const ufp4_config* cfg, bool append) {
  if (!cfg || cfg->grid < 0 || cfg->grid > 3 || cfg->scaling != UFP4_SCALE_NV16) return UFP4_ERR_INVALID_ARGUMENT;
  if (append && cfg->rounding != UFP4_ROUND_RTNE) return UFP4_ERR_INVALID_ARGUMENT;
  return UFP4_OK;
}

// The geometry alone (the workspace query knows no pointers).
int cache_shape(const ufp4_cache* c) {
  if (!c || c->pages < 0 || c->heads < 1 || c->heads > 1024 || c->dim < 1 || c->page_tokens < 1)
    return UFP4_ERR_INVALID_ARGUMENT;
  if (c->dim % 32 || c->dim > 256 || c->page_tokens % kCacheTile || c->page_tokens > 65536) return UFP4_ERR_SHAPE;
  if (c->pages >= kMaxSlots64 / c->page_tokens) return UFP4_ERR_SHAPE;
  return UFP4_OK;
}

int cache_view(const ufp4_cache* c, CacheView& v) {
  const int rc = cache_shape(c);
  if (rc) return rc;
  if (c->pages > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) || !aligned(c->v_scales, 16) ||
      !aligned(c->k_tensor_scale, 4) || !aligned(c->v_tensor_scale, 4))
    return UFP4_ERR_ALIGNMENT;
  v = CacheView{c->k_codes, c->k_scales, c->v_codes, c->v_scales, c->k_tensor_scale, c->v_tensor_scale,
                c->pages, c->page_tokens, c->heads, c->dim, fast_div((uint32_t)c->page_tokens)};
  return UFP4_OK;
}

// Two partial results a run.
size_t attend_ws(int runs, int rows, int dim) {
  return (size_t)runs * (sizeof(SplitUnit) + 2 * (size_t)rows * (sizeof(float2) + dim * sizeof(float)));
}

}  // namespace

extern "C" {

size_t ufp4_matvec_workspace(const ufp4_config* cfg, int64_t tokens, int64_t N, int64_t K) {
  if (check_matvec(cfg, tokens, N, K) || tokens == 0 || N == 0 || K == 0) return 0;
  const bool mx = cfg->scaling == UFP4_SCALE_MX32;
  const int parts = mx ? 3 : 2;
  if (matvec_in_lds(tokens, K, parts)) return 0;
  return matvec_x_bytes(tokens, K, parts) + (size_t)((tokens + 3) / 4 * 16);
}

int ufp4_matvec(const ufp4_config* cfg, const void* x, int32_t x_type, int64_t tokens, int64_t K, int64_t ldx,
                ufp4_qtensor w, int64_t N, void* y, int32_t y_type, int64_t ldy, void* ws, size_t ws_bytes,
                ufp4_stream_t stream) {
  const int rc = check_matvec(cfg, tokens, N, K);
  if (rc) return rc;
  if (!type_ok(x_type) || !type_ok(y_type) || ldx < K || ldy < N) return UFP4_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || N == 0) return UFP4_OK;
  const bool mx = cfg->scaling == UFP4_SCALE_MX32;
  if (!y || (K > 0 && (!x || !w.codes || !w.scales || (!mx && !w.tensor_scale)))) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(x, type_size(x_type)) || !aligned(y, type_size(y_type)) || !aligned(w.codes, 16) ||
      !aligned(w.scales, mx ? 1 : 2) || !aligned(w.tensor_scale, 4))
    return UFP4_ERR_ALIGNMENT;
  const size_t need = ufp4_matvec_workspace(cfg, tokens, N, K);
  if (need && (!ws || ws_bytes < need || !aligned(ws, 16))) return UFP4_ERR_WORKSPACE;
  MatvecParams p{};
  p.x = x;
  p.x_f32 = x_type == UFP4_F32;
  p.y_f32 = y_type == UFP4_F32;
  p.tokens = tokens;
  p.N = N;
  p.K = K;
  p.ldx = ldx;
  p.ldy = ldy;
  p.codes = w.codes;
  p.scales = w.scales;
  p.ts = mx ? nullptr : w.tensor_scale;
  p.grid = cfg->grid;
  p.mx = mx;
  p.rht = cfg->rht != 0;
  p.sg = signs_of(cfg);
  p.y = y;
  if (need) {
    p.xp = static_cast<uint16_t*>(ws);
    p.shift = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + matvec_x_bytes(tokens, K, mx ? 3 : 2));
  }
  return done(launch_matvec(p, (hipStream_t)stream));
}

int ufp4_cache_append(const ufp4_config* cfg, const ufp4_cache* cache, const uint16_t* k, int64_t ldk,
                      const uint16_t* v, int64_t ldv, int64_t tokens, const int64_t* slots, ufp4_stream_t stream) {
  int rc = cache_cfg(cfg, true);
  if (rc) return rc;
  CacheParams p{};
  rc = cache_view(cache, p.c);
  if (rc) return rc;
  const int64_t width = (int64_t)cache->heads * cache->dim;
  if (tokens < 0 || ldk < width || ldv < width) return UFP4_ERR_INVALID_ARGUMENT;
  if (tokens >= kMaxRows || ldk > kMaxLd || ldv > kMaxLd) return UFP4_ERR_SHAPE;
  if (tokens == 0) return UFP4_OK;
  if (!k || !v || !slots) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(k, 2) || !aligned(v, 2) || !aligned(slots, 8)) return UFP4_ERR_ALIGNMENT;
  p.grid = cfg->grid;
  p.rht = cfg->rht != 0;
  p.sg = signs_of(cfg);
  p.signs = rht_sign_mask(cfg->rht_seed);
  p.tokens = tokens;
  p.slots = slots;
  p.k = k;
  p.v = v;
  p.ldk = ldk;
  p.ldv = ldv;
  return done(launch_cache_append(p, (hipStream_t)stream));
}

int ufp4_cache_read(const ufp4_config* cfg, const ufp4_cache* cache, const int64_t* slots, int64_t tokens,
                    int32_t inverse_rht, void* k_out, int64_t ldk, void* v_out, int64_t ldv, int32_t out_type,
                    ufp4_stream_t stream) {
  int rc = cache_cfg(cfg, false);
  if (rc) return rc;
  CacheParams p{};
  rc = cache_view(cache, p.c);
  if (rc) return rc;
  const int64_t width = (int64_t)cache->heads * cache->dim;
  if (!type_ok(out_type) || tokens < 0 || (k_out && ldk < width) || (v_out && ldv < width))
    return UFP4_ERR_INVALID_ARGUMENT;
  if (tokens >= kMaxRows || (k_out && ldk > kMaxLd) || (v_out && ldv > kMaxLd)) return UFP4_ERR_SHAPE;
  if (tokens == 0 || (!k_out && !v_out)) return UFP4_OK;
  if (!slots) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(k_out, type_size(out_type)) || !aligned(v_out, type_size(out_type)) || !aligned(slots, 8))
    return UFP4_ERR_ALIGNMENT;
  p.grid = cfg->grid;
  p.rht = inverse_rht != 0;
  p.sg = signs_of(cfg);
  p.signs = rht_sign_mask(cfg->rht_seed);
  p.tokens = tokens;
  p.slots = slots;
  p.k_out = k_out;
  p.v_out = v_out;
  p.ldk = ldk;
  p.ldv = ldv;
  p.out_f32 = out_type == UFP4_F32;
  return done(launch_cache_read(p, (hipStream_t)stream));
}

size_t ufp4_tree_attention_workspace(const ufp4_cache* cache, int32_t q_heads, int32_t sequences, int32_t max_draft) {
  if (cache_shape(cache) || q_heads < 1 || q_heads > 8192 || q_heads % cache->heads || sequences < 0 ||
      sequences > kMaxSequences || max_draft < 1 || max_draft >= kMaxRows / q_heads)
    return 0;
  // fewer drafted tokens may take tiles of fewer rows and more runs: enough for them too
  const int group = q_heads / cache->heads, least = attend_rows(cache->dim, group, 1);
  const int rows = attend_rows(cache->dim, group, max_draft);
  const size_t few = attend_ws(attend_runs(cache->dim, least), least, cache->dim);
  const size_t all = attend_ws(attend_runs(cache->dim, rows), rows, cache->dim);
  return few > all ? few : all;
}

int ufp4_tree_attention(const ufp4_config* cfg, const ufp4_cache* cache, const uint16_t* q, int64_t ldq,
                        int32_t q_heads, const int64_t* q_offsets, int32_t sequences, int64_t q_rows,
                        int32_t max_draft, const int32_t* lengths, const int32_t* page_table, int64_t ld_pages,
                        const uint64_t* mask, float softmax_scale, uint16_t* out, int64_t ldo, float* lse, void* ws,
                        size_t ws_bytes, ufp4_stream_t stream) {
  int rc = cache_cfg(cfg, false);
  if (rc) return rc;
  AttendParams p{};
  rc = cache_view(cache, p.c);
  if (rc) return rc;
  if (q_heads < 1 || q_heads > 8192 || q_heads % cache->heads || sequences < 0 || q_rows < 0 || max_draft < 1 ||
      ld_pages < 0 || !(softmax_scale - softmax_scale == 0.0f) || (mask && max_draft > 64))
    return UFP4_ERR_INVALID_ARGUMENT;
  const int64_t width = (int64_t)q_heads * cache->dim;
  if (ldq < width || ldo < width) return UFP4_ERR_INVALID_ARGUMENT;
  if (sequences > kMaxSequences || q_rows >= kMaxRows || max_draft >= kMaxRows / q_heads ||
      ld_pages > ((int64_t)1 << 30) / cache->page_tokens)
    return UFP4_ERR_SHAPE;
  const size_t need = ufp4_tree_attention_workspace(cache, q_heads, sequences, max_draft);
  if (!need) return UFP4_ERR_SHAPE;
  if (sequences == 0 || q_rows == 0) return UFP4_OK;
  if (!q || !out || !q_offsets || !lengths || (ld_pages > 0 && !page_table)) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 2) || !aligned(out, 2) || !aligned(q_offsets, 8) || !aligned(lengths, 4) ||
      !aligned(page_table, 4) || !aligned(mask, 8) || !aligned(lse, 4))
    return UFP4_ERR_ALIGNMENT;
  if (!ws || ws_bytes < need || !aligned(ws, 16)) return UFP4_ERR_WORKSPACE;
  p.grid = cfg->grid;
  p.rht = cfg->rht != 0;
  p.signs = rht_sign_mask(cfg->rht_seed);
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.ldq = ldq;
  p.ldo = ldo;
  p.q_rows = q_rows;
  p.q_heads = q_heads;
  p.group = q_heads / cache->heads;
  p.q_offsets = q_offsets;
  p.lengths = lengths;
  p.table = page_table;
  p.ld_pages = ld_pages;
  p.sequences = sequences;
  p.max_draft = max_draft;
  p.mask = mask;
  p.scale = softmax_scale;
  const int rows = attend_rows(cache->dim, p.group, max_draft);
  p.row_tiles = (int32_t)(((int64_t)max_draft * p.group + rows - 1) / rows);
  p.max_runs = attend_runs(cache->dim, rows);
  uint8_t* at = static_cast<uint8_t*>(ws);
  p.split = reinterpret_cast<SplitUnit*>(at);
  at += (size_t)p.max_runs * sizeof(SplitUnit);
  p.ml = reinterpret_cast<float2*>(at);
  p.o = reinterpret_cast<float*>(at + (size_t)p.max_runs * 2 * rows * sizeof(float2));
  return done(launch_attend(p, (hipStream_t)stream));
}

}  // extern "C"
