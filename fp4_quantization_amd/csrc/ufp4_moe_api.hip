// ufp4_moe_api.hip -- the C ABI of the expert layer (include/ufp4.h): argument
// checks and launches.  Every check runs on the host before anything is
// enqueued; nothing here allocates memory or keeps state between calls.
#include "../../include/ufp4.h"
#include "ufp4_moe.hpp"

using namespace ufp4;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 25;
constexpr int64_t kMaxRows = (int64_t)1 << 28;  // a launch covers four threads a row
constexpr int64_t kMaxLines = (int64_t)0xFFFF * 256;  // of a grouped product's matrices

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool type_ok(int32_t t) { return t == UFP4_BF16 || t == UFP4_F32; }
size_t type_size(int32_t t) { return t == UFP4_F32 ? 4 : 2; }
bool format_ok(int32_t f) { return f == UFP4_CKPT_INT8 || f == UFP4_CKPT_E4M3; }
int done(hipError_t e) { return e == hipSuccess ? UFP4_OK : UFP4_ERR_HIP; }

// Sizes that all calls on rows share: cols below 2^25, fewer than 2^28 rows.
int check_rows(int64_t tokens, int32_t slots, int64_t total_rows, int64_t cols) {
  if (tokens < 0 || slots < 1 || slots > kMaxSlots || total_rows < 0 || cols < 0) return UFP4_ERR_INVALID_ARGUMENT;
  if (cols >= kMaxDim || total_rows >= kMaxRows || tokens >= kMaxRows || tokens * slots >= kMaxRows)
    return UFP4_ERR_SHAPE;
  return UFP4_OK;
}

int check_gemm_cfg(const ufp4_config* cfg) {
  if (!cfg || cfg->grid < 0 || cfg->grid > 3) return UFP4_ERR_INVALID_ARGUMENT;
  if (cfg->scaling != UFP4_SCALE_NV16) return UFP4_ERR_INVALID_ARGUMENT;
  return UFP4_OK;
}

int dispatch_args(DispatchParams& p, int64_t tokens, int64_t cols, int32_t slots, const int32_t* row_of_slot,
                  const int32_t* slot_of_row, int64_t total_rows, uint16_t* out, int64_t ldo) {
  const int rc = check_rows(tokens, slots, total_rows, cols);
  if (rc) return rc;
  if (ldo < cols) return UFP4_ERR_INVALID_ARGUMENT;
  if ((tokens > 0 && !row_of_slot) || (total_rows > 0 && (!slot_of_row || (cols > 0 && !out))))
    return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(row_of_slot, 4) || !aligned(slot_of_row, 4) || !aligned(out, 2)) return UFP4_ERR_ALIGNMENT;
  p.tokens = tokens;
  p.cols = cols;
  p.slots = slots;
  p.row_of_slot = row_of_slot;
  p.slot_of_row = slot_of_row;
  p.total_rows = total_rows;
  p.out = out;
  p.ldo = ldo;
  return UFP4_OK;
}

int grouped_operand(const ufp4_qtensor& q, size_t code_align, bool empty) {
  if (!q.tensor_scale) return UFP4_ERR_INVALID_ARGUMENT;
  if (!empty && (!q.codes || !q.scales)) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(q.codes, code_align) || !aligned(q.scales, 2) || !aligned(q.tensor_scale, 4)) return UFP4_ERR_ALIGNMENT;
  return UFP4_OK;
}

GroupedOperand operand(const ufp4_qtensor& q, int64_t pitch, int64_t seg_lines, int64_t seg_k) {
  return GroupedOperand{q.codes, q.scales, q.tensor_scale, pitch, seg_lines, seg_k};
}

}  // namespace

extern "C" {

int64_t ufp4_expert_rows(int64_t tokens, int32_t slots, int32_t num_experts, int32_t align) {
  if (tokens < 0 || tokens >= kMaxRows || slots < 1 || slots > kMaxSlots || num_experts < 1 ||
      num_experts > kMaxExperts || align < 1 || align > kMaxAlign)
    return 0;
  const int64_t n = tokens * slots, used = n < num_experts ? n : num_experts;
  return (n + used * (align - 1) + align - 1) / align * align;
}

int ufp4_expert_sort(const int32_t* ids, int64_t tokens, int32_t slots, int64_t ld_ids, int32_t num_experts,
                     int32_t align, int64_t total_rows, int64_t* offsets, int32_t* row_of_slot,
                     int32_t* slot_of_row, ufp4_stream_t stream) {
  const int rc = check_rows(tokens, slots, total_rows, 0);
  if (rc) return rc;
  if (num_experts < 1 || num_experts > kMaxExperts || align < 1 || align > kMaxAlign || ld_ids < slots)
    return UFP4_ERR_INVALID_ARGUMENT;
  if (total_rows < ufp4_expert_rows(tokens, slots, num_experts, align)) return UFP4_ERR_SHAPE;
  if (!offsets || (tokens > 0 && (!ids || !row_of_slot)) || (total_rows > 0 && !slot_of_row))
    return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(ids, 4) || !aligned(offsets, 8) || !aligned(row_of_slot, 4) || !aligned(slot_of_row, 4))
    return UFP4_ERR_ALIGNMENT;
  SortParams p;
  p.ids = ids;
  p.ld_ids = ld_ids;
  p.n = (int32_t)(tokens * slots);
  p.slots = fast_div((uint32_t)slots);
  p.experts = num_experts;
  p.align = align;
  p.total_rows = (int32_t)total_rows;
  p.offsets = offsets;
  p.row_of_slot = row_of_slot;
  p.slot_of_row = slot_of_row;
  return done(launch_expert_sort(p, (hipStream_t)stream));
}

int ufp4_expert_dispatch(const uint16_t* x, int64_t tokens, int64_t cols, int64_t ld, int32_t slots,
                         const int32_t* row_of_slot, const int32_t* slot_of_row, int64_t total_rows, uint16_t* out,
                         int64_t ldo, ufp4_stream_t stream) {
  DispatchParams p{};
  const int rc = dispatch_args(p, tokens, cols, slots, row_of_slot, slot_of_row, total_rows, out, ldo);
  if (rc) return rc;
  if (ld < cols) return UFP4_ERR_INVALID_ARGUMENT;
  if (cols == 0 || total_rows == 0) return UFP4_OK;
  if (tokens > 0 && !x) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 2)) return UFP4_ERR_ALIGNMENT;
  p.x = x;
  p.ld = ld;
  return done(launch_expert_dispatch(p, (hipStream_t)stream));
}

int ufp4_expert_dispatch_checkpoint(const uint8_t* codes, const uint16_t* scales, int32_t format, int64_t tokens,
                                    int64_t cols, int32_t slots, const int32_t* row_of_slot,
                                    const int32_t* slot_of_row, int64_t total_rows, uint16_t* out, int64_t ldo,
                                    ufp4_stream_t stream) {
  DispatchParams p{};
  const int rc = dispatch_args(p, tokens, cols, slots, row_of_slot, slot_of_row, total_rows, out, ldo);
  if (rc) return rc;
  if (!format_ok(format)) return UFP4_ERR_INVALID_ARGUMENT;
  if (cols == 0 || total_rows == 0) return UFP4_OK;
  if (tokens > 0 && (!codes || !scales)) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(scales, 2)) return UFP4_ERR_ALIGNMENT;
  p.codes = codes;
  p.scales = scales;
  p.format = format;
  return done(launch_expert_dispatch(p, (hipStream_t)stream));
}

int ufp4_expert_combine(const void* z, int32_t z_type, int64_t total_rows, int64_t cols, int64_t ldz,
                        const int32_t* row_of_slot, const float* weights, int64_t tokens, int32_t slots, void* out,
                        int32_t out_type, int64_t ldo, ufp4_stream_t stream) {
  const int rc = check_rows(tokens, slots, total_rows, cols);
  if (rc) return rc;
  if (!type_ok(z_type) || !type_ok(out_type) || ldz < cols || ldo < cols) return UFP4_ERR_INVALID_ARGUMENT;
  if (tokens == 0 || cols == 0) return UFP4_OK;
  if (!out || !row_of_slot || (total_rows > 0 && !z)) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(z, type_size(z_type)) || !aligned(out, type_size(out_type)) || !aligned(row_of_slot, 4) ||
      !aligned(weights, 4))
    return UFP4_ERR_ALIGNMENT;
  CombineParams p;
  p.z = z;
  p.z_f32 = z_type == UFP4_F32;
  p.out_f32 = out_type == UFP4_F32;
  p.total_rows = total_rows;
  p.cols = cols;
  p.ldz = ldz;
  p.row_of_slot = row_of_slot;
  p.weights = weights;
  p.tokens = tokens;
  p.slots = slots;
  p.out = out;
  p.ldo = ldo;
  return done(launch_expert_combine(p, (hipStream_t)stream));
}

int ufp4_expert_combine_backward(const void* dout, int32_t d_type, int64_t tokens, int64_t cols, int64_t ldd,
                                 int32_t slots, const void* z, int32_t z_type, int64_t total_rows, int64_t ldz,
                                 const int32_t* row_of_slot, const int32_t* slot_of_row, const float* weights,
                                 void* dz, int64_t lddz, float* dweights, ufp4_stream_t stream) {
  const int rc = check_rows(tokens, slots, total_rows, cols);
  if (rc) return rc;
  if (!type_ok(d_type) || !type_ok(z_type) || ldd < cols) return UFP4_ERR_INVALID_ARGUMENT;
  if ((dweights && ldz < cols) || (dz && lddz < cols)) return UFP4_ERR_INVALID_ARGUMENT;
  if (!dz && !dweights) return UFP4_OK;
  if (tokens > 0 && (!row_of_slot || (cols > 0 && !dout))) return UFP4_ERR_INVALID_ARGUMENT;
  if (dweights && tokens > 0 && total_rows > 0 && cols > 0 && !z) return UFP4_ERR_INVALID_ARGUMENT;
  if (dz && total_rows > 0 && !slot_of_row) return UFP4_ERR_INVALID_ARGUMENT;
  const size_t zs = type_size(z_type);
  if (!aligned(dout, type_size(d_type)) || !aligned(z, zs) || !aligned(dz, zs) || !aligned(row_of_slot, 4) ||
      !aligned(slot_of_row, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
    return UFP4_ERR_ALIGNMENT;
  CombineBwdParams p;
  p.d = dout;
  p.d_f32 = d_type == UFP4_F32;
  p.z_f32 = z_type == UFP4_F32;
  p.tokens = tokens;
  p.cols = cols;
  p.ldd = ldd;
  p.slots = slots;
  p.z = z;
  p.total_rows = total_rows;
  p.ldz = ldz;
  p.row_of_slot = row_of_slot;
  p.slot_of_row = slot_of_row;
  p.weights = weights;
  p.dz = dz;
  p.lddz = lddz;
  p.dw = dweights;
  return done(launch_expert_combine_backward(p, (hipStream_t)stream));
}

int ufp4_checkpoint_save(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, int32_t format, uint8_t* codes,
                         uint16_t* scales, ufp4_stream_t stream) {
  if (rows < 0 || cols < 0 || ld < cols || !format_ok(format)) return UFP4_ERR_INVALID_ARGUMENT;
  if (cols >= kMaxDim || rows >= kMaxRows) return UFP4_ERR_SHAPE;
  if (rows == 0 || cols == 0) return UFP4_OK;
  if (!x || !codes || !scales) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 2) || !aligned(scales, 2)) return UFP4_ERR_ALIGNMENT;
  CkptParams p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.ld = ld;
  p.format = format;
  p.codes = codes;
  p.scales = scales;
  return done(launch_ckpt_save(p, (hipStream_t)stream));
}

int ufp4_checkpoint_load(const uint8_t* codes, const uint16_t* scales, int64_t rows, int64_t cols, int32_t format,
                         void* out, int32_t out_type, int64_t ldo, ufp4_stream_t stream) {
  if (rows < 0 || cols < 0 || ldo < cols || !format_ok(format) || !type_ok(out_type)) return UFP4_ERR_INVALID_ARGUMENT;
  if (cols >= kMaxDim || rows >= kMaxRows) return UFP4_ERR_SHAPE;
  if (rows == 0 || cols == 0) return UFP4_OK;
  if (!out || !codes || !scales) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(out, type_size(out_type)) || !aligned(scales, 2)) return UFP4_ERR_ALIGNMENT;
  CkptParams p{};
  p.rows = rows;
  p.cols = cols;
  p.format = format;
  p.out_f32 = out_type == UFP4_F32;
  p.codes = const_cast<uint8_t*>(codes);
  p.scales = const_cast<uint16_t*>(scales);
  p.out = out;
  p.ldo = ldo;
  return done(launch_ckpt_load(p, (hipStream_t)stream));
}

int ufp4_gated_act(const uint16_t* gu, int64_t rows, int64_t width, int64_t ld, int32_t act, uint16_t* h, int64_t ldh,
                   int32_t format, uint8_t* codes, uint16_t* scales, ufp4_stream_t stream) {
  if (rows < 0 || width < 0 || act < 0 || act > 1 || !format_ok(format)) return UFP4_ERR_INVALID_ARGUMENT;
  if (width >= kMaxDim / 2 || rows >= kMaxRows) return UFP4_ERR_SHAPE;
  if (ld < 2 * width || ldh < width) return UFP4_ERR_INVALID_ARGUMENT;
  if (!codes != !scales) return UFP4_ERR_INVALID_ARGUMENT;
  if (rows == 0 || width == 0) return UFP4_OK;
  if (!gu || !h) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(gu, 2) || !aligned(h, 2) || !aligned(scales, 2)) return UFP4_ERR_ALIGNMENT;
  GatedParams p{};
  p.in = gu;
  p.ld_in = ld;
  p.rows = rows;
  p.width = width;
  p.act = act;
  p.format = format;
  p.codes = codes;
  p.scales = scales;
  p.h = h;
  p.ldh = ldh;
  return done(launch_gated(p, (hipStream_t)stream));
}

int ufp4_gated_act_backward(const uint16_t* dh, int64_t lddh, const uint8_t* codes, const uint16_t* scales,
                            int32_t format, int64_t rows, int64_t width, int32_t act, uint16_t* dgu, int64_t lddg,
                            uint16_t* h_out, int64_t ldho, ufp4_stream_t stream) {
  if (rows < 0 || width < 0 || act < 0 || act > 1 || !format_ok(format)) return UFP4_ERR_INVALID_ARGUMENT;
  if (width >= kMaxDim / 2 || rows >= kMaxRows) return UFP4_ERR_SHAPE;
  if (lddh < width || lddg < 2 * width || (h_out && ldho < width)) return UFP4_ERR_INVALID_ARGUMENT;
  if (rows == 0 || width == 0) return UFP4_OK;
  if (!dh || !codes || !scales || !dgu) return UFP4_ERR_INVALID_ARGUMENT;
  if (!aligned(dh, 2) || !aligned(dgu, 2) || !aligned(h_out, 2) || !aligned(scales, 2)) return UFP4_ERR_ALIGNMENT;
  GatedParams p{};
  p.in = dh;
  p.ld_in = lddh;
  p.rows = rows;
  p.width = width;
  p.act = act;
  p.format = format;
  p.codes = const_cast<uint8_t*>(codes);
  p.scales = const_cast<uint16_t*>(scales);
  p.h = h_out;
  p.ldh = ldho;
  p.dgu = dgu;
  p.lddg = lddg;
  return done(launch_gated_backward(p, (hipStream_t)stream));
}

int ufp4_gemm_grouped_nt(const ufp4_config* cfg, int64_t total_rows, int64_t N, int64_t K, ufp4_qtensor a,
                         ufp4_qtensor b, int32_t b_layout, const int64_t* offsets_dev, int32_t num_groups, void* c,
                         int32_t c_type, int64_t ldc, ufp4_stream_t stream) {
  int rc = check_gemm_cfg(cfg);
  if (rc) return rc;
  if (total_rows < 0 || N < 0 || K < 0 || ldc < N || num_groups < 1 || num_groups > 1024 || !type_ok(c_type) ||
      (b_layout != 0 && b_layout != 1))
    return UFP4_ERR_INVALID_ARGUMENT;
  if (K % 32 || K >= kMaxDim || (b_layout == 1 && K * num_groups >= kMaxDim) || N > kMaxLines || total_rows >= kMaxDim) return UFP4_ERR_SHAPE;
  if (total_rows == 0 || N == 0) return UFP4_OK;
  if (!c || !offsets_dev) return UFP4_ERR_INVALID_ARGUMENT;
  if ((rc = grouped_operand(a, 16, K == 0)) || (rc = grouped_operand(b, 16, K == 0))) return rc;
  if (!aligned(c, type_size(c_type)) || !aligned(offsets_dev, 8)) return UFP4_ERR_ALIGNMENT;
  GroupedParams p{};
  p.a = operand(a, K, 0, 0);
  p.b = b_layout == 0 ? operand(b, K, N, 0) : operand(b, K * num_groups, 0, K);
  p.offsets = offsets_dev;
  p.groups = num_groups;
  p.grid = cfg->grid;
  p.c_f32 = c_type == UFP4_F32;
  p.total_rows = total_rows;
  p.N = N;
  p.K = K;
  p.c = c;
  p.ldc = ldc;
  if (grouped_tiles(p, false) >> 31) return UFP4_ERR_SHAPE;
  return done(launch_grouped_nt(p, (hipStream_t)stream));
}

int ufp4_gemm_grouped_dw(const ufp4_config* cfg, int64_t M, int64_t N, int64_t padded_rows, ufp4_qtensor a,
                         ufp4_qtensor b, const int64_t* offsets_dev, int32_t num_groups, void* c, int32_t c_type,
                         ufp4_stream_t stream) {
  int rc = check_gemm_cfg(cfg);
  if (rc) return rc;
  if (M < 0 || N < 0 || padded_rows < 0 || num_groups < 1 || num_groups > 1024 || !type_ok(c_type))
    return UFP4_ERR_INVALID_ARGUMENT;
  if (padded_rows % 16 || M > kMaxLines || N > kMaxLines || padded_rows >= kMaxDim) return UFP4_ERR_SHAPE;
  if (M == 0 || N == 0) return UFP4_OK;
  if (!c || !offsets_dev) return UFP4_ERR_INVALID_ARGUMENT;
  if ((rc = grouped_operand(a, 16, padded_rows == 0)) || (rc = grouped_operand(b, 16, padded_rows == 0))) return rc;
  if (!aligned(c, type_size(c_type)) || !aligned(offsets_dev, 8)) return UFP4_ERR_ALIGNMENT;
  GroupedParams p{};
  p.a = operand(a, padded_rows, 0, 0);
  p.b = operand(b, padded_rows, 0, 0);
  p.offsets = offsets_dev;
  p.groups = num_groups;
  p.grid = cfg->grid;
  p.c_f32 = c_type == UFP4_F32;
  p.total_rows = padded_rows;
  p.M = M;
  p.N = N;
  p.c = c;
  p.ldc = N;
  if (grouped_tiles(p, true) >> 31) return UFP4_ERR_SHAPE;
  return done(launch_grouped_dw(p, (hipStream_t)stream));
}

}  // extern "C"
