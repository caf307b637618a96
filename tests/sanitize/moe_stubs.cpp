// moe_stubs.cpp -- stand-ins for the expert layer's kernel launchers, linked
// instead of the device code into a sanitized host build of its C ABI.  Each
// checks the parameter block the ABI prepared and returns success.
#include <stdio.h>
#include <stdlib.h>

#include "../../fp4_quantization_amd/csrc/ufp4_moe.hpp"

namespace ufp4 {

int g_moe_calls = 0;

static void require(bool ok, const char* what) {
  if (!ok) {
    fprintf(stderr, "moe stub: %s\n", what);
    abort();
  }
}

hipError_t launch_expert_sort(const SortParams& p, hipStream_t) {
  ++g_moe_calls;
  require(p.offsets && p.experts >= 1 && p.experts <= kMaxExperts && p.align >= 1, "sort");
  require(p.n == 0 || (p.ids && p.row_of_slot), "sort slots");
  require(p.total_rows >= p.n && (p.total_rows == 0 || p.slot_of_row), "sort rows");
  for (uint32_t n : {0u, 1u, 7u, 1023u, 65536u, 0x7FFFFFFFu}) require(p.slots.div(n) == n / p.slots.d, "slot division");
  return hipSuccess;
}
hipError_t launch_expert_dispatch(const DispatchParams& p, hipStream_t) {
  ++g_moe_calls;
  require(p.cols > 0 && p.total_rows > 0 && p.out && p.slot_of_row && p.ldo >= p.cols, "dispatch");
  require(p.tokens == 0 || (p.row_of_slot && (p.x ? p.ld >= p.cols : p.codes && p.scales)), "dispatch source");
  return hipSuccess;
}
hipError_t launch_expert_combine(const CombineParams& p, hipStream_t) {
  ++g_moe_calls;
  require(p.cols > 0 && p.tokens > 0 && p.out && p.row_of_slot && (p.total_rows == 0 || p.z), "combine");
  return hipSuccess;
}
hipError_t launch_expert_combine_backward(const CombineBwdParams& p, hipStream_t) {
  ++g_moe_calls;
  require((p.dz || p.dw) && (!p.dz || p.total_rows == 0 || p.slot_of_row), "combine backward");
  return hipSuccess;
}
static hipError_t ckpt(const CkptParams& p, bool load) {
  ++g_moe_calls;
  require(p.rows > 0 && p.cols > 0 && p.codes && p.scales && (load ? p.out != nullptr : p.x != nullptr), "checkpoint");
  return hipSuccess;
}
hipError_t launch_ckpt_save(const CkptParams& p, hipStream_t) { return ckpt(p, false); }
hipError_t launch_ckpt_load(const CkptParams& p, hipStream_t) { return ckpt(p, true); }
hipError_t launch_gated(const GatedParams& p, hipStream_t) {
  ++g_moe_calls;
  require(p.rows > 0 && p.width > 0 && p.in && p.h && !p.codes == !p.scales, "gated");
  return hipSuccess;
}
hipError_t launch_gated_backward(const GatedParams& p, hipStream_t) {
  ++g_moe_calls;
  require(p.rows > 0 && p.width > 0 && p.in && p.codes && p.scales && p.dgu, "gated backward");
  return hipSuccess;
}
int64_t grouped_tiles(const GroupedParams& p, bool dw) {
  return (p.N + 255) / 256 * (dw ? (p.M + 255) / 256 * p.groups : p.total_rows / 256 + p.groups + 1);
}
static hipError_t grouped(const GroupedParams& p, bool dw) {
  ++g_moe_calls;
  require(p.N > 0 && p.c && p.offsets && p.groups >= 1 && p.groups <= 1024 && p.ldc >= p.N, "grouped");
  require(dw ? p.M > 0 && p.total_rows % 16 == 0 : p.K % 32 == 0 && p.total_rows > 0, "grouped shape");
  require(p.a.pitch < (1 << 25) && p.b.pitch < (1 << 25), "line length");
  return hipSuccess;
}
hipError_t launch_grouped_nt(const GroupedParams& p, hipStream_t) { return grouped(p, false); }
hipError_t launch_grouped_dw(const GroupedParams& p, hipStream_t) { return grouped(p, true); }

}  // namespace ufp4
